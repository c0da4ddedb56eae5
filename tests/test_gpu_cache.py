"""The page operations of the cache against plain Python, and a run of them with
the attention that reads the cache."""
import pytest
import torch

import cascade_paged_attention_gb300 as cpa
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fork_ref(table, lens, parents, children, refs, P):
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    free = iter([p for p, c in enumerate(refs) if c == 0])
    src, dst = [], []
    for r, c in zip(parents, children):
        L = lens[r]
        row = [-1] * len(table[0])
        for k in range(L // P):
            row[k] = table[r][k]
            refs[row[k]] += 1
        pair = (-1, -1)
        if L % P:
            new = next(free)
            row[L // P] = new
            refs[new] = 1
            pair = (table[r][L // P], new)
        table[c], lens[c] = row, L
        src.append(pair[0])
        dst.append(pair[1])
    return table, lens, refs, src, dst


def counts_of(table, pool):
    n = torch.zeros(pool, dtype=torch.int32, device="cuda")
    flat = table[table >= 0].long()
    return n.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))


@pytest.mark.parametrize("lens,fan,P,spare", [([1], 1, 8, 1), ([16], 3, 16, 0), ([17], 4, 16, 9),
                                             ([0, 5, 32, 100], 3, 16, 20), ([777], 600, 8, 900),
                                             (list(range(1, 70)), 4, 32, 9000), ([5000, 3], 2, 64, 40)])
def test_fork(lens, fan, P, spare):
    g = ref.gen(len(lens))
    table, pool = ref.table_of(lens, P, g, spare)
    refs = counts_of(table, pool)
    n = len(lens) * fan
    rows = torch.cat([table, torch.randint(-5, 5, (n + 2, table.shape[1]), generator=g,
                                           device="cuda").to(torch.int32)])
    dl = torch.cat([i32(lens), torch.full((n + 2,), 9, dtype=torch.int32, device="cuda")])
    parents = [i % len(lens) for i in range(n)]
    children = [len(lens) + n - i for i in range(n)]  # (the first and last rows stay)
    want = fork_ref(rows.tolist(), dl.tolist(), parents, children, refs.tolist(), P)
    before = rows.clone()
    src, dst = cpa.cpa_cache_fork(rows, dl, i32(parents), i32(children), refs, P, check=True)
    assert rows.tolist() == want[0] and dl.tolist() == want[1] and refs.tolist() == want[2]
    assert src.tolist() == want[3] and dst.tolist() == want[4]
    assert torch.equal(rows[len(lens)], before[len(lens)]) and torch.equal(rows[-1], before[-1])
    # giving the children back restores the counts
    cpa.cpa_cache_free(rows, i32(children), i32([0] * n), i32([rows.shape[1]] * n), refs, check=True)
    assert torch.equal(refs, counts_of(table, pool))
    assert bool((rows[i32(children).long()] == -1).all())


def test_fork_with_too_few_pages():
    """The children without a page have -1 there, all else is done, and freeing undoes it."""
    table, pool = ref.table_of([40, 8], 16, ref.gen(1), 2)
    refs = counts_of(table, pool)
    before = refs.clone()
    rows = torch.cat([table, torch.zeros(4, table.shape[1], dtype=torch.int32, device="cuda")])
    dl = i32([40, 8, 1, 1, 1, 1])
    ws = torch.empty(cpa.cpa_cache_fork_workspace_size(pool), dtype=torch.uint8, device="cuda")
    src, dst = cpa.cpa_cache_fork(rows, dl, i32([0, 1, 0, 1]), i32([2, 3, 4, 5]), refs, 16,
                                  workspace=ws)
    st, word = cpa.cpa_get_device_status(ws)
    assert st == 11 and word == 0x20
    free = [p for p in range(pool) if int(before[p]) == 0]
    assert dst.tolist() == free + [-1, -1] and src.tolist()[2:] == [-1, -1]
    assert rows[4].tolist() == table[0, :2].tolist() + [-1] and rows[5].tolist() == [-1, -1, -1]
    assert dl.tolist() == [40, 8, 40, 8, 40, 8]
    cpa.cpa_cache_free(rows, i32([2, 3, 4, 5]), i32([0] * 4), i32([3] * 4), refs, check=True)
    assert torch.equal(refs, before)


def test_fork_refuses_rows_that_collide():
    table, pool = ref.table_of([20, 20], 16, ref.gen(2), 8)
    for parents, children in (([0, 1], [2, 2]), ([0, 2], [2, 3]), ([0, 0], [0, 2]), ([4, 0], [2, 3]),
                              ([-1, 0], [2, 3]), ([0, 0], [4, 2]), ([0, 0], [-1, 2])):
        rows = torch.cat([table, torch.full((2, 2), 77, dtype=torch.int32, device="cuda")])
        refs, dl = counts_of(table, pool), i32([20, 20, 7, 7])
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_cache_fork(rows, dl, i32(parents), i32(children), refs, 16, check=True)
        assert e.value.status == 10
        assert torch.equal(rows[:2], table) and dl[:2].tolist() == [20, 20]
    rows = torch.cat([table, table])
    dl = i32([20, 33, 20, 20])
    refs = counts_of(table, pool)
    with pytest.raises(cpa.CpaError) as e:
        cpa.cpa_cache_fork(rows, dl, i32([1]), i32([2]), refs, 16, check=True)
    assert e.value.status == 8
    rows[0, 0] = pool
    with pytest.raises(cpa.CpaError) as e:
        cpa.cpa_cache_fork(rows, dl, i32([0]), i32([2]), refs, 16, check=True)
    assert e.value.status == 5


def test_free_ranges_shared_pages_and_bad_calls():
    """Pages of three rows that share some; ranges; an entry named twice counts once."""
    table = i32([[0, 1, 2, 3, -1], [0, 1, 4, -1, -1], [0, 5, 6, 7, 8]])
    refs = counts_of(table, 10)
    cpa.cpa_cache_free(table, i32([0, 2, 2, 1]), i32([1, 0, 1, 0]), i32([3, 2, 4, 0]), refs,
                       check=True)
    assert table.tolist() == [[0, -1, -1, 3, -1], [0, 1, 4, -1, -1], [-1, -1, -1, -1, 8]]
    assert torch.equal(refs, counts_of(table, 10))
    for rows, first, last, status in (([3], [0], [1], 10), ([-1], [0], [1], 10), ([0], [-1], [1], 8),
                                      ([0], [0], [6], 8)):
        before, was = table.clone(), refs.clone()
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_cache_free(table, i32(rows), i32(first), i32(last), refs, check=True)
        assert e.value.status == status
        assert torch.equal(table, before) and torch.equal(refs, was)
    cpa.cpa_cache_free(table, i32([1]), i32([4]), i32([1]), refs, check=True)  # an empty range
    refs[4] = 0
    with pytest.raises(cpa.CpaError) as e:
        cpa.cpa_cache_free(table, i32([1]), i32([2]), i32([3]), refs, check=True)
    assert e.value.status == 12 and int(refs[4]) == 0
    table[1, 0] = 10
    with pytest.raises(cpa.CpaError) as e:
        cpa.cpa_cache_free(table, i32([1]), i32([0]), i32([1]), refs, check=True)
    assert e.value.status == 5


@pytest.mark.parametrize("n,P,H_kv,dtype", [(1, 8, 1, torch.uint8), (3, 16, 8, torch.bfloat16),
                                           (700, 16, 2, torch.bfloat16), (33, 256, 8, torch.uint8),
                                           (0, 16, 1, torch.bfloat16), (5, 8, 3, torch.bfloat16)])
def test_copy_pages(n, P, H_kv, dtype):
    g = ref.gen(n)
    pool = 2 * n + 3
    k, v = (torch.randint(0, 255, (pool, P, H_kv, 128), generator=g, device="cuda").to(dtype)
            for _ in range(2))
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:n].contiguous(), perm[n:2 * n].contiguous()
    if n > 2:  # a source may serve twice, and a pair of -1 is passed over
        src[1] = src[0]
        src[2] = dst[2] = -1
    want_k, want_v = k.clone(), v.clone()
    ok = dst >= 0
    want_k[dst[ok].long()] = k[src[ok].long()]
    want_v[dst[ok].long()] = v[src[ok].long()]
    cpa.cpa_cache_copy_pages(k, v, src, dst, check=True)
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_copy_pages_reports_bad_pairs():
    k = torch.zeros(4, 8, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    for s, d in ((0, 4), (4, 0), (-1, 0), (0, -1), (-2, -2), (2 ** 31 - 1, 0)):
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_cache_copy_pages(k, v, i32([1, s]), i32([2, d]), check=True)
        assert e.value.status == 5
    assert bool((k == 0).all()) and bool((v == 1).all())


@pytest.mark.parametrize("P,H_kv,dtype", [(16, 8, torch.bfloat16), (8, 1, torch.uint8),
                                         (64, 3, torch.bfloat16), (256, 2, torch.uint8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(P, H_kv, dtype, in_place):
    g = ref.gen(P)
    B, span = 5, 3 * P + 5
    keep = [0, 1, 2, span // 2, span]
    start = [3, 0, 1, 0, 0] if in_place else [P - 1, 0, 7, 2 * P + 1, 3]
    table, pool = ref.table_of([span] * B + [s + n for s, n in zip(start, keep)], P, g)
    rows = i32([4, 2, 0, 1, 3])
    k, v = (torch.randint(0, 255, (pool, P, H_kv, 128), generator=g, device="cuda").to(dtype)
            for _ in range(2))
    pos = torch.zeros(B, span, dtype=torch.int32, device="cuda")
    for b in range(B):
        p = torch.randperm(span - start[b] if in_place else span, generator=g, device="cuda")[:keep[b]]
        pos[b, :keep[b]] = (p.sort().values if in_place else p) + (start[b] if in_place else 0)
    src_t, dst_t = table[:B].contiguous(), table[B:].contiguous()
    want = [x.clone() for x in (k, v)]
    for x, y in zip(want, (k, v)):
        for b in range(B):
            for i in range(keep[b]):
                a, z = int(pos[b, i]), start[b] + i
                srow = src_t[int(rows[b])]
                drow = srow if in_place else dst_t[b]
                x[int(drow[z // P]), z % P] = y[int(srow[a // P]), a % P]
    cpa.cpa_cache_compact(k, v, src_t, pos, i32(keep), None if in_place else dst_t, i32(start),
                          src_rows=rows, check=True)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_compact_of_many_tokens_and_its_report():
    """Past the size at which one block looks the call over: every warp reports for itself."""
    g = ref.gen(9)
    B, span, P = 9, 600, 16
    keep = [500 - 7 * b for b in range(B)]
    table, pool = ref.table_of([span] * B + keep, P, g)
    k, v = ref.pool_of(pool, P, 2, g), ref.pool_of(pool, P, 2, g)
    src, dst = table[:B].contiguous(), table[B:, :32].contiguous()
    pos = torch.stack([torch.randperm(span, generator=g, device="cuda")[:500] for _ in range(B)])
    want = []
    for x in (k, v):
        y = x.clone().view(-1, 2, 128)
        for b in range(B):
            a, z = pos[b, :keep[b]], torch.arange(keep[b], device="cuda")
            y[dst[b].long()[z // P] * P + z % P] = x.view(-1, 2, 128)[src[b].long()[a // P] * P + a % P]
        want.append(y.view_as(x))
    pos = pos.to(torch.int32).contiguous()
    cpa.cpa_cache_compact(k, v, src, pos, i32(keep), dst, i32([0] * B), check=True)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    bad_pos, bad_src = pos.clone(), src.clone()
    bad_pos[8, 3] = span + 40
    bad_src[8] = pool
    for s, p, status in ((src, bad_pos, 8), (bad_src, pos, 5)):
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_cache_compact(k, v, s, p, i32(keep), dst, i32([0] * B), check=True)
        assert e.value.status == status


def test_compact_reports_bad_calls():
    k = torch.zeros(8, 8, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    src, dst = i32([[0, 1], [2, 3]]), i32([[4, 5], [6, 7]])
    pos, keep, start = i32([[0, 9], [3, 4]]), i32([2, 2]), i32([0, 3])

    def status(**kw):
        a = dict(src=src, pos=pos, keep=keep, dst=dst, start=start, rows=None)
        a.update(kw)
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        cpa.cpa_cache_compact(k, v, a["src"], a["pos"], a["keep"], a["dst"], a["start"],
                              src_rows=a["rows"], workspace=ws)
        return cpa.cpa_get_device_status(ws)[0]

    assert status() == 0
    assert status(pos=i32([[0, 16], [3, 4]])) == 8
    assert status(pos=i32([[0, -1], [3, 4]])) == 8
    assert status(keep=i32([2, 3])) == 8 and status(keep=i32([-1, 2])) == 8
    assert status(start=i32([0, 15])) == 8 and status(start=i32([-1, 0])) == 8
    assert status(start=i32([0, 2 ** 31 - 1])) == 8
    assert status(rows=i32([0, 2])) == 10 and status(rows=i32([-1, 0])) == 10
    assert status(src=i32([[0, 8], [2, 3]])) == 5 and status(dst=i32([[4, 5], [-1, 7]])) == 5
    assert status(dst=None) == 0
    assert status(dst=None, pos=i32([[4, 4], [3, 4]])) == 8  # not ascending
    assert status(dst=None, start=i32([0, 4])) == 8          # upwards


def test_offsets_past_32_bits():
    """Slots beyond 2^31 bytes and 2^32 elements of a pool are reached (copy, compact, decode)."""
    pool, P, H_kv = 300_000, 16, 8  # 9.8 GB a pool, 4.9e9 elements
    k = torch.zeros(pool, P, H_kv, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[5].normal_()
    v[5].normal_()
    cpa.cpa_cache_copy_pages(k, v, i32([5]), i32([pool - 1]), check=True)
    assert torch.equal(k[-1], k[5]) and torch.equal(v[-1], v[5])
    table = i32([[pool - 2]])
    cpa.cpa_cache_compact(k, v, i32([[pool - 1]]), i32([[1, 3, 4]]), i32([3]), table, i32([2]),
                          check=True)
    assert torch.equal(k[-2, 2:5], k[5, [1, 3, 4]]) and torch.equal(v[-2, 2:5], v[5, [1, 3, 4]])
    q = torch.randn(1, 32, 128, device="cuda").to(torch.bfloat16)
    o, lse = cpa.cpa_decode(q, k, v, i32([[pool - 1, pool - 2]]), i32([21]), check=True)
    K = torch.cat([k[-1], k[-2]])[:21].double()
    V = torch.cat([v[-1], v[-2]])[:21].double()
    ref.close(o, lse, ref.attend(q, K, V, ref.seen([20], 21, 0, 0, "cuda"), 128 ** -0.5))
    qs = torch.randn(5, 32, 128, device="cuda").to(torch.bfloat16)
    o, lse = cpa.cpa_window_prefill(qs, k, v, i32([[pool - 1, pool - 2]]), i32([0, 5]), i32([21]),
                                    check=True)
    ref.close(o, lse, ref.attend(qs, K, V, ref.seen(range(16, 21), 21, 0, 0, "cuda"), 128 ** -0.5,
                                 ref.E_P_BF16))


def test_a_conversation():
    """Prefill a prompt, fork it, decode the branches with a token of their own each, give back
    what the window left, verify a draft and move it behind the prefix, end the branches."""
    P, H_q, H_kv, W, S = 16, 8, 2, 64, 4
    g = ref.gen(77)
    pool, width = 120, 24
    k, v = ref.pool_of(pool, P, H_kv, g), ref.pool_of(pool, P, H_kv, g)
    table = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table[0, :13] = perm[:13]
    refs = counts_of(table, pool)
    start = refs.clone()
    lens = i32([200, 0, 0, 0, 0, 0])
    scale = 128 ** -0.5
    q = torch.randn(200, H_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    o, lse = cpa.cpa_window_prefill(q, k, v, table[:1], i32([0, 200]), lens[:1], window=W, sinks=S,
                                    check=True)
    ref.close(o, lse, ref.attend(q, ref.dense(k, table[0], 200, P), ref.dense(v, table[0], 200, P),
                                 ref.seen(range(200), 200, W, S, "cuda"), scale, ref.E_P_BF16))
    kids = i32([1, 2, 3])
    src, dst = cpa.cpa_cache_fork(table, lens, i32([0, 0, 0]), kids, refs, P, check=True)
    cpa.cpa_cache_copy_pages(k, v, src, dst, check=True)
    lens[1:4] += 1  # each branch's own token goes to slot 200 of its own last page
    for r in (1, 2, 3):
        k[table[r, 12].long(), 8] = torch.randn(H_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
        v[table[r, 12].long(), 8] = torch.randn(H_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, H_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    for window in (0, W):
        o, lse = cpa.cpa_decode(q, k, v, table[1:4], lens[1:4], window=window, sinks=S, check=True)
        for i in range(3):
            ref.close(o[i:i + 1], lse[i:i + 1], ref.attend(
                q[i:i + 1], ref.dense(k, table[i + 1], 201, P), ref.dense(v, table[i + 1], 201, P),
                ref.seen([200], 201, window, S, "cuda"), scale))
    # pages ceil(4 / 16) .. (201 - 64) / 16 have left the window of the branches
    whole = table.clone()
    cpa.cpa_cache_free(table, kids, i32([1] * 3), i32([8] * 3), refs, check=True)
    assert torch.equal(refs, counts_of(table, pool)) and bool((table[1:4, 1:8] == -1).all())
    o2, lse2 = cpa.cpa_decode(q, k, v, table[1:4], lens[1:4], window=W, sinks=S, check=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # a draft of four tokens in a page of its own; nodes 0, 2, 3 are accepted behind branch 2
    draft = i32([[int(perm[-1])]])
    refs[perm[-1].long()] = 1
    cpa.cpa_cache_compact(k, v, draft, i32([[0, 2, 3]]), i32([3]), table[2:3], lens[2:3], check=True)
    lens[2] += 3
    page = perm[-1].long()
    for x in (k, v):
        assert torch.equal(x[table[2, 12].long(), 9:12], x[page, [0, 2, 3]])
    o, lse = cpa.cpa_decode(q[:1], k, v, table[2:3], lens[2:3], window=W, sinks=S, check=True)
    ref.close(o, lse, ref.attend(q[:1], ref.dense(k, whole[2], 204, P), ref.dense(v, whole[2], 204, P),
                                 ref.seen([203], 204, W, S, "cuda"), scale))
    refs[page] = 0
    cpa.cpa_cache_free(table, kids, i32([0] * 3), i32([width] * 3), refs, check=True)
    assert torch.equal(refs, start)


def test_fork_free_copy_in_a_graph():
    """A captured step (give back, fork, copy) replayed with other parents."""
    table, pool = ref.table_of([50, 70], 16, ref.gen(5), 8)
    rows = torch.cat([table, torch.full((2, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
    refs, dl = counts_of(rows, pool), i32([50, 70, 0, 0])
    k = torch.randn(pool, 16, 2, 128, device="cuda").to(torch.bfloat16)
    v = torch.randn(pool, 16, 2, 128, device="cuda").to(torch.bfloat16)
    par, kid = i32([0, 1]), i32([2, 3])
    z, w = i32([0, 0]), i32([rows.shape[1]] * 2)
    src, dst = i32([0, 0]), i32([0, 0])

    def step():
        cpa.cpa_cache_free(rows, kid, z, w, refs)
        cpa.cpa_cache_fork(rows, dl, par, kid, refs, 16, copy_src=src, copy_dst=dst)
        cpa.cpa_cache_copy_pages(k, v, src, dst)

    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for parents in ([0, 1], [1, 1], [1, 0]):
        par.copy_(i32(parents))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(refs, counts_of(rows, pool))
        for i, r in enumerate(parents):
            L = int(dl[2 + i])
            assert L == [50, 70][r]
            assert torch.equal(ref.dense(k, rows[2 + i], L, 16), ref.dense(k, rows[r], L, 16))
            assert torch.equal(ref.dense(v, rows[2 + i], L, 16), ref.dense(v, rows[r], L, 16))


@pytest.mark.parametrize("op", ["free", "compact", "compact_many", "compact_in_place"])
def test_status_of_replayed_calls(op):
    """Every replay writes the status of its own inputs, whatever the word held before."""
    n = 600 if op == "compact_many" else 12
    B = 8
    per = (n + 15) // 16
    pool = 2 * B * per
    ids = torch.arange(pool, dtype=torch.int32, device="cuda").view(2 * B, per)
    k = torch.randn(pool, 16, 1, 128, device="cuda").to(torch.bfloat16)
    v = torch.randn(pool, 16, 1, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    table, refs = ids.clone(), torch.ones(pool, dtype=torch.int32, device="cuda")
    rows, zero, last, keep = (i32(x) for x in (list(range(B)), [0] * B, [per] * B, [n] * B))

    def call():
        if op == "free":
            table.copy_(ids)
            refs.fill_(1)
            cpa.cpa_cache_free(table, rows, zero, last, refs, workspace=ws)
        else:
            dst = None if op == "compact_in_place" else table[B:]
            cpa.cpa_cache_compact(k, v, table[:B], pos, keep, dst, zero, src_rows=rows, workspace=ws)

    call()
    assert cpa.cpa_get_device_status(ws)[0] == 0
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for bad, status in ((B - 1, 0), (2 * B + 1, 10), (B - 1, 0), (-1, 10), (B - 1, 0)):
        rows[B - 1] = bad
        for _ in range(2):
            gr.replay()
        assert cpa.cpa_get_device_status(ws)[0] == status


@pytest.mark.parametrize("n,stride", [(1, 1024), (16, 64), (17, 64), (1025, 1), (40, 300), (3, 341)])
def test_free_around_one_block(n, stride):
    """Up to 1024 entries by one block, more by a block per range; ranges of unequal length."""
    g = ref.gen(n + stride)
    table = torch.randperm(n * stride, generator=g, device="cuda").to(torch.int32).view(n, stride)
    table[n // 2] = table[0] if n > 1 else table[0].clone()  # shared by two rows
    refs = counts_of(table, n * stride)
    first = torch.randint(0, stride + 1, (n,), generator=g, device="cuda").to(torch.int32)
    last = torch.randint(0, stride + 1, (n,), generator=g, device="cuda").to(torch.int32)
    rows = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    k = torch.arange(stride, device="cuda")
    want = table.clone()
    want[rows.long()] = torch.where((k >= first[:, None]) & (k < last[:, None]), -1,
                                    table[rows.long()])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    cpa.cpa_cache_free(table, rows, first, last, refs, workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == 0
    assert torch.equal(table, want) and torch.equal(refs, counts_of(table, n * stride))
    first[0], last[0] = 0, stride + 1
    cpa.cpa_cache_free(table, rows, first, last, refs, workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == 8
    assert torch.equal(table, want) and torch.equal(refs, counts_of(table, n * stride))


@pytest.mark.parametrize("stride", [16, 600])
@pytest.mark.parametrize("first,last,status", [("past", 3, 8), (0, -1, 8), (-5, -1, 8), ("past", 0, 8),
                                               (-1, 3, 8), (5, "past", 8), ("past", "past", 8),
                                               ("end", "end", 0), ("end", 0, 0), (7, 2, 0)])
def test_free_looks_at_both_bounds(first, last, status, stride):
    """Each bound by itself, also where the range would be empty; by one block and by one a range."""
    at = {"past": stride + 1, "end": stride}
    table = torch.arange(2 * stride, dtype=torch.int32, device="cuda").view(2, stride)
    refs = torch.ones(2 * stride, dtype=torch.int32, device="cuda")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    cpa.cpa_cache_free(table, i32([0, 1]), i32([2, at.get(first, first)]), i32([5, at.get(last, last)]),
                       refs, workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == status
    want = torch.arange(2 * stride, dtype=torch.int32, device="cuda").view(2, stride)
    want[0, 2:5] = -1
    assert torch.equal(table, want) and torch.equal(refs, counts_of(table, 2 * stride))


def test_fork_of_a_sequence_whose_window_has_moved_on():
    """Pages that a window has left are given back; a fork of what is left passes over them,
    and decode of the child sees what decode of the parent sees."""
    P, L, W, S = 16, 200, 64, 4
    g = ref.gen(9)
    table, pool = ref.table_of([L, L], P, g, 6)
    k, v = ref.pool_of(pool, P, 2, g), ref.pool_of(pool, P, 2, g)
    rows = torch.cat([table, torch.full((2, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
    refs, dl = counts_of(table, pool), i32([L, L, 0, 0])
    cpa.cpa_cache_free(rows, i32([0]), i32([1]), i32([(L - W) // P]), refs, check=True)
    before = refs.clone()
    src, dst = cpa.cpa_cache_fork(rows, dl, i32([0, 1]), i32([2, 3]), refs, P, check=True)
    cpa.cpa_cache_copy_pages(k, v, src, dst, check=True)
    assert rows[2, :12].tolist() == rows[0, :12].tolist() and rows[3, :12].tolist() == table[1, :12].tolist()
    assert bool((rows[2, 1:8] == -1).all()) and dl.tolist() == [L] * 4
    assert torch.equal(refs, counts_of(rows, pool))
    q = torch.randn(2, 8, 128, generator=g, device="cuda").to(torch.bfloat16)[[0, 1, 0, 1]].contiguous()
    o, lse = cpa.cpa_decode(q, k, v, rows, dl, window=W, sinks=S, check=True)
    assert torch.equal(o[:2], o[2:]) and torch.equal(lse[:2], lse[2:])
    cpa.cpa_cache_free(rows, i32([2, 3]), i32([0, 0]), i32([rows.shape[1]] * 2), refs, check=True)
    assert torch.equal(refs, before)
    for entry, bad in ((3, -2), (3, pool), (12, -1), (12, -2)):  # (entry 12 is the last, partly filled)
        was = rows[1, entry].clone()
        rows[1, entry] = bad
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_cache_fork(rows, dl, i32([1]), i32([3]), refs.clone(), P, check=True)
        assert e.value.status == 5
        rows[1, entry] = was


def test_fork_in_a_pool_of_many_chunks():
    """Free pages far apart, around and past the 256 chunks of 1024 that a block looks over at
    a time; one child more than there are pages."""
    pool = 700_001
    refs = torch.ones(pool, dtype=torch.int32, device="cuda")
    for lo, hi in ((1023, 1025), (262_140, 262_150), (263_000, 263_001), (524_280, 524_300),
                   (pool - 1, pool)):
        refs[lo:hi] = 0
    free = torch.nonzero(refs == 0).view(-1).to(torch.int32)
    n = free.numel() + 1
    rows = torch.full((n + 1, 2), -1, dtype=torch.int32, device="cuda")
    rows[0, 0] = 7
    dl = torch.full((n + 1,), 5, dtype=torch.int32, device="cuda")
    ws = torch.empty(cpa.cpa_cache_fork_workspace_size(pool), dtype=torch.uint8, device="cuda")
    src, dst = cpa.cpa_cache_fork(rows, dl, i32([0] * n), i32(list(range(1, n + 1))), refs, 16,
                                  workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == 11
    assert torch.equal(dst[:-1], free) and int(dst[-1]) == -1
    assert src.tolist() == [7] * (n - 1) + [-1] and bool((refs == 1).all())
