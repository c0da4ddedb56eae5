"""Windowed prefill of ragged chunks against a 64-bit reference."""
import pytest
import torch

import cascade_paged_attention_gb300 as cpa
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def make(news, lens, H_q, H_kv, P, seed, lead=0, trail=0):
    g = ref.gen(seed)
    table, pool = ref.table_of(lens, P, g)
    start = [lead]
    for m in news:
        start.append(start[-1] + m)
    T = start[-1] + trail
    q = torch.randn(T, H_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    k, v = ref.pool_of(pool, P, H_kv, g), ref.pool_of(pool, P, H_kv, g)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return q, k, v, table, i32(start), i32(lens), start


def check(news, lens, H_q, H_kv, P, window=0, sinks=0, seed=0, lead=0, trail=0, hide=True, **kw):
    q, k, v, table, qs, dl, start = make(news, lens, H_q, H_kv, P, seed, lead, trail)
    full = table.clone()
    masks = [ref.seen(range(L - m, L), L, window, sinks, "cuda") for m, L in zip(news, lens)]
    if hide:
        ref.hide_unseen(k, v, table, lens, [m.any(0) for m in masks], P)
    o = torch.full_like(q, 7.0)
    lse = torch.full((q.shape[0], H_q), 7.0, device="cuda")
    cpa.cpa_window_prefill(q, k, v, table, qs, dl, window=window, sinks=sinks, o=o, lse=lse,
                           check=True, **kw)
    if hide:
        for x in (k, v):
            x.nan_to_num_(0.0)
    for b, (m, L) in enumerate(zip(news, lens)):
        a = start[b]
        K, V = ref.dense(k, full[b], L, P), ref.dense(v, full[b], L, P)
        for i0 in range(0, m, 256):
            i1 = min(m, i0 + 256)
            want = ref.attend(q[a + i0:a + i1], K, V, masks[b][i0:i1], 128 ** -0.5, ref.E_P_BF16)
            ref.close(o[a + i0:a + i1], lse[a + i0:a + i1], want)
    for r in (slice(0, lead), slice(start[-1], q.shape[0])):  # rows of no request
        assert bool((o[r] == 7).all()) and bool((lse[r] == 7).all())


@pytest.mark.parametrize("H_q,H_kv,P", [(32, 8, 16), (8, 8, 8), (5, 1, 64), (12, 4, 32), (16, 1, 256),
                                        (64, 8, 128), (1, 1, 16), (128, 1, 16), (100, 2, 16)])
def test_ragged_chunks(H_q, H_kv, P):
    check([1, 2, 0, 17, 64, 65, 128, 31], [1, 300, 5, 17, 200, 129, 128, 1000], H_q, H_kv, P,
          seed=H_q, lead=3, trail=5)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (5, 3), (64, 4), (100, 130), (128, 0),
                                          (129, 16), (255, 128), (1000, 4), (3, 5000)])
@pytest.mark.parametrize("P", [8, 64])
def test_windows_and_sinks(window, sinks, P):
    check([300, 1, 70, 129], [300, 600, 1200, 129], 8, 2, P, window, sinks, seed=window + P, trail=1)


@pytest.mark.parametrize("news,lens,window,sinks", [
    ([1], [1], 0, 0), ([1], [5000], 0, 0), ([7], [9000], 0, 0), ([3, 1, 2], [4000, 1, 2500], 1500, 4),
    ([1500], [1500], 0, 0), ([1100], [2000], 700, 16), ([513, 700], [513, 3333], 512, 64),
    ([0, 0], [10, 0], 0, 0), ([2000], [2000], 128, 4)])
def test_short_and_long(news, lens, window, sinks):
    check(news, lens, 32, 8, 16, window, sinks, seed=sum(news), hide=False)
    check(news, lens, 4, 1, 32, window, sinks, seed=sum(news) + 1, hide=False)


def test_bounds_given_and_repeat():
    """max_new and max_seq_len as tight as they may be; the same call twice gives the same bits."""
    news, lens = [40, 3, 200], [1000, 3, 900]
    check(news, lens, 16, 4, 16, 300, 4, seed=2, max_new=200, max_seq_len=1000)
    q, k, v, table, qs, dl, _ = make(news, lens, 16, 4, 16, 2)
    ws = torch.full((cpa.cpa_window_prefill_workspace_size(3, q.shape[0], 16, 4, 128, 16, 200),),
                    0xA5, dtype=torch.uint8, device="cuda")
    kw = dict(max_new=200, max_seq_len=1000, workspace=ws)
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, **kw)
    ws.fill_(0x5A)
    o2, lse2 = cpa.cpa_window_prefill(q, k, v, table, qs, dl, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_scores_that_grow():
    """Scores that climb along the keys by far more than 2^8: the running maximum moves often."""
    q, k, v, table, qs, dl, _ = make([300], [900], 4, 1, 16, 5)
    pos = torch.arange(900, device="cuda")
    q.copy_(q[:1, :1].expand_as(q))
    k[table[0].long()[pos // 16], pos % 16] = \
        (q[0, 0] / 12).to(torch.bfloat16)[None, None] * (pos / 20).to(torch.bfloat16)[:, None, None]
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, window=500, sinks=2, check=True)
    want = ref.attend(q, ref.dense(k, table[0], 900, 16), ref.dense(v, table[0], 900, 16),
                      ref.seen(range(600, 900), 900, 500, 2, "cuda"), 128 ** -0.5, ref.E_P_BF16)
    ref.close(o, lse, want)


def test_nan_that_is_seen_and_one_that_is_not():
    q, k, v, table, qs, dl, _ = make([200], [400], 4, 2, 16, 11)
    at = 350
    v[table[0, at // 16].long(), at % 16, 1, 9] = float("nan")
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, window=30, check=True)
    bad = torch.isnan(o)
    pos = torch.arange(200, 400, device="cuda")
    hit = (pos >= at) & (pos < at + 30)
    assert bool(bad[hit][:, 2:, 9].all()) and bool(torch.isfinite(lse).all())
    assert int(bad.sum()) == 2 * int(hit.sum())


def test_bad_starts_lengths_and_pages_are_reported():
    q, k, v, table, qs, dl, _ = make([30, 40], [100, 200], 8, 2, 16, 13)
    call = lambda **kw: cpa.cpa_window_prefill(q, k, v, table, qs, dl, check=True, **kw)  # noqa: E731
    call()
    for where, bad, status in ((qs, [0, 30, 71], 8), (qs, [-1, 30, 70], 8), (qs, [0, 80, 70], 8),
                               (qs, [0, 31, 30], 8), (dl, [29, 200], 8), (dl, [100, 209], 8),
                               (dl, [-1, 200], 8), (qs, [0, -2 ** 31, 70], 8),
                               (dl, [2 ** 31 - 1, 200], 8)):
        good = where.clone()
        where.copy_(torch.tensor(bad, dtype=torch.int32))
        with pytest.raises(cpa.CpaError) as e:
            call()
        assert e.value.status == status, bad
        where.copy_(good)
    with pytest.raises(cpa.CpaError) as e:
        call(max_new=39)
    assert e.value.status == 8
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        good = table[1, 3].clone()
        table[1, 3] = bad
        with pytest.raises(cpa.CpaError) as e:
            call()
        assert e.value.status == 5
        call(window=64)  # positions 160 - 63 and on: page 3 (48..63) is not seen
        table[1, 3] = good
    call()


def test_graph_replay_and_streams():
    """A captured call serves other lengths and chunks; two streams at once share nothing."""
    q, k, v, table, qs, dl, _ = make([100, 60], [600, 500], 16, 4, 16, 17)
    o, lse = torch.empty_like(q), torch.empty(160, 16, device="cuda")
    kw = dict(max_new=120, window=200, sinks=4)
    cpa.cpa_window_prefill(q, k, v, table, qs, dl, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cpa.cpa_window_prefill(q, k, v, table, qs, dl, o=o, lse=lse, **kw)
    for news, lens in (([100, 60], [600, 500]), ([40, 120], [44, 480]), ([1, 0], [3, 200])):
        qs.copy_(torch.tensor([0, news[0], sum(news)], dtype=torch.int32))
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            o2, lse2 = cpa.cpa_window_prefill(q, k, v, table, qs, dl, **kw)
        o3, lse3 = cpa.cpa_window_prefill(q, k, v, table, qs, dl, **kw)
        torch.cuda.synchronize()
        n = sum(news)
        assert torch.equal(o[:n], o2[:n]) and torch.equal(o[:n], o3[:n])
        a = 0
        for b, (m, L) in enumerate(zip(news, lens)):
            want = ref.attend(q[a:a + m], ref.dense(k, table[b], L, 16), ref.dense(v, table[b], L, 16),
                              ref.seen(range(L - m, L), L, 200, 4, "cuda"), 128 ** -0.5, ref.E_P_BF16)
            ref.close(o[a:a + m], lse[a:a + m], want)
            a += m


def test_agrees_with_prefill_hit():
    """One length for all and no window is cpa_prefill_hit's case."""
    q, k, v, table, qs, dl, _ = make([190, 190], [500, 500], 32, 8, 16, 23)
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, check=True)
    o2, lse2 = cpa.cpa_prefill_hit(q, k, v, table, 2, 500, 310, check=True)
    # each within 2^-8 (|o| + sum w |v|) of the exact value, |o| < 1 here
    assert float((o.float() - o2.float()).abs().max()) <= 2e-2
    assert float((lse - lse2).abs().max()) <= 1e-3


def test_many_requests_some_long_some_empty():
    """More requests than threads, lengths from none to several units, on a stream given by
    argument; rows of the reference by the decode call, whose keys a last token sees alike."""
    g = torch.Generator().manual_seed(5)
    n = 1100
    news = [int(x) for x in torch.randint(0, 4, (n,), generator=g)]
    news[700] = 900
    news[3] = 300
    lens = [m + int(x) for m, x in zip(news, torch.randint(0, 60, (n,), generator=g))]
    q, k, v, table, qs, dl, start = make(news, lens, 8, 2, 8, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, window=50, sinks=2, stream=side, check=True)
    torch.cuda.current_stream().wait_stream(side)
    # the last token of each request that has one
    some = torch.tensor([b for b in range(n) if news[b]], device="cuda")
    last = (qs[1:].long() - 1)[some]
    o1, lse1 = cpa.cpa_decode(q[last], k, v, table[some].contiguous(), dl[some].contiguous(), window=50,
                              sinks=2, check=True)
    # weights to 2^-8 here, to 2^-15 there; |o| and the mean |v| stay below 5
    assert float((o[last].float() - o1.float()).abs().max()) <= 3 * 2.0 ** -8 * 5
    assert float((lse[last] - lse1).abs().max()) <= 1e-4
    for b in (3, 700):
        a, m, L = start[b], news[b], lens[b]
        want = ref.attend(q[a:a + m], ref.dense(k, table[b], L, 8), ref.dense(v, table[b], L, 8),
                          ref.seen(range(L - m, L), L, 50, 2, "cuda"), 128 ** -0.5, ref.E_P_BF16)
        ref.close(o[a:a + m], lse[a:a + m], want)


def test_values_that_are_not_numbers_only_where_they_are_seen():
    """NaN and infinity among K and V, in whole and in cut units: rows that see them have what
    the definition gives, the others are as if they were not there."""
    news, lens = [700, 30], [1500, 4000]
    q, k, v, table, qs, dl, start = make(news, lens, 4, 1, 16, 8)
    clean = (k.clone(), v.clone())
    hits = [(0, 900, "v", float("inf")), (0, 1200, "k", float("nan")), (1, 3985, "v", float("nan"))]
    for b, at, which, x in hits:
        pool = k if which == "k" else v
        pool[table[b, at // 16].long(), at % 16, 0, 5] = x
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, window=100, check=True)
    for b in range(2):
        a, m, L = start[b], news[b], lens[b]
        pos = torch.arange(L - m, L, device="cuda")
        sick = torch.zeros(m, dtype=torch.bool, device="cuda")
        for hb, at, which, x in hits:
            if hb != b:
                continue
            sees = (pos >= at) & (pos < at + 100)
            rows = o[a:a + m][sees]
            if which == "k":
                assert bool(torch.isnan(rows).all()) and bool(torch.isnan(lse[a:a + m][sees]).all())
            else:
                assert bool((~torch.isfinite(rows[:, :, 5])).all())
                assert bool(torch.isfinite(lse[a:a + m][sees & ~sick]).all())
            sick |= sees
        want = ref.attend(q[a:a + m], ref.dense(clean[0], table[b], L, 16),
                          ref.dense(clean[1], table[b], L, 16),
                          ref.seen(range(L - m, L), L, 100, 0, "cuda"), 128 ** -0.5, ref.E_P_BF16)
        ref.close(o[a:a + m][~sick], lse[a:a + m][~sick], [t[~sick] for t in want])


@pytest.mark.parametrize("M", [1, 40, 129])
def test_against_the_oracle(M):
    """The library's own fp64 oracle (plain C) on its seeded workloads, slots past the end NaN."""
    import numpy as np

    import cpa_synth
    import oracle
    from tests.gpu_util import dev_bf16, dev_i32

    wl = cpa_synth.make_prefill(B=3, N=300, H=300 - M, H_q=16, H_kv=4, page_size=32, seed=M,
                                pad_fill="nan")
    ref_o, ref_lse = oracle.prefill_wl(wl)
    kv = (dev_bf16(wl.k_pages), dev_bf16(wl.v_pages), dev_i32(wl.page_table))
    q, lens = dev_bf16(wl.q), dev_i32([300] * 3)
    outs = [cpa.cpa_window_prefill(q, *kv, dev_i32(np.arange(4) * M), lens, check=True)]
    if M == 1:
        outs.append(cpa.cpa_decode(q, *kv, lens, check=True))
    for o, lse in outs:
        o = o.double().cpu().numpy().reshape(ref_o.shape)
        # half a step of bf16 for the output, as much for the weights: sum w |v| is about 0.8 over
        # the 170 keys and more that a row sees
        assert np.all(np.abs(o - ref_o) <= 2.0 ** -8 * (np.abs(ref_o) + 1.0) + 1e-4)
        assert float(np.abs(lse.double().cpu().numpy().reshape(ref_lse.shape) - ref_lse).max()) <= 1e-4


@pytest.mark.parametrize("spare", [-1, 0, 1])
@pytest.mark.parametrize("news", [[1], [30, 1]])
def test_as_many_tiles_as_blocks(news, spare):
    """Calls of about one key tile a block: below and above where the split changes."""
    tiles = torch.cuda.get_device_properties(0).multi_processor_count + spare
    lens = [128 * (tiles - 3 * (len(news) - 1))] + [300] * (len(news) - 1)
    check(news, lens, 4, 1, 16, seed=spare + 5, hide=False)
    check(news, [128 * (tiles // 2)] + [129] * (len(news) - 1), 8, 2, 64, seed=spare + 6, hide=False)


@pytest.mark.parametrize("spare", [-1, 0, 1])
def test_as_many_tiles_as_twice_the_blocks(spare):
    """Two tiles a block: the most that are shared out without regard to units."""
    tiles = 2 * torch.cuda.get_device_properties(0).multi_processor_count + spare
    check([3], [128 * tiles], 2, 1, 16, seed=spare + 7, hide=False)
    check([20] * 6, [128 * (tiles // 12)] * 5 + [128 * (tiles - 11 * (tiles // 12))], 8, 2, 64,
          seed=spare + 8, hide=False)


def test_rows_done_again_for_longer_than_a_wait_may_last():
    """A unit of 450000 keys, every row of which is done again key by key (some seconds), and one
    of 8 keys after it in every block: no wait of the second gives up meanwhile."""
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    g = ref.gen(31)
    L, m, P = 450_000, 8, 256
    table, pool = ref.table_of([L, m], P, g)
    k, v = ref.pool_of(pool, P, 1, g), ref.pool_of(pool, P, 1, g)
    v[table[0, 0].long(), 0, 0, 5] = float("nan")
    q = torch.randn(2 * m, 32, 128, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    start = torch.arange(2 * n_sm + 1, dtype=torch.int32, device="cuda") * m
    o, lse = cpa.cpa_window_prefill(q.repeat(n_sm, 1, 1), k, v, table.repeat(n_sm, 1), start,
                                    i32([L, m] * n_sm), check=True)
    o, lse = o.view(n_sm, 2 * m, 32, 128), lse.view(n_sm, 2 * m, 32)
    assert torch.equal(lse, lse[:1].expand_as(lse))
    assert bool(torch.isnan(o[:, :m, :, 5]).all())
    o[:, :m, :, 5] = 0
    assert torch.equal(o, o[:1].expand_as(o))
    v[table[0, 0].long(), 0, 0, 5] = 0
    for a, n, row in ((0, L, table[0]), (m, m, table[1])):
        K, V = ref.dense(k, row, n, P), ref.dense(v, row, n, P)
        for i in range(m):
            want = ref.attend(q[a + i:a + i + 1].view(32, 1, 128), K, V,
                              ref.seen([n - m + i] * 32, n, 0, 0, "cuda"), 128 ** -0.5, ref.E_P_BF16)
            if a == 0:
                want[0][..., 5] = 0
                want[2][..., 5] = 0
            ref.close(o[0, a + i].view(32, 1, 128), lse[0, a + i].view(32, 1), want)
