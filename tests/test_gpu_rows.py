"""Rows written to the pages of a cache and read back, against indexing in PyTorch.  What is
copied is equal bit for bit; FP8 codes equal those of the quotient in 32 bits rounded by PyTorch,
and what is read back equals the product in 32 bits rounded once."""
import pytest
import torch

import cascade_paged_attention_gb300 as cpa
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(n, lead=0):
    out = [lead]
    for m in n:
        out.append(out[-1] + m)
    return out


def slots(table, firsts, news, P):
    """Slot of every token, request by request."""
    out = []
    for b, (f, m) in enumerate(zip(firsts, news)):
        pos = torch.arange(f, f + m, device="cuda")
        out.append(table[b].long()[pos // P] * P + pos % P)
    return torch.cat(out)


def random_bits(shape, dtype, g):
    """Any bit pattern: what is copied is not looked at."""
    n = torch.empty(shape, dtype=dtype).element_size()
    x = torch.randint(0, 256, (*shape[:-1], shape[-1] * n), generator=g, device="cuda", dtype=torch.uint8)
    return x.view(dtype)


def bits(x):
    return x.contiguous().view(torch.uint8)


CASES = [([1], [1]), ([1, 1, 1], [1, 17, 300]), ([0, 5, 0, 33, 1], [0, 5, 9, 40, 64]),
         ([64, 65, 31, 32], [64, 100, 31, 1000]), ([700, 3], [700, 1000]), ([1] * 40, range(1, 41)),
         ([0] * 70 + [9] + [0] * 3, [5] * 70 + [20] + [0] * 3)]


def quantised(x, scale):
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    assert torch.equal((got & 0x7F) == 0x7F, nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("H,d,P,dtype", [(8, 128, 16, torch.bfloat16), (1, 128, 8, torch.bfloat16),
                                         (3, 128, 256, torch.float16), (2, 8, 64, torch.uint8),
                                         (1, 8, 32, torch.bfloat16), (5, 24, 16, torch.float32)])
def test_copies(case, H, d, P, dtype):
    news, lens = (list(x) for x in CASES[case])
    g = ref.gen(case)
    table, pool = ref.table_of(lens, P, g)
    st = starts(news, lead=2)
    T = st[-1] + 3
    k, v = (random_bits((pool, P, H, d), dtype, g) for _ in "kv")
    wide = random_bits((T, 2 * H + 3, d * 16), dtype, g)  # (whole pieces of 16 bytes before it)
    kn = wide.view(T, -1)[:, 16 * d:16 * d + H * d].view(T, H, d)
    vn = random_bits((T, H, d), dtype, g)
    want = [x.clone() for x in (k, v)]
    at = slots(table, [L - m for L, m in zip(lens, news)], news, P)
    for x, n in zip(want, (kn, vn)):
        bits(x.view(-1, H * d))  # (contiguous)
        x.view(-1, H, d).view(torch.uint8)[at] = n[2:st[-1]].contiguous().view(torch.uint8)
    cpa.cpa_cache_append(kn, vn, k, v, table, i32(st), i32(lens), check=True)
    for x, w in zip((k, v), want):
        assert torch.equal(bits(x), bits(w))
    # read back: the same rows, and rows of no request as they were
    first = [L - m for L, m in zip(lens, news)]
    out = [torch.zeros((T, H, d), dtype=dtype, device="cuda") for _ in "kv"]
    for o in out:
        o.view(torch.uint8).fill_(0x5A)
    cpa.cpa_cache_gather(k, v, table, i32(st), first=i32(first), k_out=out[0], v_out=out[1], check=True)
    for o, n in zip(out, (kn, vn)):
        assert torch.equal(bits(o[2:st[-1]]), bits(n[2:st[-1]]))
        assert bool((o[:2].view(torch.uint8) == 0x5A).all()) and bool((o[st[-1]:].view(torch.uint8) == 0x5A).all())


@pytest.mark.parametrize("H,P", [(8, 16), (1, 8), (5, 128)])
@pytest.mark.parametrize("per_channel", [False, True])
def test_fp8(H, P, per_channel):
    news, lens = [0, 5, 33, 1, 200], [7, 5, 100, 64, 333]
    g = ref.gen(H + P)
    table, pool = ref.table_of(lens, P, g)
    st = starts(news)
    n = (H, 128) if per_channel else (1,)
    scale = [torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001 for _ in "kv"]
    if per_channel:
        scale[0][0, :4] = torch.tensor([2.0 ** -7, 0.03125, 1.0, 3.0], device="cuda")  # exact ties
    new = [torch.randn(st[-1], H, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    new[0][::7, :, 5] = 1e30
    new[0][::5, :, 6] = float("inf")
    new[0][::3, :, 7] = float("-inf")
    new[1][::4, :, 8] = float("nan")
    new[1][:, :, 9] = 0.0
    new[1][:, :, 10] = 1e-30
    pages = [torch.randint(0, 256, (pool, P, H, 128), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv"]
    want = [x.clone() for x in pages]
    at = slots(table, [L - m for L, m in zip(lens, news)], news, P)
    for w, x, s in zip(want, new, scale):
        w.view(-1, H, 128)[at] = quantised(x, s)
    cpa.cpa_cache_append_fp8(*new, *pages, *scale, table, i32(st), i32(lens), check=True)
    for x, w in zip(pages, want):
        same_codes(x, w)
    # from the first position on
    full = starts(lens)
    got = cpa.cpa_cache_gather_fp8(*pages, *scale, table, i32(full), T=full[-1], check=True)
    at = slots(table, [0] * len(lens), lens, P)
    for o, x, s in zip(got, pages, scale):
        x = x.view(-1, H, 128)[at].view(torch.float8_e4m3fn).float() * s
        w = x.to(torch.bfloat16)
        assert torch.equal(torch.isnan(o), torch.isnan(w)) and torch.equal(o.nan_to_num(7), w.nan_to_num(7))


@pytest.mark.parametrize("P", [8, 64, 256])
def test_latents(P):
    news, lens = [3, 0, 40, 513], [3, 2, 100, 700]
    g = ref.gen(P)
    table, pool = ref.table_of(lens, P, g)
    st = starts(news, lead=1)
    pages = random_bits((pool, P, 576), torch.bfloat16, g)
    wide = random_bits((st[-1], 640), torch.bfloat16, g)
    c, r = random_bits((st[-1], 512), torch.bfloat16, g), wide[:, 64:128]
    want = pages.clone()
    first = [L - m for L, m in zip(lens, news)]
    at = slots(table, first, news, P)
    want.view(-1, 576).view(torch.int16)[at] = torch.cat([c, r], 1)[1:].view(torch.int16)
    cpa.cpa_latent_append(c, r, pages, table, i32(st), i32(lens), check=True)
    assert torch.equal(bits(pages), bits(want))
    got = cpa.cpa_latent_gather(pages, table, i32(st), T=st[-1], first=i32(first), check=True)
    assert torch.equal(bits(got[0][1:]), bits(c[1:])) and torch.equal(bits(got[1][1:]), bits(r[1:].contiguous()))


@pytest.mark.parametrize("big", [False, True])
def test_what_is_wrong_is_reported_and_left_out(big):
    """(big: the form whose warps report by themselves.)"""
    P, H = 8 if big else 16, 1 if big else 2
    news, lens = [10, 140000 if big else 20, 7], [50, 140000 if big else 30, 9]
    g = ref.gen(3)
    table, pool = ref.table_of(lens, P, g)
    st = starts(news)
    new = random_bits((st[-1], H, 128), torch.bfloat16, g)
    ws = torch.full((256,), 0xA5, dtype=torch.uint8, device="cuda")

    def go(t, s, n, status):
        pages = torch.zeros(pool, P, H, 128, dtype=torch.bfloat16, device="cuda")
        cpa.cpa_cache_append(new, new, pages, pages.clone(), t, s, n, workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == status
        out = torch.zeros_like(new)
        cpa.cpa_cache_gather(pages, pages, t, s, first=n - (s[1:] - s[:-1]), k_out=out,
                             v_out=torch.zeros_like(new), workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == status
        return pages, bits(out) == bits(new)
    pages, same = go(table, i32(st), i32(lens), 0)
    assert bool(same.all())
    for bad in (pool, -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad  # positions P .. 2 P - 1 of the second request
        pages, same = go(t, i32(st), i32(lens), 5)
        lo, hi = max(P, lens[1] - news[1]), min(2 * P, lens[1])
        hit = torch.zeros(st[-1], dtype=torch.bool, device="cuda")
        a = st[1] - (lens[1] - news[1])
        hit[a + lo:a + hi] = True
        assert bool(same[~hit].all()) and bool((pages.view(-1, H, 128)[slots(table, [lo], [hi - lo], P)] == 0).all())
    for lengths in ([50, 4, 9], [50, 140000 * 16, 9], [50, -1, 9], [50, 2 ** 31 - 1, 9]):
        pages, same = go(table, i32(st), i32(lengths), 8)
        assert bool(same[:st[1]].all()) and bool(same[st[2]:].all())
    for s in ([0, 10, 5, st[-1]], [0, 10, st[2], st[-1] + 1], [-1, 10, st[2], st[-1]]):
        go(table, i32(s), i32(lens), 8)


def rows_of_valid_requests(st, lens, T, most):
    """(request, first row, tokens) of each request whose own start, end and length are in range."""
    return [(b, s0, s1 - s0) for b, (s0, s1) in enumerate(zip(st, st[1:]))
            if 0 <= s0 <= s1 <= T and 0 <= lens[b] - (s1 - s0) and lens[b] <= most]


def _one_bad_start():
    st = list(range(0, 404, 4))
    st[64] = 0  # requests 63 (descending) and 64 (longer than its sequence) are wrong
    return st, [4 + b % 30 for b in range(100)]


def _starts_past_the_rows():
    st = list(range(0, 153, 3))
    st[7], st[20], st[41] = 10 ** 9, -5, 2 ** 31 - 1
    return st, [3 + b for b in range(50)]


BAD_STARTS = [_one_bad_start(), ([0, 10, 0, 30], [50, 30, 20]), ([0, 10, 0, 30], [50, 30, 40]),
              _starts_past_the_rows(), ([9, 9, 40, 12, 33, 33, 50], [5, 31, 28, 21, 3, 60])]


@pytest.mark.parametrize("kind", ["copy", "fp8", "latent"])
@pytest.mark.parametrize("case", range(len(BAD_STARTS)))
@pytest.mark.parametrize("big", [False, True])
def test_starts_that_are_not_ascending(kind, case, big):
    """Requests beside a wrong start: every row of those that are right is moved, whatever the
    search by start would find, and nothing else is.  (big: the form whose warps report by
    themselves.)"""
    st, lens = (list(x) for x in BAD_STARTS[case])
    P, H = 8, 2
    if big:
        lens += [1] * 9000
        st += list(range(st[-1] + 1, st[-1] + 9001))
    T = st[-1] + 2
    g = ref.gen(case)
    table, pool = ref.table_of(lens, P, g)
    most = table.shape[1] * P
    valid = rows_of_valid_requests(st, lens, T, most)
    assert 0 < len(valid) < len(lens) and sorted(st) != st
    rows = torch.cat([torch.arange(s0, s0 + m, device="cuda") for _, s0, m in valid])
    req = torch.repeat_interleave(i32([b for b, _, _ in valid]).long(), i32([m for _, _, m in valid]).long())
    pos = rows - i32([s0 for _, s0, m in valid for _ in range(m)]).long() + \
        i32([lens[b] - m for b, _, m in valid for _ in range(m)]).long()
    at = table[req, pos // P].long() * P + pos % P
    ws = torch.full((256,), 0xA5, dtype=torch.uint8, device="cuda")
    scale = [torch.rand(H, 128, generator=g, device="cuda") * 0.02 + 0.001 for _ in "kv"]
    widths = (512, 64) if kind == "latent" else (H * 128, H * 128)
    new = [torch.randn(T, w, generator=g, device="cuda").to(torch.bfloat16) for w in widths]
    args = (table, i32(st), i32(lens))
    if kind == "latent":
        pages = torch.full((pool, P, 576), 7.0, device="cuda").to(torch.bfloat16)
        want = pages.clone()
        want.view(-1, 576)[at] = torch.cat(new, 1)[rows]
        cpa.cpa_latent_append(*new, pages, *args, workspace=ws)
        got, want = [pages], [want]
    else:
        kv = [x.view(T, H, 128) for x in new]
        kind_of = torch.uint8 if kind == "fp8" else torch.bfloat16
        got = [torch.full((pool, P, H, 128), 7, dtype=kind_of, device="cuda") for _ in "kv"]
        want = [x.clone() for x in got]
        for w, x, s in zip(want, kv, scale):
            w.view(-1, H, 128)[at] = quantised(x[rows], s) if kind == "fp8" else x[rows]
        if kind == "fp8":
            cpa.cpa_cache_append_fp8(*kv, *got, *scale, *args, workspace=ws)
        else:
            cpa.cpa_cache_append(*kv, *got, *args, workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == 8
    for x, w in zip(got, want):
        assert torch.equal(bits(x), bits(w))
    # and back: rows of one valid request have its slots, rows of none are as they were
    first = i32([lens[b] - (s1 - s0) if abs(s1 - s0) < 2 ** 20 else 0 for b, (s0, s1) in enumerate(zip(st, st[1:]))])
    out = [torch.full((T, w) if kind == "latent" else (T, H, 128), 5.0, device="cuda").to(torch.bfloat16) for w in widths]
    kw = dict(first=first, workspace=ws)
    if kind == "latent":
        cpa.cpa_latent_gather(*got, table, i32(st), c_out=out[0], r_out=out[1], **kw)
    elif kind == "fp8":
        cpa.cpa_cache_gather_fp8(*got, *scale, table, i32(st), k_out=out[0], v_out=out[1], **kw)
    else:
        cpa.cpa_cache_gather(*got, table, i32(st), k_out=out[0], v_out=out[1], **kw)
    assert cpa.cpa_get_device_status(ws)[0] == 8
    times = torch.bincount(rows, minlength=T)
    one = times[rows] == 1
    for i, o in enumerate(out):
        if kind == "latent":
            src = got[0].view(-1, 576)[at][:, :512] if i == 0 else got[0].view(-1, 576)[at][:, 512:]
        else:
            src = got[i].view(-1, H, 128)[at]
            if kind == "fp8":
                src = (src.view(torch.float8_e4m3fn).float() * scale[i]).to(torch.bfloat16)
        assert torch.equal(bits(o[rows[one]]), bits(src[one]))
        assert bool((o[times == 0] == 5).all())


@pytest.mark.parametrize("B", [5000, 9000])
def test_many_requests_and_empty_ones(B):
    g = ref.gen(9)
    P = 8
    news = torch.randint(0, 3, (B,), generator=g, device="cuda")
    news[100:400] = 0
    lens = (news + torch.randint(0, 5, (B,), generator=g, device="cuda")).tolist()
    news = news.tolist()
    table, pool = ref.table_of(lens, P, g)
    st = starts(news)
    new = random_bits((st[-1], 1, 128), torch.bfloat16, g)
    k, v = torch.zeros(pool, P, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(pool, P, 1, 128, dtype=torch.bfloat16, device="cuda")
    cpa.cpa_cache_append(new, new, k, v, table, i32(st), i32(lens), check=True)
    rows = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(news, device="cuda"))
    pos = torch.arange(st[-1], device="cuda") - i32(st)[rows].long() + (i32(lens) - i32(news))[rows].long()
    at = table[rows, pos // P].long() * P + pos % P
    for x in (k, v):
        assert torch.equal(bits(x.view(-1, 1, 128)[at]), bits(new))
        left = torch.ones(pool * P, dtype=torch.bool, device="cuda")
        left[at] = False
        assert bool((x.view(-1, 128)[left] == 0).all())


def test_nothing_to_do():
    k = torch.full((2, 16, 1, 128), 3.0, device="cuda").to(torch.bfloat16)
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    cpa.cpa_cache_append(none, none, k, k, i32([[0]]), i32([0, 0]), i32([0]), workspace=ws, check=True)
    assert bool((k == 3).all())
    ws.fill_(0xFF)
    out = cpa.cpa_cache_gather(k, k, i32([[0]]), i32([0, 0]), T=0, workspace=ws, check=True)
    assert out[0].shape == (0, 1, 128)


def test_offsets_past_32_bits():
    """Slots past 2^31 elements and 2^32 bytes of the pools."""
    P, H = 256, 8
    pool = 2 ** 32 // (P * H * 128) + 2
    k, v = (torch.zeros(pool, P, H, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = ref.gen(1)
    new = random_bits((300, H, 128), torch.bfloat16, g)
    table = i32([[pool - 1, pool - 2]])
    cpa.cpa_cache_append(new, new, k, v, table, i32([0, 300]), i32([300]), check=True)
    got = cpa.cpa_cache_gather(k, v, table, i32([0, 300]), T=300, check=True)
    for o, x in zip(got, (k, v)):
        assert torch.equal(bits(o), bits(new))
        assert torch.equal(bits(x[-1]), bits(new[:256])) and torch.equal(bits(x[-2, :44]), bits(new[256:]))
        assert int(x.view(torch.int16)[:-2].count_nonzero()) == 0


def test_streams_and_graphs():
    """A captured decode step's append, replayed with other rows and lengths, on its own stream."""
    g = ref.gen(4)
    B, P, H = 9, 16, 4
    lens = list(range(30, 30 + B))
    table, pool = ref.table_of([64] * B, P, g)
    new = [torch.randn(B, H, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    scale = [torch.rand(1, generator=g, device="cuda") * 0.01 + 0.01 for _ in "kv"]
    pages = [torch.zeros(pool, P, H, 128, dtype=torch.uint8, device="cuda") for _ in "kv"]
    st, n = i32(list(range(B + 1))), i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cpa.cpa_cache_append_fp8(*new, *pages, *scale, table, st, n, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cpa_cache_append_fp8(*new, *pages, *scale, table, st, n)
        out = cpa.cpa_cache_gather_fp8(*pages, *scale, table, st, T=B, first=n - 1)
    for step in range(3):
        for x in new:
            x.copy_(torch.randn(B, H, 128, generator=g, device="cuda"))
        n.add_(1)
        graph.replay()
        at = table[torch.arange(B), ((n - 1) // P).long()].long() * P + ((n - 1) % P).long()
        for x, p, s, o in zip(new, pages, scale, out):
            want = quantised(x, s)
            assert torch.equal(p.view(-1, H, 128)[at], want)
            assert torch.equal(o, (want.view(torch.float8_e4m3fn).float() * s).to(torch.bfloat16))


def test_binding_refuses():
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    t, s, n = i32([[0], [1]]), i32([0, 1, 3]), i32([1, 2])
    for bad in (new.transpose(0, 1).contiguous().transpose(0, 1), new[..., ::2], new[:, :1], new[0]):
        with pytest.raises(ValueError):
            cpa.cpa_cache_append(bad, new, k, k, t, s, n)
    with pytest.raises(TypeError):
        cpa.cpa_cache_append(new.half(), new, k, k, t, s, n)
    with pytest.raises(ValueError, match="row for each request"):
        cpa.cpa_cache_append(new, new, k, k, t, s[:2], n)
    with pytest.raises(ValueError, match="row for each request"):
        cpa.cpa_cache_append(new, new, k, k, t, s, n[:1])
    with pytest.raises(ValueError, match="T, the number"):
        cpa.cpa_cache_gather(k, k, t, s)
    with pytest.raises(ValueError, match="the output has"):
        cpa.cpa_cache_gather(k, k, t, s, T=4, k_out=new)
    with pytest.raises(ValueError, match="shape"):
        cpa.cpa_cache_gather(k, k, t, s, k_out=new, v_out=new[:2].clone())
    with pytest.raises(TypeError):
        cpa.cpa_cache_append_fp8(new, new, k, k, torch.ones(1, device="cuda"), torch.ones(1, device="cuda"), t, s, n)
    with pytest.raises(ValueError, match="1 or H_kv"):
        cpa.cpa_cache_gather_fp8(k.byte(), k.byte(), torch.ones(2, device="cuda"), torch.ones(2, device="cuda"), t, s, T=3)
    odd = torch.zeros(3, 257, dtype=torch.bfloat16, device="cuda")[:, :256].view(3, 2, 128)
    with pytest.raises(cpa.CpaError, match="INVALID_ARG"):
        cpa.cpa_cache_append(odd, new, k, k, t, s, n)
    with pytest.raises(ValueError, match="576"):
        cpa.cpa_latent_gather(k.view(4, 16, 256), t, s, T=3)


@pytest.mark.parametrize("B", [3, 9000])
def test_a_call_without_rows_looks_its_requests_over(B):
    """T = 0: starts and lengths are looked at all the same, and nothing is written."""
    k = torch.full((4, 16, 1, 128), 3.0, device="cuda").to(torch.bfloat16)
    lat = torch.full((4, 16, 576), 3.0, device="cuda").to(torch.bfloat16)
    one = torch.ones(1, device="cuda")
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    c, r = none.new_empty(0, 512), none.new_empty(0, 64)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    good, lens = i32([0] * (B + 1)), i32([0, 16] + [5] * (B - 2))

    def status(start, n):
        out = []
        for call in (lambda: cpa.cpa_cache_append(none, none, k, k, table, start, n, workspace=ws),
                     lambda: cpa.cpa_cache_append_fp8(none, none, k.view(torch.uint8)[..., :128].contiguous(),
                                                      k.view(torch.uint8)[..., :128].contiguous(), one, one, table,
                                                      start, n, workspace=ws),
                     lambda: cpa.cpa_latent_append(c, r, lat, table, start, n, workspace=ws),
                     lambda: cpa.cpa_cache_gather(k, k, table, start, T=0, first=n, workspace=ws),
                     lambda: cpa.cpa_latent_gather(lat, table, start, T=0, first=n, workspace=ws)):
            ws.fill_(0xFF)
            call()
            out.append(cpa.cpa_get_device_status(ws)[0])
        return out

    assert status(good, lens) == [0] * 5
    for at, x in ((B, 5), (0, -1), (B // 2, 1), (B // 2, -1)):
        bad = good.clone()
        bad[at] = x
        assert status(bad, lens) == [8] * 5, (at, x)
    for x in (-1, 17, 2 ** 31 - 1, -2 ** 31):
        n = lens.clone()
        n[B - 1] = x
        assert status(good, n) == [8] * 5, x
    assert bool((k == 3).all()) and bool((lat == 3).all())


EDGE_SCALES = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), 2.0 ** -120, -2.0 ** -120, 2.0 ** 120,
               -2.0 ** 120, 2.0 ** -149, 3.0e38, 2.0 ** -100, 2.0 ** 100, -0.013, -1.0, -3.0, 2.0 ** -7, 0.5, 1.0,
               3.0, 0.007, 0.25, 1.1, 2.0 ** -9]


def test_fp8_scales_of_every_kind():
    """0, infinities, NaN, scales too far from 1 for their reciprocal, negative ones; powers of two and
    others side by side in one group of channels; over values of every kind."""
    g = ref.gen(31)
    H, P, T = 2, 16, 600
    scale = [torch.empty(H, 128, device="cuda") for _ in "kv"]
    for i, s in enumerate(scale):
        order = torch.randint(0, len(EDGE_SCALES), (H * 128,), generator=g, device="cuda")
        order[:len(EDGE_SCALES)] = torch.arange(len(EDGE_SCALES), device="cuda")
        s.copy_(torch.tensor(EDGE_SCALES, device="cuda")[order].view(H, 128))
        s[1, 64:] = torch.rand(64, generator=g, device="cuda") * 0.02 + 0.001
        s[1, 64::3] = 2.0 ** -6
    new = [torch.randn(T, H, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    special = torch.tensor([0.0, -0.0, 1e30, -1e30, float("inf"), float("-inf"), float("nan"), 1e-30, -1e-30, 1e-38,
                            448.0, 1.0], device="cuda").to(torch.bfloat16)
    for x in new:
        x[:len(special)] = special[:, None, None]
    check_fp8(new, scale, P)
    for one in EDGE_SCALES:  # one scale for all channels
        check_fp8(new, [torch.tensor([one], device="cuda"), torch.tensor([-one], device="cuda")], P)


def test_fp8_values_beside_the_borders_of_codes():
    """The bf16 values nearest to (the middle between two codes) x scale, and those beside them."""
    P, H = 16, 1
    g = ref.gen(32)
    codes = torch.arange(0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    mid = (codes[1:] + codes[:-1]) / 2                                  # 126 of them
    scale = torch.exp(torch.randn(128, generator=g, device="cuda") * 3)
    scale[::9] = torch.exp2(torch.randint(-12, 12, scale[::9].shape, generator=g, device="cuda").float())
    x = (mid[:, None] * scale).to(torch.bfloat16).view(torch.int16)     # positive: bit patterns ascend
    x = torch.cat([x + i for i in (-1, 0, 1)]).view(torch.bfloat16)
    x = torch.cat([x, -x]).view(-1, H, 128)
    check_fp8([x, x.flip(0)], [scale.view(H, 128), scale.view(H, 128)], P)


def check_fp8(new, scale, P):
    """Appended and read back, against PyTorch's quotient and product."""
    T, H = new[0].shape[:2]
    n = (T + P - 1) // P
    table, st, lens = i32([list(range(n))[::-1]]), i32([0, T]), i32([T])
    pages = [torch.zeros(n, P, H, 128, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cpa.cpa_cache_append_fp8(*new, *pages, *scale, table, st, lens, check=True)
    pos = torch.arange(T, device="cuda")
    codes = [p[table[0].long()[pos // P], pos % P] for p in pages]
    for c, x, s in zip(codes, new, scale):
        same_codes(c, quantised(x, s))
    back = cpa.cpa_cache_gather_fp8(*pages, *scale, table, st, T=T, check=True)
    for o, c, s in zip(back, codes, scale):
        w = (c.view(torch.float8_e4m3fn).float() * s).to(torch.bfloat16)
        assert torch.equal(torch.isnan(o), torch.isnan(w))
        assert torch.equal(o[~torch.isnan(w)], w[~torch.isnan(w)])
