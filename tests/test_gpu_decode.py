"""Decode over the paged cache against a 64-bit reference: lengths from none to
long, odd groups, windows and sinks, FP8 pages, splits, refusals by the device."""
import math

import pytest
import torch

import cascade_paged_attention_gb300 as cpa
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

EDGE_LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 300]


def make(lens, H_q, H_kv, P, seed, fp8=False, per_channel=True, hide=None):
    g = ref.gen(seed)
    table, pool = ref.table_of(lens, P, g)
    q = torch.randn(len(lens), H_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    if fp8:
        k, v = (torch.randn(pool, P, H_kv, 128, generator=g, device="cuda")
                .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
        n = (H_kv, 128) if per_channel else (1,)
        ks, vs = (torch.rand(n, generator=g, device="cuda") * 0.5 + 0.5 for _ in range(2))
    else:
        k, v = ref.pool_of(pool, P, H_kv, g), ref.pool_of(pool, P, H_kv, g)
        ks = vs = None
    return q, k, v, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(lens, H_q, H_kv, P, window=0, sinks=0, seed=0, fp8=False, per_channel=True, hide=True,
          max_len=None):
    q, k, v, ks, vs, table, dl = make(lens, H_q, H_kv, P, seed, fp8, per_channel)
    full = table.clone()
    masks = [ref.seen([L - 1], L, window, sinks, "cuda")[0] for L in lens]
    if hide:
        ref.hide_unseen(k, v, table, lens, masks, P)
    kw = dict(window=window, sinks=sinks, check=True, max_seq_len=max_len)
    if fp8:
        o, lse = cpa.cpa_decode_fp8(q, k, v, ks, vs, table, dl, **kw)
    else:
        o, lse = cpa.cpa_decode(q, k, v, table, dl, **kw)
    if hide:  # (the reference multiplies what it does not see by 0)
        for x in (k, v):
            if fp8:
                x[x == 0x7F] = 0
            else:
                x.nan_to_num_(0.0)
    for b, L in enumerate(lens):
        K = ref.dense(k, full[b], L, P, ks)
        V = ref.dense(v, full[b], L, P, vs)
        want = ref.attend(q[b:b + 1], K, V, masks[b][None], 128 ** -0.5,
                          ref.E_F16 if fp8 else ref.E_P_SPLIT, ref.E_Q_SPLIT if fp8 else 0.0)
        ref.close(o[b:b + 1], lse[b:b + 1], want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H_q,H_kv,P", [(32, 8, 16), (8, 8, 8), (3, 1, 64), (10, 2, 256), (64, 8, 32),
                                        (28, 4, 16), (12, 1, 128), (32, 2, 16), (40, 1, 8),
                                        (1, 1, 16), (130, 1, 32)])
def test_edge_lengths_and_groups(H_q, H_kv, P, fp8):
    check(EDGE_LENS, H_q, H_kv, P, seed=H_q, fp8=fp8)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (64, 4), (100, 130),
                                          (128, 16), (1000, 4), (7, 1000)])
@pytest.mark.parametrize("P", [8, 16, 64])
def test_windows_and_sinks(window, sinks, P):
    check(EDGE_LENS + [1111, 2050], 16, 4, P, window, sinks, seed=window + P)


@pytest.mark.parametrize("per_channel", [True, False])
def test_fp8_scales_and_window(per_channel):
    check([0, 5, 200, 777, 1500], 16, 2, 16, 300, 4, seed=3, fp8=True, per_channel=per_channel)


@pytest.mark.parametrize("B,lo,hi,H_q,H_kv,P", [(1, 9000, 9000, 32, 8, 16), (2, 1, 40000, 8, 1, 64),
                                               (70, 1, 3000, 32, 8, 16), (1, 20001, 20001, 16, 1, 16),
                                               (600, 0, 90, 8, 2, 16), (5, 1000, 1100, 64, 4, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_split_lengths(B, lo, hi, H_q, H_kv, P, fp8):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    check(lens, H_q, H_kv, P, seed=B, fp8=fp8, hide=False)
    check(lens, H_q, H_kv, P, window=700, sinks=5, seed=B + 1, fp8=fp8, hide=False)


def test_scores_that_grow_and_shrink():
    """Keys whose scores climb over the sequence by far more than 2^8, then fall: the running
    maximum moves many times, and weights that round to 0 stay 0."""
    q, k, v, _, _, table, dl = make([1500, 700], 8, 2, 16, 5)
    for b, L in enumerate([1500, 700]):
        pos = torch.arange(L, device="cuda")
        ramp = (torch.sin(pos / 90.0) * 40).to(torch.bfloat16)
        k[table[b].long()[pos // 16], pos % 16] = \
            (q[b].view(2, 4, 128)[:, 0] / 12).to(torch.bfloat16)[None] * ramp[:, None, None]
    o, lse = cpa.cpa_decode(q, k, v, table, dl, check=True)
    for b, L in enumerate([1500, 700]):
        m = ref.seen([L - 1], L, 0, 0, "cuda")
        ref.close(o[b:b + 1], lse[b:b + 1],
                  ref.attend(q[b:b + 1], ref.dense(k, table[b], L, 16),
                             ref.dense(v, table[b], L, 16), m, 128 ** -0.5))


def test_scale_output_buffers_and_repeat():
    """A given sm_scale and given buffers; the same call twice gives the same bits."""
    lens = [4000, 1, 333, 12000]
    q, k, v, _, _, table, dl = make(lens, 32, 8, 16, 9)
    o, lse = torch.empty_like(q), torch.empty(4, 32, device="cuda")
    ws = torch.full((cpa.cpa_decode_workspace_size(4, 32, 8, 128, 16),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    r = cpa.cpa_decode(q, k, v, table, dl, sm_scale=0.03, o=o, lse=lse, workspace=ws, check=True)
    assert r[0] is o and r[1] is lse
    for b, L in enumerate(lens):
        ref.close(o[b:b + 1], lse[b:b + 1],
                  ref.attend(q[b:b + 1], ref.dense(k, table[b], L, 16),
                             ref.dense(v, table[b], L, 16), ref.seen([L - 1], L, 0, 0, "cuda"), 0.03))
    ws.fill_(0x5A)
    o2, lse2 = cpa.cpa_decode(q, k, v, table, dl, sm_scale=0.03, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_nan_and_infinity_that_are_seen():
    """A NaN among the seen values reaches the rows that see it and no other; FP8 NaN codes too."""
    q, k, v, _, _, table, dl = make([200, 200], 4, 2, 16, 11)
    v[table[0, 3].long(), 5, 1, 17] = float("nan")
    o, lse = cpa.cpa_decode(q, k, v, table, dl, check=True)
    bad = torch.isnan(o)
    assert bool(bad[0, 2:, 17].all()) and int(bad.sum()) == 2
    assert bool(torch.isfinite(lse).all())
    q, k, v, ks, vs, table, dl = make([200, 200], 4, 2, 16, 12, fp8=True)
    v[table[1, 0].long(), 0, 0, 3] = 0xFF
    o, lse = cpa.cpa_decode_fp8(q, k, v, ks, vs, table, dl, check=True)
    bad = torch.isnan(o)
    assert bool(bad[1, :2, 3].all()) and int(bad.sum()) == 2


def test_bad_pages_and_lengths_are_reported():
    q, k, v, _, _, table, dl = make([300, 300], 8, 2, 16, 13)
    good = table.clone()
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table.copy_(good)
        table[1, 7] = bad
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_decode(q, k, v, table, dl, check=True)
        assert e.value.status == 5
        # outside the window it is not read
        cpa.cpa_decode(q, k, v, table, dl, window=100, check=True)
    table.copy_(good)
    for bad in (-1, 305, 2 ** 31 - 1, -2 ** 31):
        dl[0] = bad
        with pytest.raises(cpa.CpaError) as e:
            cpa.cpa_decode(q, k, v, table, dl, check=True)
        assert e.value.status == 8
    dl[0] = 300
    cpa.cpa_decode(q, k, v, table, dl, check=True)  # the next clean call clears the word


def test_graph_replay_with_growing_lengths():
    """One capture serves every step: lengths, tables and queries change in place."""
    lens = [700, 30, 1]
    q, k, v, _, _, table, dl = make([x + 40 for x in lens], 16, 4, 16, 17)
    dl.copy_(torch.tensor(lens, dtype=torch.int32))
    o, lse = torch.empty_like(q), torch.empty(3, 16, device="cuda")
    cpa.cpa_decode(q, k, v, table, dl, window=256, sinks=4, o=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cpa_decode(q, k, v, table, dl, window=256, sinks=4, o=o, lse=lse)
    for step in range(4):
        dl += 9
        q.normal_()
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for b, L in enumerate(dl.tolist()):
            ref.close(o[b:b + 1], lse[b:b + 1],
                      ref.attend(q[b:b + 1], ref.dense(k, table[b], L, 16),
                                 ref.dense(v, table[b], L, 16),
                                 ref.seen([L - 1], L, 256, 4, "cuda"), 128 ** -0.5))


def test_two_streams_and_two_graphs_share_nothing():
    """Calls on two streams at once, and two captured graphs replayed at once, without a
    workspace from the caller."""
    a = make([9000, 4000], 32, 8, 16, 19)
    b = make([7000, 5000], 32, 8, 16, 20)
    want = [cpa.cpa_decode(x[0], x[1], x[2], x[5], x[6], check=True) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for x, s in zip((a, b), streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(cpa.cpa_decode(x[0], x[1], x[2], x[5], x[6]))
        graphs.append(gr)
    for _ in range(20):
        got = []
        for x, s, gr in zip((a, b), streams, graphs):
            with torch.cuda.stream(s):
                got.append(cpa.cpa_decode(x[0], x[1], x[2], x[5], x[6]))
                gr.replay()
        torch.cuda.synchronize()
        for r, o, w in zip(got, outs, want):
            assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_agrees_with_cascade_verify_of_one_token():
    """topk = 1, S = 1 over a prefix of L - 1 tokens is the same attention."""
    lens = [300, 1000, 17]
    q, k, v, _, _, table, dl = make(lens, 32, 8, 16, 23)
    o, lse = cpa.cpa_decode(q, k, v, table, dl, check=True)
    k2, v2 = torch.cat([k, k[:3]]), torch.cat([v, v[:3]])
    draft = torch.arange(3, dtype=torch.int32, device="cuda")[:, None] + k.shape[0]
    for b, L in enumerate(lens):
        pg = table[b, (L - 1) // 16].long()
        for x, y in ((k2, k), (v2, v)):
            x[k.shape[0] + b, 0] = y[pg, (L - 1) % 16]
    o2, lse2 = cpa.cpa_cascade_verify(q, k2, v2, table, draft.contiguous(), dl - 1, 1, 1, check=True)
    # both round o to bf16 once; verify's weights are bf16 (2^-8 each way)
    assert float((o.float() - o2.float()).abs().max()) <= 1e-2
    assert float((lse - lse2).abs().max()) <= 1e-3


def test_many_requests_and_a_stream_of_ones_own():
    """Thousands of short requests (several a thread in the split of the work), on a stream given
    by argument."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (3001,), generator=g).tolist()
    q, k, v, _, _, table, dl = make(lens, 8, 2, 8, 41)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = cpa.cpa_decode(q, k, v, table, dl, stream=side, check=True)
    torch.cuda.current_stream().wait_stream(side)
    pos = torch.arange(40, device="cuda")
    idx = table.long()[:, pos // 8].clamp(min=0)
    K, V = k[idx, pos % 8].double(), v[idx, pos % 8].double()
    seen = pos[None] < dl[:, None]
    x = torch.einsum("bhgd,bjhd->bhgj", q.double().view(-1, 2, 4, 128), K) * 128 ** -0.5
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    want = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(want == float("-inf"), 0.0, want)[..., None])
    wo = torch.einsum("bhgj,bjhd->bhgd", w, V)
    none = (dl == 0)
    assert bool((o[none] == 0).all()) and bool((lse[none] == float("-inf")).all())
    # half a step of bf16, and weights to 2^-15 (see tests/paged_ref.py)
    tol = 2.0 ** -8 * wo.abs() + 2.0 ** -14 * torch.einsum("bhgj,bjhd->bhgd", w, V.abs())
    assert bool(((o.double().view_as(wo) - wo).abs() <= tol).all())
    assert float((lse.double().view_as(want) - want)[~none].abs().max()) <= 1e-4


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spare", [-1, 0, 1])
def test_tiles_around_the_blocks(spare, fp8):
    """Around two tiles for every block, the fewest that a block takes; odd tiles last."""
    blocks = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    for tiles in (2 * blocks + spare, 2 * (blocks // 4) + spare):
        check([64 * tiles], 4, 1, 64, seed=tiles, fp8=fp8, hide=False)
        check([64 * (tiles - 3) - 1, 65, 64], 8, 1, 16, seed=tiles + 1, fp8=fp8, hide=False)


@pytest.mark.parametrize("H_kv", [1, 2])
@pytest.mark.parametrize("bits", [12.4, 20.5])
@pytest.mark.parametrize("many,L", [(False, 300), (True, 20000)])
def test_fp8_weights_far_below_the_largest(many, L, bits, H_kv):
    """One key `bits` powers of two above all others, whose own value is 0: the output is made
    of the small weights alone.  Many requests over the same pages, so that one block walks a
    whole one.  f16 holds a lifted weight to 2^-11 of itself down to 2^-21 of the largest."""
    B = 3 * torch.cuda.get_device_properties(0).multi_processor_count // H_kv if many else 1
    g = ref.gen(L)
    table, pool = ref.table_of([L], 16, g)
    k = torch.zeros(pool, 16, H_kv, 128, dtype=torch.uint8, device="cuda")
    v = torch.randn(pool, 16, H_kv, 128, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    k[table[0, 0].long(), 0] = 0x38  # 1.0
    v[table[0, 0].long(), 0] = 0
    ks, vs = torch.ones(1, device="cuda"), torch.full((1,), 0.75, device="cuda")
    q = torch.ones(B, 4 * H_kv, 128, dtype=torch.bfloat16, device="cuda")
    scale = bits * math.log(2) / 128  # (the strong key's score is 128 * scale, the others' 0)
    o, lse = cpa.cpa_decode_fp8(q, k, v, ks, vs, table.expand(B, -1).contiguous(),
                                torch.full((B,), L, dtype=torch.int32, device="cuda"),
                                sm_scale=scale, check=True)
    want = ref.attend(q[:1], ref.dense(k, table[0], L, 16, ks), ref.dense(v, table[0], L, 16, vs),
                      ref.seen([L - 1], L, 0, 0, "cuda"), scale, ref.E_F16, ref.E_Q_SPLIT)
    for b in range(0, B, 37):
        ref.close(o[b:b + 1], lse[b:b + 1], want)


@pytest.mark.parametrize("step", [0.9, 6.9, 7.1, 40.0])
def test_fp8_scores_that_grow_and_shrink(step):
    """FP8 scores that climb by `step` powers of two a key, then fall: the running maximum lags
    by up to 2^7, and the lifted weights stay within f16."""
    L = 400
    g = ref.gen(int(step * 10))
    table, pool = ref.table_of([L, L], 16, g)
    v = torch.randn(pool, 16, 1, 128, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    k = torch.zeros(pool, 16, 1, 128, device="cuda")
    level = (8 - (torch.arange(L, device="cuda") % 33 - 16).abs() / 2)  # 0 .. 8 and back
    pos = torch.arange(L, device="cuda")
    for b in range(2):
        k[table[b].long()[pos // 16], pos % 16] = level[:, None, None].expand(L, 1, 128)
    k = k.to(torch.float8_e4m3fn).view(torch.uint8)
    ks, vs = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    q = torch.ones(2, 6, 128, dtype=torch.bfloat16, device="cuda")
    scale = 2 * step * math.log(2) / 128
    o, lse = cpa.cpa_decode_fp8(q, k, v, ks, vs, table,
                                torch.full((2,), L, dtype=torch.int32, device="cuda"),
                                sm_scale=scale, check=True)
    for b in range(2):
        ref.close(o[b:b + 1], lse[b:b + 1], ref.attend(
            q[b:b + 1], ref.dense(k, table[b], L, 16, ks), ref.dense(v, table[b], L, 16, vs),
            ref.seen([L - 1], L, 0, 0, "cuda"), scale, ref.E_F16, ref.E_Q_SPLIT))


@pytest.mark.parametrize("H_q,H_kv", [(8, 2), (12, 1)])
def test_infinities_in_v(H_q, H_kv):
    """An infinity in V that a row sees is one in its output (two of unlike sign: a NaN), also
    where weights are 1 or any other value that bf16 holds; nothing else changes."""
    lens = [1, 2, 200, 9000]
    q, k, v, _, _, table, dl = make(lens, H_q, H_kv, 16, 51)
    inf = float("inf")
    for b, at, c, x in ((0, 0, 3, inf), (0, 0, 4, -inf), (1, 0, 9, -inf), (1, 1, 10, inf), (2, 3, 17, inf),
                        (2, 77, 40, -inf), (2, 5, 41, inf), (2, 199, 41, -inf), (3, 4000, 5, inf),
                        (3, 20, 99, -inf), (3, 8999, 98, inf), (3, 0, 97, inf), (3, 8000, 97, inf)):
        v[table[b, at // 16].long(), at % 16, H_kv - 1, c] = x
    o, lse = cpa.cpa_decode(q, k, v, table, dl, check=True)
    for b, L in enumerate(lens):
        want = ref.attend(q[b:b + 1], ref.dense(k, table[b], L, 16), ref.dense(v, table[b], L, 16),
                          ref.seen([L - 1], L, 0, 0, "cuda"), 128 ** -0.5)
        got, w = o[b:b + 1].double(), want[0]
        odd = ~torch.isfinite(w)
        assert torch.equal(got[odd].nan_to_num(nan=7.0), w[odd].nan_to_num(nan=7.0))
        assert int(odd.sum()) == H_q // H_kv * {0: 2, 1: 2, 2: 3, 3: 4}[b]
        ref.close(torch.where(odd, 0.0, got), lse[b:b + 1],
                  [torch.where(odd, 0.0, w), want[1], torch.where(odd, 0.0, want[2]), want[3]])


def test_numbers_past_32_bits_are_refused():
    """The C entry points take 32 bits: a larger number is not cut to them."""
    q, k, v, _, _, table, dl = make([200], 8, 2, 16, 61)
    qs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for name in ("window", "sinks", "max_seq_len", "max_new"):
        for x in (2 ** 31, 2 ** 32, 2 ** 32 + 200, -2 ** 31 - 1):
            if name != "max_new":
                with pytest.raises(ValueError, match=name):
                    cpa.cpa_decode(q, k, v, table, dl, **{name: x})
            with pytest.raises(ValueError, match=name):
                cpa.cpa_window_prefill(q, k, v, table, qs, dl, **{name: x})
    with pytest.raises(ValueError, match="page_size"):
        cpa.cpa_cache_fork(table, dl, dl, dl, dl, 2 ** 32 + 16)
    # the largest number is as good as none
    o, lse = cpa.cpa_decode(q, k, v, table, dl, check=True)
    for kw in (dict(window=2 ** 31 - 1), dict(window=3, sinks=2 ** 31 - 1),
               dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1)):
        o2, lse2 = cpa.cpa_decode(q, k, v, table, dl, check=True, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o, lse = cpa.cpa_window_prefill(q, k, v, table, qs, dl, check=True)
    for kw in (dict(window=2 ** 31 - 1), dict(window=3, sinks=2 ** 31 - 1),
               dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(max_new=2 ** 31 - 1)):
        o2, lse2 = cpa.cpa_window_prefill(q, k, v, table, qs, dl, check=True, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_table_wider_than_any_sequence():
    """2^23 + 1 columns of pages of 256: more than 2^31 tokens, of which a sequence may have 2^30."""
    q, k, v, _, _, table, dl = make([300], 8, 2, 256, 62)
    wide = torch.full((1, 2 ** 23 + 1), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    qs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for a, b in ((cpa.cpa_decode(q, k, v, table, dl, check=True),
                  cpa.cpa_decode(q, k, v, wide, dl, check=True)),
                 (cpa.cpa_window_prefill(q, k, v, table, qs, dl, check=True),
                  cpa.cpa_window_prefill(q, k, v, wide, qs, dl, check=True))):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
