"""Latent attention, absorbed and expanded, against a 64-bit reference."""
import pytest
import torch

import cascade_paged_attention_gb300 as cpa
from tests import latent_ref as lref
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
C, R, D = lref.C, lref.R, lref.D


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


# ----------------------------------------------------------------- absorbed
def make(lens, S, H, P, seed, spare=2, width=None):
    g = ref.gen(seed)
    table, pool = ref.table_of(lens, P, g, spare, width)
    n = len(lens) * S
    return (randn(n, H, C, g=g), randn(n, H, R, g=g), randn(pool, P, C + R, g=g), table, i32(lens))


def visible(L, S):
    """[S, L]: the keys that each token of a request sees."""
    p = torch.arange(L - S, L, device="cuda")[:, None]
    return torch.arange(L, device="cuda")[None] <= p


def hide(pages, table, lens, P):
    """NaN in every slot past a sequence's end, -1 for pages that no sequence has."""
    keep = torch.zeros(pages.shape[0] * P, dtype=torch.bool, device="cuda")
    for b, L in enumerate(lens):
        pos = torch.arange(L, device="cuda")
        keep[table[b].long()[pos // P] * P + pos % P] = True
    pages.view(-1, C + R)[~keep] = float("nan")


def against(q_c, q_r, pages, table, lens, S, o, lse, P, scale=lref.SCALE, rows=None):
    for b, L in enumerate(lens):
        pos = torch.arange(L, device="cuda")
        lat = pages[table[b].long()[pos // P], pos % P]
        r = slice(b * S, (b + 1) * S)
        ref.close(o[r], lse[r], lref.absorbed(q_c[r], q_r[r], lat, visible(L, S), scale))


def check(lens, S, H, P, seed=0, **kw):
    q_c, q_r, pages, table, dl = make(lens, S, H, P, seed)
    hide(pages, table, lens, P)
    o = torch.full((len(lens) * S, H, C), 7.0, device="cuda").to(torch.bfloat16)
    lse = torch.full((len(lens) * S, H), 7.0, device="cuda")
    cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, o=o, lse=lse, check=True, **kw)
    against(q_c, q_r, pages, table, lens, S, o, lse, P)


LENS = [0, 1, 2, 5, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("H", [1, 2, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_heads_of_one_tile(H):
    check(LENS, 1, H, 16, seed=H)


@pytest.mark.parametrize("H", [65, 80, 96, 127, 128, 130, 200])
def test_heads_of_many_tiles(H):
    check(LENS, 1, H, 16, seed=H)


@pytest.mark.parametrize("S,H", [(2, 1), (2, 16), (3, 20), (5, 32), (7, 9), (4, 64), (3, 65),
                                 (2, 128), (6, 5), (33, 2), (64, 1), (50, 3)])
def test_tokens_causal_among_themselves(S, H):
    check(LENS, S, H, 16, seed=S + H)


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("S,H", [(1, 16), (1, 128), (4, 40)])
def test_page_sizes(P, S, H):
    check([1, 7, 40, 255, 256, 257, 777], S, H, P, seed=P)


@pytest.mark.parametrize("lens", [[20000], [9000, 3], [1] * 300, [2000] * 20, [0, 0, 0], [0, 5000],
                                  [130] * 200 + [6000]])
@pytest.mark.parametrize("S,H", [(1, 16), (1, 128), (3, 32)])
def test_batches_and_splits(lens, S, H):
    check(lens, S, H, 16, seed=len(lens) + H)


def test_thousands_of_requests():
    """More requests than blocks and warps, none to a few tokens each, two tokens of queries."""
    B, S, H, P = 4099, 2, 3, 8
    g = ref.gen(21)
    lens = torch.randint(0, 12, (B,), generator=g, device="cuda").tolist()
    q_c, q_r, pages, table, dl = make(lens, S, H, P, 22)
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
    pos = torch.arange(12, device="cuda")
    page = table[:, (pos // P).clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    lat = pages[page, pos % P].double()                                   # [B, 12, C + R]
    q = torch.cat([q_c, q_r], 2).double().view(B, S, H, C + R)
    p = dl.long()[:, None] - S + torch.arange(S, device="cuda")[None]
    mask = pos[None, None] <= p[..., None]                                # [B, S, 12]
    x = torch.einsum("bshd,bjd->bshj", q, lat) * lref.SCALE
    big = torch.einsum("bshd,bjd->bshj", q.abs(), lat.abs()) * lref.SCALE
    x = x.masked_fill(~mask[:, :, None], float("-inf"))
    ds = big.masked_fill(~mask[:, :, None], 0.0).amax(-1) * (C + R) * 2.0 ** -23
    z = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(z == float("-inf"), 0.0, z)[..., None])
    want = torch.einsum("bshj,bjc->bshc", w, lat[..., :C])
    size = torch.einsum("bshj,bjc->bshc", w, lat[..., :C].abs())
    tol = ref.U_BF16 * want.abs() + (ref.E_P_BF16 + 2 * ds + 2.0 ** -18)[..., None] * size
    tol_l = ds + 2.0 ** -20 * (1 + torch.where(z == float("-inf"), 0.0, z).abs())
    ref.close(o, lse, [y.reshape(B * S, *y.shape[2:]) for y in (want, z, tol, tol_l)])



def test_bounds_given_and_repeat():
    """The same call twice gives the same bits, whatever its workspace held."""
    lens = [1000, 3, 900, 5000]
    q_c, q_r, pages, table, dl = make(lens, 2, 128, 16, 2)
    n = cpa.cpa_latent_decode_workspace_size(4, 2, 128, C, R, 16)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    kw = dict(S=2, max_seq_len=5000, workspace=ws, sm_scale=0.05)
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, **kw)
    against(q_c, q_r, pages, table, lens, 2, o, lse, 16, 0.05)
    ws.fill_(0x5A)
    o2, lse2 = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("S,H", [(1, 16), (3, 100), (1, 1), (4, 5)])
def test_queries_as_they_lie(S, H):
    """Heads before tokens (as a batched product leaves them), slices of wider rows."""
    lens = [5, 300, 64]
    q_c, q_r, pages, table, dl = make(lens, S, H, 16, 7)
    g = ref.gen(8)
    want = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S)
    head_first = q_c.transpose(0, 1).contiguous().transpose(0, 1)
    wide = randn(len(lens) * S, H, D + R, g=g)
    wide[..., D:] = q_r
    both = randn(len(lens) * S + 1, H + 2, C + R + 24, g=g)[1:, 1:-1]
    both[..., 8:8 + C], both[..., 8 + C:8 + C + R] = q_c, q_r
    for a, b in ((head_first, wide[..., D:]), (both[..., 8:8 + C], both[..., 8 + C:8 + C + R])):
        got = cpa.cpa_latent_decode(a, b, pages, table, dl, S=S, check=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_scores_that_grow():
    """Scores that climb along the keys by far more than 2^8: the running maximum moves often."""
    lens, P = [900, 130], 16
    for S, H in ((1, 20), (2, 128)):
        q_c, q_r, pages, table, dl = make(lens, S, H, P, 5)
        q_c.copy_(q_c[:1, :1].expand_as(q_c))
        for b, L in enumerate(lens):
            pos = torch.arange(L, device="cuda")
            pages[table[b].long()[pos // P], pos % P, :C] = \
                (q_c[0, 0] / 24)[None] * (pos / 20).to(torch.bfloat16)[:, None]
        o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
        against(q_c, q_r, pages, table, lens, S, o, lse, P)
        pages.neg_()
        o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
        against(q_c, q_r, pages, table, lens, S, o, lse, P)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lens", [[300, 90], [5000, 90]])
def test_values_that_are_not_numbers(value, lens):
    """In a draft's latent: the drafts before it do not see it.  In a request's: no other does."""
    S, H, P = 4, 20, 16
    q_c, q_r, pages, table, dl = make(lens, S, H, P, 11)
    at = lens[0] - 2  # seen by the last two tokens
    clean = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
    pages[table[0, at // P].long(), at % P, 9] = value
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
    finite = torch.isfinite(o.float())
    assert not bool(finite[2:4, :, 9].any())
    lat_row = pages[table[0, at // P].long(), at % P].clone()
    pages[table[0, at // P].long(), at % P, 9] = 0.0
    against(q_c[4:], q_r[4:], pages, table[1:], lens[1:], S, o[4:], lse[4:], P)
    pos = torch.arange(lens[0], device="cuda")
    lat = pages[table[0].long()[pos // P], pos % P]
    ref.close(o[:2], lse[:2], lref.absorbed(q_c[:2], q_r[:2], lat, visible(lens[0], S)[:2]))
    assert torch.equal(clean[0][4:], o[4:])
    # (a score that is infinite or not a number takes the whole row with it)
    x = q_c[2:4, :, 9].float() * lat_row[9].float()
    assert not bool(torch.isfinite(lse[2:4])[torch.isnan(x) | (x > 0)].any())


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("L", [3, 65, 300, 5000])
def test_an_infinite_latent_is_the_same_wherever_it_lies(value, L):
    """Its score is infinite.  Minus infinity: weight 0, and 0 x infinity in its own column, whether
    all of a request's tokens see the key or only the last ones; plus infinity: the whole row."""
    S, H, P = 4, 20, 16
    lens = [L, 40]
    for at in sorted({1, L - 1, L - 2, L - 3, L - 4, L // 2} & set(range(1, L))):
        q_c, q_r, pages, table, dl = make(lens, S, H, P, 13)
        where = (table[0, at // P].long(), at % P, 9)
        pages[where] = 0.0
        pos = torch.arange(L, device="cuda")
        lat = pages[table[0].long()[pos // P], pos % P].clone()
        pages[where] = value
        o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, check=True)
        last = cpa.cpa_latent_decode(q_c[S - 1::S], q_r[S - 1::S], pages, table, dl, check=True)
        seen = torch.arange(L - S, L, device="cuda")[:, None] >= at
        score = q_c[:S, :, 9].float() * value
        lost, kept = seen & (score > 0), ~(seen & (score > 0))
        assert bool(torch.isnan(o[:S][lost]).all()) and not bool(torch.isfinite(lse[:S][lost]).any())
        hit = seen & (score < 0)
        assert bool(torch.isnan(o[:S, :, 9][hit]).all())
        # all else is as without the key
        mask = visible(L, S) & (pos != at)
        want = lref.absorbed(q_c[:S], q_r[:S], lat, mask)
        got, ref_o = o[:S].clone(), want[0]
        got[:, :, 9][hit] = 0.0
        ref_o[:, :, 9][hit] = 0.0
        ref.close(got[kept], lse[:S][kept], [x[kept] for x in want])
        assert torch.equal(torch.isnan(last[0][0]), torch.isnan(o[S - 1]))
        assert torch.equal(torch.isinf(last[0][0]), torch.isinf(o[S - 1]))
        against(q_c[S:], q_r[S:], pages, table[1:], lens[1:], S, o[S:], lse[S:], P)


def test_unseen_infinite_score():
    """A key whose score is minus infinity has weight 0, in any tile."""
    lens, P = [200], 16
    q_c, q_r, pages, table, dl = make(lens, 1, 16, P, 3)
    q_r[..., 0] = 1.0
    for at in (0, 70, 199):
        pages[table[0, at // P].long(), at % P, C] = float("-inf")  # in the part that is no value
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, check=True)
    assert bool(torch.isfinite(lse).all())
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[torch.tensor([0, 70, 199], device="cuda")] = False
    pos = torch.arange(200, device="cuda")[keep]
    lat = pages[table[0].long()[pos // P], pos % P]
    ref.close(o, lse, lref.absorbed(q_c, q_r, lat, torch.ones(1, 197, dtype=torch.bool, device="cuda")))


def test_bad_pages_and_lengths_are_reported():
    lens = [100, 500, 64]
    q_c, q_r, pages, table, dl = make(lens, 1, 16, 16, 1)
    ws = torch.full((cpa.cpa_latent_decode_workspace_size(3, 1, 16),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    for bad in (pages.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 20] = bad
        cpa.cpa_latent_decode(q_c, q_r, pages, t, dl, workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == 5
    for bad in (-1, 501, 2 ** 31 - 1, -2 ** 31):
        cpa.cpa_latent_decode(q_c, q_r, pages, table, i32([100, bad, 64]), max_seq_len=500, workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == 8
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, max_seq_len=500, workspace=ws)
    assert cpa.cpa_get_device_status(ws) == (0, 0)
    against(q_c, q_r, pages, table, lens, 1, o, lse, 16)


def test_offsets_past_32_bits():
    P = 256
    g = ref.gen(2)
    pool = 2 ** 32 // (P * (C + R)) + 3
    pages = torch.zeros(pool, P, C + R, dtype=torch.bfloat16, device="cuda")
    table = i32([[pool - 1, 0, pool - 3, 1, pool - 2]])
    lens = [5 * P - 100]
    for pg in table[0].tolist():
        pages[pg] = randn(P, C + R, g=g)
    q_c, q_r = randn(2, 64, C, g=g), randn(2, 64, R, g=g)
    o, lse = cpa.cpa_latent_decode(q_c, q_r, pages, table, i32(lens), S=2, check=True)
    against(q_c, q_r, pages, table, lens, 2, o, lse, P)


def test_streams_and_graphs():
    """A captured step replayed as the sequences grow; two graphs that share a workspace run one
    after the other; a call on another stream."""
    lens, S, H, P = [100, 700, 63], 2, 32, 16
    q_c, q_r, pages, table, dl = make([x + 40 for x in lens], S, H, P, 6, width=50)
    dl.copy_(i32(lens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, stream=side, check=True)
    side.synchronize()
    against(q_c, q_r, pages, table, lens, S, *got, P)
    ws = torch.empty(cpa.cpa_latent_decode_workspace_size(3, S, H), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=S, max_seq_len=800, workspace=ws))
        graphs.append(gr)
    for step in range(3):
        lens = [x + 13 for x in lens]
        dl.copy_(i32(lens))
        for gr in graphs:
            gr.replay()
        for out in outs:
            against(q_c, q_r, pages, table, lens, S, *out, P)


def test_calls_one_after_the_other():
    """Appends, decodes and copies of one stream in a graph, each reading what the one before wrote,
    with one workspace: launches that overlap change nothing."""
    H, P, B = 32, 16, 5
    lens = [70, 300, 5, 1000, 64]
    q_c, q_r, pages, table, dl = make([x + 8 for x in lens], 1, H, P, 14, width=64)
    dl.copy_(i32(lens))
    ws = torch.empty(cpa.cpa_latent_decode_workspace_size(B, 1, H), dtype=torch.uint8, device="cuda")
    start = i32(range(B + 1))
    steps = 4
    g = ref.gen(15)
    c, r = randn(steps, B, C, g=g), randn(steps, B, R, g=g)
    qc, qr = q_c.clone(), q_r.clone()
    outs = []
    graph = torch.cuda.CUDAGraph()
    before = pages.clone()
    with torch.cuda.graph(graph):
        for i in range(steps):
            dl.add_(1)
            cpa.cpa_latent_append(c[i], r[i], pages, table, start, dl, workspace=ws)
            o, lse = cpa.cpa_latent_decode(qc, qr, pages, table, dl, max_seq_len=1024, workspace=ws)
            outs.append((qc.clone(), qr.clone(), o, lse, dl.clone()))
            qc.copy_(o)                       # the next step's queries come from this one's output
            qr.copy_(o[..., :R])
    for _ in range(2):
        pages.copy_(before)
        dl.copy_(i32(lens))
        qc.copy_(q_c)
        qr.copy_(q_r)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, o, lse, n in outs:
            against(a, b, pages, table, n.tolist(), 1, o, lse, P)


def test_binding_refuses():
    q_c, q_r, pages, table, dl = make([20, 30], 2, 8, 16, 0)
    for bad in (dict(S=1), dict(S=3), dict(S=0)):
        with pytest.raises(ValueError, match="inconsistent"):
            cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, **bad)
    with pytest.raises(ValueError, match="shape"):
        cpa.cpa_latent_decode(q_c, q_r[:, :7], pages, table, dl, S=2)
    with pytest.raises(ValueError, match="contiguous"):
        cpa.cpa_latent_decode(q_c, q_r.transpose(1, 2).contiguous().transpose(1, 2), pages, table, dl, S=2)
    with pytest.raises(cpa.CpaError, match="INVALID_ARG"):
        cpa.cpa_latent_decode(q_c[:, :1].expand(-1, 8, -1), q_r, pages, table, dl, S=2)
    with pytest.raises(ValueError, match="576"):
        cpa.cpa_latent_decode(q_c, q_r, pages[..., :512].contiguous(), table, dl, S=2)
    with pytest.raises(ValueError, match="shape"):
        cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=2, o=q_c[:2].clone())
    with pytest.raises(cpa.CpaError, match="INVALID_ARG"):
        cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=2, sm_scale=0.0)
    with pytest.raises(cpa.CpaError, match="WORKSPACE"):
        cpa.cpa_latent_decode(q_c, q_r, pages, table, dl, S=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ----------------------------------------------------------------- expanded
def starts(n, lead=0):
    out = [lead]
    for m in n:
        out.append(out[-1] + m)
    return out


def make_prefill(news, lens, H, seed, lead=0, trail=0, k_lead=0, k_trail=0):
    g = ref.gen(seed)
    qs, ks = starts(news, lead), starts(lens, k_lead)
    kv = randn(ks[-1] + k_trail, H, 2 * D, g=g)
    q = randn(qs[-1] + trail, H, D + R, g=g)
    return q, kv[..., :D], randn(ks[-1] + k_trail, R, g=g), kv[..., D:], qs, ks


def against_prefill(q, nope, rope, v, qs, ks, o, lse, which=None, scale=lref.SCALE):
    for b in range(len(qs) - 1) if which is None else which:
        m, L = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        k = slice(ks[b], ks[b + 1])
        for i0 in range(0, m, 256):
            i1 = min(m, i0 + 256)
            r = slice(qs[b] + i0, qs[b] + i1)
            mask = ref.seen(range(L - m + i0, L - m + i1), L, 0, 0, "cuda")
            ref.close(o[r], lse[r], lref.expanded(q[r], nope[k], rope[k], v[k], mask, scale))


def check_prefill(news, lens, H, seed=0, lead=0, trail=0, k_lead=0, k_trail=0, **kw):
    q, nope, rope, v, qs, ks = make_prefill(news, lens, H, seed, lead, trail, k_lead, k_trail)
    for x in (nope, rope, v):  # what no request has
        x[:k_lead] = float("nan")
        x[ks[-1]:] = float("nan")
    o = torch.full((q.shape[0], H, D), 7.0, device="cuda").to(torch.bfloat16)
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), o=o, lse=lse, check=True, **kw)
    against_prefill(q, nope, rope, v, qs, ks, o, lse)
    for r in (slice(0, lead), slice(qs[-1], q.shape[0])):
        assert bool((o[r] == 7).all()) and bool((lse[r] == 7).all())


@pytest.mark.parametrize("H", [1, 2, 5, 8, 20, 128])
def test_ragged_chunks(H):
    check_prefill([1, 2, 0, 17, 64, 65, 128, 31, 129], [1, 300, 5, 17, 200, 129, 128, 1000, 129], H,
                  seed=H, lead=3, trail=5, k_lead=2, k_trail=7)


@pytest.mark.parametrize("news,lens", [
    ([1], [1]), ([1], [5000]), ([7], [9000]), ([3, 1, 2], [4000, 1, 2500]), ([1500], [1500]),
    ([1100], [2000]), ([513, 700], [513, 3333]), ([0, 0, 1], [10, 0, 1]), ([2000], [2000]),
    ([255, 256, 257], [255, 256, 257]), ([127, 128, 129], [255, 256, 257]), ([256] * 12, [256] * 12)])
def test_short_and_long(news, lens):
    check_prefill(news, lens, 8, seed=sum(news), k_trail=1)
    check_prefill(news, lens, 3, seed=sum(news) + 1)


def test_prefill_repeats_bit_for_bit():
    q, nope, rope, v, qs, ks = make_prefill([40, 3, 700], [1000, 3, 900], 16, 2)
    ws = torch.full((cpa.cpa_latent_prefill_workspace_size(3, q.shape[0], rope.shape[0], 16),), 0xA5,
                    dtype=torch.uint8, device="cuda")
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), workspace=ws, sm_scale=0.05)
    against_prefill(q, nope, rope, v, qs, ks, o, lse, scale=0.05)
    ws.fill_(0x5A)
    o2, lse2 = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), workspace=ws, sm_scale=0.05)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_keys_as_they_lie():
    """Slices of one product, arrays of their own, heads before tokens, a slice of the cache's
    rows for the shared part."""
    q, nope, rope, v, qs, ks = make_prefill([100, 300], [200, 300], 5, 4)
    want = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
    g = ref.gen(5)
    lat = randn(rope.shape[0], C + R, g=g)
    lat[:, C:] = rope
    odd = randn(rope.shape[0], 5, D + 8, g=g)
    odd[..., 8:] = v
    for k2, r2, v2 in ((nope.contiguous(), lat[:, C:], v.contiguous()),
                       (nope.transpose(0, 1).contiguous().transpose(0, 1), rope, odd[..., 8:])):
        got = cpa.cpa_latent_prefill(q, k2, r2, v2, i32(qs), i32(ks), check=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefill_scores_that_grow():
    q, nope, rope, v, qs, ks = make_prefill([300], [900], 4, 5)
    q.copy_(q[:1, :1].expand_as(q))
    pos = torch.arange(900, device="cuda")
    nope.copy_(((q[0, 0, :D] / 12)[None] * (pos / 20).to(torch.bfloat16)[:, None])[:, None].expand(-1, 4, -1))
    for _ in range(2):
        o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
        against_prefill(q, nope, rope, v, qs, ks, o, lse)
        nope.neg_()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prefill_values_that_are_not_numbers(value):
    """In v: the rows that see it have it in that column, and no others; in another request's keys
    or values, even in the same tile: no row."""
    q, nope, rope, v, qs, ks = make_prefill([200, 30], [400, 50], 4, 11)
    at = 350
    v[at, 2, 9] = value
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
    bad = ~torch.isfinite(o.float())
    pos = torch.arange(200, 400, device="cuda")
    hit = pos >= at
    assert bool(bad[:200][hit][:, 2, 9].all()) and bool(torch.isfinite(lse).all())
    assert int(bad.sum()) == int(hit.sum())
    v[at, 2, 9] = 0.0
    want = lref.expanded(q[:200][~hit], nope[:400], rope[:400], v[:400],
                         ref.seen(pos[~hit].tolist(), 400, 0, 0, "cuda"))
    ref.close(o[:200][~hit], lse[:200][~hit], want)
    # the second request's keys and values lie behind the first's
    nope[400:], v[400:], rope[400:] = value, value, value
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
    against_prefill(q, nope, rope, v, qs, ks, o, lse, which=[0])


def test_prefill_bad_starts_are_reported():
    q, nope, rope, v, qs, ks = make_prefill([40, 30], [60, 50], 2, 1)
    ws = torch.full((cpa.cpa_latent_prefill_workspace_size(2, 70, 110, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    for a, b in (([0, 40, 30], ks), ([0, 40, 71], ks), ([-1, 40, 70], ks), (qs, [0, 60, 50]), (qs, [0, 60, 111]),
                 (qs, [-1, 60, 110]), (qs, [0, 39, 110]), (qs, [0, 81, 110])):
        cpa.cpa_latent_prefill(q, nope, rope, v, i32(a), i32(b), workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == 8
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), workspace=ws)
    assert cpa.cpa_get_device_status(ws) == (0, 0)
    against_prefill(q, nope, rope, v, qs, ks, o, lse)
    none = torch.empty(0, 2, D + R, dtype=torch.bfloat16, device="cuda")
    ws.fill_(0xFF)
    got = cpa.cpa_latent_prefill(none, nope, rope, v, i32([0, 0, 0]), i32(ks), workspace=ws, check=True)
    assert got[0].shape == (0, 2, D)


def test_prefill_without_rows_looks_its_requests_over():
    _, nope, rope, v, _, ks = make_prefill([4, 3], [6, 5], 2, 1)
    none = torch.empty(0, 2, D + R, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(cpa.cpa_latent_prefill_workspace_size(2, 0, 11, 2), dtype=torch.uint8, device="cuda")
    for a, b, status in (([0, 0, 0], ks, 0), ([0, 0, 5], ks, 8), ([0, -1, 0], ks, 8), ([0, 5, 0], ks, 8),
                         ([0, 0, 0], [0, 6, 12], 8), ([0, 0, 0], [0, 6, 5], 8), ([0, 0, 0], [-1, 6, 11], 8)):
        ws.fill_(0xFF)
        cpa.cpa_latent_prefill(none, nope, rope, v, i32(a), i32(b), workspace=ws)
        assert cpa.cpa_get_device_status(ws)[0] == status, (a, b)
    many = i32([0] * 5001)
    ws.fill_(0xFF)
    cpa.cpa_latent_prefill(none, nope, rope, v, many, many, workspace=ws, check=True)
    many[4000] = 1
    cpa.cpa_latent_prefill(none, nope, rope, v, i32([0] * 5001), many, workspace=ws)
    assert cpa.cpa_get_device_status(ws)[0] == 8


@pytest.mark.parametrize("news,lens,H", [
    ([2500], [2500], 32), ([300, 0, 1, 700, 1500], [400, 7, 3000, 700, 1500], 32),
    ([900, 70], [1000, 4000], 96), ([40] * 130, [41] * 130, 16),
    ([37 * i % 61 for i in range(75)], [37 * i % 61 + 53 * i % 900 for i in range(75)], 40)])
def test_prefill_units_handed_out_whole(news, lens, H):
    """Enough rows that blocks take whole units, a few heads at a time."""
    assert sum(news) * H >= 2 * 152 * 256
    check_prefill(news, lens, H, seed=H, lead=1, trail=2, k_lead=3, k_trail=1)


def test_prefill_last_query_tiles_alone():
    """Whole units of one query tile with one key tile and with many, odd and even in number, one
    after another and between those of two: every request's result, the same in each run."""
    g = torch.Generator().manual_seed(7)
    news = [1, 128, 127, 300, 100, 129, 64, 5, 257, 380, 128, 40] * 2
    lens = [m + int(torch.randint(0, 1400, (1,), generator=g)) * (i % 4 != 0) for i, m in enumerate(news)]
    H = 32
    assert sum(news) * H >= 2 * 152 * 256
    q, nope, rope, v, qs, ks = make_prefill(news, lens, H, 5)
    args = (q, nope, rope, v, i32(qs), i32(ks))
    first = cpa.cpa_latent_prefill(*args, check=True)
    against_prefill(q, nope, rope, v, qs, ks, *first)
    for _ in range(20):
        o, lse = cpa.cpa_latent_prefill(*args)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    cpa.cpa_latent_prefill(*args, check=True)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prefill_values_that_are_not_numbers_in_whole_units(value):
    """Behind the first rows of a query tile that is its unit's only one, in an even and in an odd key
    tile: the rows that see it have it in that column, the others are as without it."""
    news, lens, H = [70, 2400], [700, 2400], 32
    assert sum(news) * H >= 2 * 152 * 256
    for at in (690, 635):  # key tiles 5 and 4; rows 630 and on
        q, nope, rope, v, qs, ks = make_prefill(news, lens, H, 11)
        want, want_lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
        v[at, 2, 9] = value
        o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
        bad = ~torch.isfinite(o.float())
        hit = torch.arange(630, 700, device="cuda") >= at
        assert bool(bad[:70][hit][:, 2, 9].all()) and int(bad.sum()) == int(hit.sum())
        v[at, 2, 9] = 0.0
        seen = ref.seen(torch.arange(630, 700)[~hit.cpu()].tolist(), 700, 0, 0, "cuda")
        ref.close(o[:70][~hit], lse[:70][~hit], lref.expanded(q[:70][~hit], nope[:700], rope[:700], v[:700], seen))
        assert torch.equal(o[70:], want[70:]) and torch.equal(lse[70:], want_lse[70:])


def test_prefill_units_handed_out_whole_in_a_graph():
    """Captured behind a copy, replayed: each replay hands out its units from the first."""
    news, lens, H = [1300, 1300], [1300, 1500], 32
    q, nope, rope, v, qs, ks = make_prefill(news, lens, H, 3)
    src, dq, dk = torch.empty_like(q), i32(qs), i32(ks)
    ws = torch.full((cpa.cpa_latent_prefill_workspace_size(2, q.shape[0], rope.shape[0], H),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.copy_(src)
        out = cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, workspace=ws)
        again = cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, workspace=ws)
    for seed in (1, 2):
        src.copy_(randn(*q.shape, g=ref.gen(seed)))
        ws.fill_(0x5A)
        graph.replay()
        against_prefill(src, nope, rope, v, qs, ks, *out)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("news,lens,H,trail", [
    ([20, 2420], [20000, 2420], 32, 0),           # one long context beside a prompt
    ([2430, 1, 17], [2430, 9000, 12000], 32, 3),
    ([2500], [7000], 32, 0), ([256] * 10, [2300] * 10, 32, 5),  # a last wave of like units
    ([40, 0, 33, 27], [300, 5, 900, 700], 32, 2400),          # few tokens in a large buffer
    ([1300, 1300], [1300, 1300], 32, 0), ([600] * 9, [900] * 9, 32, 0)])
def test_prefill_whole_units_and_ranges(news, lens, H, trail):
    """Calls of enough rows for whole units, some of which are shared out in ranges all the same."""
    assert (sum(news) + trail) * H >= 2 * 152 * 256
    check_prefill(news, lens, H, seed=len(news), trail=trail, k_trail=2)


def test_prefill_replays_that_change_how_units_are_shared_out():
    """One captured call, whose starts make it one of whole units, of ranges, of little work and of
    none."""
    H = 32
    q, nope, rope, v, qs, ks = make_prefill([1250, 1250], [6000, 6000], H, 17)
    dq, dk = i32(qs), i32(ks)
    o = torch.zeros((2500, H, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2500, H), device="cuda")
    ws = torch.full((cpa.cpa_latent_prefill_workspace_size(2, 2500, 12000, H),), 0xA5, dtype=torch.uint8, device="cuda")
    cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, o=o, lse=lse, workspace=ws, check=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, o=o, lse=lse, workspace=ws)
    for a, b in (([0, 1250, 2500], [0, 1300, 2600]), ([0, 2490, 2500], [0, 2490, 12000]), ([5, 45, 70], [0, 900, 1000]),
                 ([0, 0, 0], [0, 0, 9]), ([0, 2500, 2500], [0, 12000, 12000]), ([0, 1250, 2500], [0, 1300, 2600])):
        dq.copy_(i32(a))
        dk.copy_(i32(b))
        o.fill_(7)
        lse.fill_(7)
        graph.replay()
        assert cpa.cpa_get_device_status(ws) == (0, 0)
        against_prefill(q, nope, rope, v, a, b, o, lse)
        for r in (slice(0, a[0]), slice(a[-1], 2500)):
            assert bool((o[r] == 7).all()) and bool((lse[r] == 7).all())


def test_prefill_with_one_long_context_is_shared_out():
    """A few tokens behind a long context beside a prompt take no more than twice as long as the two
    one after the other (a unit of the long one on each of a few blocks: three times)."""
    news, lens, H = [32, 2400], [100000, 2400], 32
    q, nope, rope, v, qs, ks = make_prefill(news, lens, H, 19)
    both = (i32(qs), i32(ks))
    ws = torch.empty(cpa.cpa_latent_prefill_workspace_size(2, q.shape[0], rope.shape[0], H), dtype=torch.uint8, device="cuda")

    def together():
        cpa.cpa_latent_prefill(q, nope, rope, v, *both, workspace=ws)

    parts = [(slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1]), i32([0, news[b]]), i32([0, lens[b]])) for b in range(2)]

    def one_by_one():
        for a, b, x, y in parts:
            cpa.cpa_latent_prefill(q[a], nope[b], rope[b], v[b], x, y, workspace=ws)

    def us(f):
        best = 1e9
        for _ in range(8):
            t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            t0.record()
            f()
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1) * 1e3)
        return best

    a, b = us(together), us(one_by_one)
    assert a <= 2 * b, (a, b)


def test_prefill_many_requests():
    g = torch.Generator().manual_seed(3)
    news = torch.randint(0, 5, (900,), generator=g).tolist()
    lens = [m + int(torch.randint(0, 9, (1,), generator=g)) for m in news]
    check_prefill(news, lens, 1, seed=2)


@pytest.mark.parametrize("H,m", [(1, 300), (32, 2500)])
def test_prefill_among_empty_requests(H, m):
    """Thousands of requests without new tokens before, between and behind a few that have some."""
    news = [0] * 5000 + [m] + [0] * 3000 + [1] + [0] * 2000
    lens = [1] * 5000 + [m + 50] + [0] * 3000 + [70] + [2] * 2000
    q, nope, rope, v, qs, ks = make_prefill(news, lens, H, 5)
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, i32(qs), i32(ks), check=True)
    against_prefill(q, nope, rope, v, qs, ks, o, lse, which=[5000, 8001])


def test_prefill_walks_over_millions_of_empty_requests():
    """What one warp takes seconds to pass over puts off the limit of the other warps' waits."""
    H, m, n = 16, 5000, 1 << 24
    q, nope, rope, v, qs, ks = make_prefill([m, 3], [m, 40], H, 3)
    a, b = (torch.full((n + 3,), m, dtype=torch.int32, device="cuda") for _ in "qk")
    a[0], a[-1], b[0], b[-1] = 0, m + 3, 0, m + 40
    ws = torch.empty(cpa.cpa_latent_prefill_workspace_size(n + 2, m + 3, m + 40, H), dtype=torch.uint8, device="cuda")
    o, lse = cpa.cpa_latent_prefill(q, nope, rope, v, a, b, workspace=ws, check=True)
    against_prefill(q, nope, rope, v, [0, m, m + 3], [0, m, m + 40], o, lse)


def test_prefill_offsets_past_32_bits():
    """Keys past 2^31 elements of the expanded array."""
    H, g = 64, ref.gen(2)
    T_k = 2 ** 31 // (H * 2 * D) + 1000
    kv = torch.zeros(T_k, H, 2 * D, dtype=torch.bfloat16, device="cuda")
    kv[-600:] = randn(600, H, 2 * D, g=g)
    rope, q = randn(T_k, R, g=g), randn(300, H, D + R, g=g)
    qs, ks = [0, 300], [T_k - 600, T_k]
    o, lse = cpa.cpa_latent_prefill(q, kv[..., :D], rope, kv[..., D:], i32(qs), i32(ks), check=True)
    against_prefill(q, kv[..., :D], rope, kv[..., D:], qs, ks, o, lse)


def test_prefill_streams_and_graphs():
    q, nope, rope, v, qs, ks = make_prefill([100, 60], [300, 500], 8, 9)
    dq, dk = i32(qs), i32(ks)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk, stream=side, check=True)
    side.synchronize()
    against_prefill(q, nope, rope, v, qs, ks, *got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cpa.cpa_latent_prefill(q, nope, rope, v, dq, dk)
    for mid, kmid in ((10, 200), (150, 700), (0, 400)):
        dq[1], dk[1] = mid, kmid
        q.copy_(randn(*q.shape, g=ref.gen(mid)))
        graph.replay()
        against_prefill(q, nope, rope, v, [0, mid, qs[-1]], [0, kmid, ks[-1]], *out)


def test_prefill_binding_refuses():
    q, nope, rope, v, qs, ks = make_prefill([4, 3], [6, 5], 2, 1)
    a, b = i32(qs), i32(ks)
    with pytest.raises(ValueError, match="inconsistent"):
        cpa.cpa_latent_prefill(q, nope, rope, v, a, b[:2])
    with pytest.raises(ValueError, match="inconsistent"):
        cpa.cpa_latent_prefill(q[..., :128].contiguous(), nope, rope, v, a, b)
    with pytest.raises(ValueError, match="shape"):
        cpa.cpa_latent_prefill(q, nope[:, :1], rope, v, a, b)
    with pytest.raises(ValueError, match="shape"):
        cpa.cpa_latent_prefill(q, nope, rope[:5], v, a, b)
    with pytest.raises(ValueError, match="contiguous"):
        cpa.cpa_latent_prefill(q, nope, rope, v.transpose(0, 2).contiguous().transpose(0, 2), a, b)
    with pytest.raises(cpa.CpaError, match="INVALID_ARG"):
        cpa.cpa_latent_prefill(q, nope[:, :1].expand(-1, 2, -1), rope, v, a, b)


# ----------------------------------------------------------------- together
def test_both_forms_agree_over_one_cache():
    """Prompts appended to the cache, read back and expanded for prefill; then a step of two drafts
    appended and decoded in the absorbed form, against the expanded form over everything."""
    H, P, prompts, S = 8, 16, [70, 200, 33], 2
    g = ref.gen(12)
    # (small integers over powers of two: both forms' products are near exact)
    w_k, w_v = (torch.randint(-2, 3, (H, D, C), generator=g, device="cuda").double() / 32 for _ in "kv")
    lens = [m + S for m in prompts]
    table, pool = ref.table_of(lens, P, g)
    pages = torch.full((pool, P, C + R), float("nan"), device="cuda").to(torch.bfloat16)
    c, r = randn(sum(lens), C, g=g), randn(sum(lens), R, g=g)
    full = starts(lens)
    part = [torch.cat([torch.arange(full[b], full[b] + m) for b, m in enumerate(prompts)]),
            torch.cat([torch.arange(full[b + 1] - S, full[b + 1]) for b in range(3)])]
    for rows, news, n in ((part[0], prompts, prompts), (part[1], [S] * 3, lens)):
        cpa.cpa_latent_append(c[rows], r[rows], pages, table, i32(starts(news)), i32(n), check=True)
    c_all, r_all = cpa.cpa_latent_gather(pages, table, i32(full), T=full[-1], check=True)
    assert torch.equal(c_all, c) and torch.equal(r_all, r)
    q = randn(3 * S, H, D + R, g=g)
    nope = torch.einsum("hdc,jc->jhd", w_k, c_all.double()).to(torch.bfloat16)
    v = torch.einsum("hdc,jc->jhd", w_v, c_all.double()).to(torch.bfloat16)
    o, lse = cpa.cpa_latent_prefill(q, nope, r_all, v, i32(starts([S] * 3)), i32(full), check=True)
    q_c = torch.einsum("thd,hdc->thc", q[..., :D].double(), w_k).to(torch.bfloat16)
    z, lse2 = cpa.cpa_latent_decode(q_c, q[..., D:], pages, table, i32(lens), S=S, check=True)
    o2 = torch.einsum("thc,hdc->thd", z.double(), w_v)
    # the forms differ by the rounding of the products between them: half a step of bf16 on
    # 512-term sums of the size of o, and on the scores (192 and 576 terms, |x| of a few units)
    x = torch.einsum("thd,jhd->thj", q[..., :D].double().abs(), nope.double().abs()).amax() * lref.SCALE
    y = torch.einsum("thc,jc->thj", q_c.double().abs(), c.double().abs()).amax() * lref.SCALE
    ds = 2.0 ** -8 * (x + y)
    assert float((lse - lse2).abs().max()) <= ds
    size = torch.einsum("thc,hdc->thd", z.double().abs(), w_v.abs()) + v.double().abs().amax()
    assert bool(((o.double() - o2).abs() <= (2 * ds + 4 * 2.0 ** -8) * size).all())


def test_fp8_cache_written_decoded_and_read_back():
    """Tokens appended in FP8, decoded there, and the same from the rows read back."""
    B, H_q, H_kv, P, L = 3, 8, 2, 16, 100
    g = ref.gen(13)
    table, pool = ref.table_of([L] * B, P, g)
    new = [randn(B * L, H_kv, D, g=g) for _ in "kv"]
    scale = [x.float().abs().amax(0) / 448 for x in new]
    pages = [torch.full((pool, P, H_kv, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
    lens, st = i32([L] * B), i32(starts([L] * B))
    cpa.cpa_cache_append_fp8(*new, *pages, *scale, table, st, lens, check=True)
    q = randn(B, H_q, D, g=g)
    o, lse = cpa.cpa_decode_fp8(q, *pages, *scale, table, lens, check=True)
    back = cpa.cpa_cache_gather_fp8(*pages, *scale, table, st, T=B * L, check=True)
    for b in range(B):
        K, V = (ref.dense(p, table[b], L, P, s) for p, s in zip(pages, scale))
        want = ref.attend(q[b:b + 1], K, V, ref.seen([L - 1], L, 0, 0, "cuda"), D ** -0.5, ref.E_F16, ref.E_Q_SPLIT)
        ref.close(o[b:b + 1], lse[b:b + 1], want)
        rows = slice(b * L, (b + 1) * L)
        assert torch.equal(back[0][rows].double(), K.to(torch.bfloat16).double())
