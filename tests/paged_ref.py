"""Plain 64-bit references and inputs for decode, windowed prefill and the page
operations: logical sequences, masks written out, no paging inside the
arithmetic.

The tolerance of an output follows from what is rounded on the way.  With u =
2^-8 (half a step of bf16) for the output, e_p for a weight before it meets V,
e_q for an element of q before it meets K (0 where q is used as it is), and a
dot product of 128 products summed in 32 bits:

    |ds|   <= (128 * 2^-23 + e_q) * scale * max_j sum_c |q_c k_jc|
    |do|   <= u |o| + (e_p + 2 |ds| + 2^-18) * sum_j w_j |v_j|
    |dlse| <= |ds| + 2^-20 * (1 + |lse|)

2^-23 and not 2^-24 a sum, because a tensor core may cut where a scalar sum
rounds; 2^-18 and 2^-20 cover 2^x and log2 of the hardware (2^-22 each), the
argument of 2^x (about 2^-24 times its size, under 64 here), and the sums in
32 bits of up to some thousand terms of one sign, added in many partial sums.
"""
from __future__ import annotations

import math

import torch

D = 128
U_BF16 = 2.0 ** -8
E_P_BF16 = 2.0 ** -8      # a weight rounded to bf16
E_P_SPLIT = 2.0 ** -15    # a weight held as two bf16 terms
E_F16 = 2.0 ** -11        # a weight rounded to f16
E_Q_SPLIT = 2.0 ** -20    # an element of q x k_scale held as two f16 terms


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def table_of(lens, P, g, spare=2, width=None):
    """Block table of pages scattered over a pool, -1 past each row's pages."""
    dev = g.device
    need = [-(-x // P) for x in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    t = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, pool


def pool_of(pool, P, H_kv, g):
    return torch.randn(pool, P, H_kv, D, generator=g, device=g.device).to(torch.bfloat16)


def dense(pages, row, L, P, scale=None):
    """[L, H_kv, D] in 64 bits: the logical sequence behind a table row."""
    pos = torch.arange(L, device=pages.device)
    x = pages[row.long()[pos // P], pos % P]
    x = x.view(torch.float8_e4m3fn).double() if pages.dtype == torch.uint8 else x.double()
    return x if scale is None else x * scale.double()


def seen(pos, L, window, sinks, device):
    """Boolean [len(pos), L]: which keys the queries at positions pos see."""
    p = torch.as_tensor(pos, device=device).view(-1, 1)
    j = torch.arange(L, device=device).view(1, -1)
    m = j <= p
    if window:
        m = m & ((p - j < window) | (j < sinks))
    return m


def attend(q, K, V, mask, scale, e_p=E_P_SPLIT, e_q=0.0):
    """q [n, H_q, D], K/V [L, H_kv, D] (64 bits): (o, lse, tolerance of o, of lse)."""
    n, H_q, _ = q.shape
    G = H_q // K.shape[1]
    q = q.double()
    K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
    x = torch.einsum("ihd,jhd->ihj", q, K) * scale
    x = x.masked_fill(~mask[:, None], -math.inf)
    big = torch.einsum("ihd,jhd->ihj", q.abs(), K.abs()).masked_fill(~mask[:, None], 0.0)
    ds = (big.amax(-1) if K.shape[0] else torch.zeros(n, H_q, device=q.device)) * scale
    ds = ds * (128 * 2.0 ** -23 + e_q)
    lse = torch.logsumexp(x, -1) if K.shape[0] else torch.full((n, H_q), -math.inf, device=q.device)
    w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = torch.einsum("ihj,jhd->ihd", w, V)
    tol_o = U_BF16 * o.abs() + (e_p + 2 * ds + 2.0 ** -18)[..., None] * \
        torch.einsum("ihj,jhd->ihd", w, V.abs())
    tol_l = ds + 2.0 ** -20 * (1 + torch.where(lse == -math.inf, 0.0, lse).abs())
    return o, lse, tol_o, tol_l


def close(got_o, got_lse, want):
    """got against attend()'s answer, element by element."""
    o, lse, tol_o, tol_l = want
    go, gl = got_o.double(), got_lse.double()
    assert bool(torch.isfinite(go).all()), "non-finite output"
    none = lse == -math.inf
    assert torch.equal(gl == -math.inf, none)
    assert bool((go[none] == 0).all())
    over = ((go - o).abs() - tol_o).max().item() if go.numel() else 0.0
    assert over <= 0, f"o off by {over:.3e} more than its tolerance"
    over = ((gl - lse).abs() - tol_l)[~none]
    assert over.numel() == 0 or over.max().item() <= 0, f"lse off by {over.max().item():.3e} more"


def hide_unseen(k, v, table, lens, masks, P, poison=float("nan")):
    """Fill every slot that no query sees with NaN, and take pages that hold none out of the
    table (-1).  masks[b]: boolean [L] of the keys that some query of request b sees."""
    for x in (k, v):
        keep = torch.zeros(x.shape[0] * P, dtype=torch.bool, device=x.device)
        for b, L in enumerate(lens):
            pos = torch.nonzero(masks[b]).view(-1)
            keep[table[b].long()[pos // P] * P + pos % P] = True
        flat = x.view(-1, *x.shape[2:])
        if x.dtype == torch.uint8:
            flat[~keep] = 0x7F
        else:
            flat[~keep] = poison
    for b, L in enumerate(lens):
        pages = torch.zeros(table.shape[1], dtype=torch.bool, device=table.device)
        pages[torch.nonzero(masks[b]).view(-1) // P] = True
        table[b][~pages] = -1
