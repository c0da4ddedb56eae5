"""Plain 64-bit references for latent attention, absorbed and expanded.

Tolerances follow from what is rounded on the way, as in paged_ref: a dot product of n
products is off by n * 2^-23 of the sum of its terms' sizes, a weight by half a step of
bf16 (2^-8) before it meets V, the output by half a step.
"""
from __future__ import annotations

import math

import torch

from tests import paged_ref as ref

C, R, D = 512, 64, 128
SCALE = (D + R) ** -0.5


def attend(x, big, V, mask, terms):
    """x, big [n, H, L]: scaled scores and the sums of their terms' sizes; V [L, H or 1, width]:
    (o, lse, tolerance of o, of lse)."""
    n, H, L = x.shape
    x = x.masked_fill(~mask[:, None], -math.inf)
    big = big.masked_fill(~mask[:, None], 0.0)
    ds = (big.amax(-1) if L else torch.zeros(n, H, device=x.device)) * terms * 2.0 ** -23
    lse = torch.logsumexp(x, -1) if L else torch.full((n, H), -math.inf, device=x.device,
                                                      dtype=torch.float64)
    w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    V = V.expand(-1, H, -1)
    o = torch.einsum("ihj,jhd->ihd", w, V)
    tol_o = ref.U_BF16 * o.abs() + (ref.E_P_BF16 + 2 * ds + 2.0 ** -18)[..., None] * \
        torch.einsum("ihj,jhd->ihd", w, V.abs())
    tol_l = ds + 2.0 ** -20 * (1 + torch.where(lse == -math.inf, 0.0, lse).abs())
    return o, lse, tol_o, tol_l


def absorbed(q_c, q_r, lat, mask, scale=SCALE):
    """q_c [n, H, C], q_r [n, H, R], lat [L, C + R]."""
    q, lat = torch.cat([q_c, q_r], 2).double(), lat.double()
    x = torch.einsum("ihd,jd->ihj", q, lat) * scale
    big = torch.einsum("ihd,jd->ihj", q.abs(), lat.abs()) * scale
    return attend(x, big, lat[:, None, :C], mask, C + R)


def expanded(q, nope, rope, v, mask, scale=SCALE):
    """q [n, H, D + R], nope and v [L, H, D], rope [L, R]."""
    q, k = q.double(), torch.cat([nope, rope[:, None].expand(-1, nope.shape[1], -1)], 2).double()
    x = torch.einsum("ihd,jhd->ihj", q, k) * scale
    big = torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()) * scale
    return attend(x, big, v.double(), mask, D + R)
