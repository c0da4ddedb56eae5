"""Measured cases of writing a paged cache and reading it back (in bf16, and
quantised to FP8 on the way), and of latent attention: keys and values of every
head from one latent vector a token, absorbed (decode over the paged latents) and
expanded (causal prefill of ragged chunks).

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library's entry points.
"""
import math

import torch

own = False

D = 128            # head_dim of the K/V pools, and of an expanded head's part without position
C, R = 512, 64     # a latent: its compressed part, and the part that carries the position
SCALE = (D + R) ** -0.5
E4M3_MAX = 448.0
DEV = "cuda"


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # the new token of each request of a batch, into FP8 pages: once a layer and step, so
        # latency is all of it
        dict(name="append_step", op="append", kind="fp8", B=64, new_lo=1, new_hi=1, len_lo=1500,
             len_hi=2500, P=16, H_kv=8, per_channel=True),
        # whole prompts into FP8 pages, K and V as they lie in the fused projection's rows
        dict(name="append_prompts", op="append", kind="fp8", B=16, new_lo=1024, new_hi=4096,
             len_lo=4096, len_hi=9001, P=16, H_kv=8, per_channel=True),
        # chunks of prompts into the latent cache (the compressed part from its norm, the other
        # from its rotation)
        dict(name="append_latents", op="append", kind="latent", B=12, new_lo=777, new_hi=8192,
             len_lo=8192, len_hi=16001, P=64, H_kv=1, per_channel=False),
        # an FP8 cache read back as bf16 rows (for a layer or a device that takes no FP8)
        dict(name="gather_fp8", op="gather", kind="fp8", B=16, n_lo=1000, n_hi=8192, first_hi=0,
             P=16, H_kv=8, per_channel=True),
        # the latents of the contexts of a prefill step, about to be expanded
        dict(name="gather_latents", op="gather", kind="latent", B=6, n_lo=1000, n_hi=9001,
             first_hi=0, P=16, H_kv=1, per_channel=False),
        # one request in a chat window: the smallest decode, latency is all of it
        dict(name="latent_decode_single", op="decode", B=1, S=1, H=16, P=16, len_lo=777,
             len_hi=777),
        # a batch of the benchmark's lengths, the heads of one of eight devices
        dict(name="latent_decode_batch", op="decode", B=64, S=1, H=16, P=16, len_lo=2000,
             len_hi=2000),
        # every head on one device, long and unequal contexts
        dict(name="latent_decode_heads", op="decode", B=32, S=1, H=128, P=64, len_lo=1024,
             len_hi=16384),
        # a verify step of four drafts and the token before them, causal among themselves
        dict(name="latent_decode_drafts", op="decode", B=20, S=5, H=32, P=16, len_lo=500,
             len_hi=6000),
        # the end of a prompt, a tool's short answer
        dict(name="latent_prefill_few", op="prefill", B=3, H=32, new_lo=5, new_hi=37, len_lo=100,
             len_hi=701),
        # chunked prefill: some hundred tokens of each request behind a long context
        dict(name="latent_prefill_chunk", op="prefill", B=6, H=32, new_lo=200, new_hi=640,
             len_lo=1000, len_hi=9001),
        # whole prompts of the benchmark's prefill length
        dict(name="latent_prefill_long", op="prefill", B=2, H=32, new_lo=8192, new_hi=8192,
             len_lo=8192, len_hi=8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill", "prefill"])
    P = rng.choice([8, 16, 32, 64, 128, 256])
    if op in ("append", "gather"):
        kind = rng.choice(["bf16", "fp8", "fp8", "latent"])
        H_kv = 1 if kind == "latent" else rng.choice([1, 2, 4, 5, 8])
        hi = _log_int(rng, 1, 9000)
        B = _log_int(rng, 1, max(1, min(256, 40000 // hi)))
        c = dict(op=op, kind=kind, B=B, P=P, H_kv=H_kv,
                 per_channel=kind == "fp8" and rng.random() < 0.7)
        lo = max(1, hi // rng.choice([1, 2, 30]))
        if op == "append":
            return dict(c, new_lo=lo, new_hi=hi, len_lo=hi, len_hi=hi + rng.choice([0, 7, 1000]))
        return dict(c, n_lo=lo, n_hi=hi, first_hi=rng.choice([0, 1, 500]))
    if op == "decode":
        H, S = rng.choice([1, 2, 5, 8, 16, 20, 32, 40, 64, 80, 128]), rng.choice([1, 1, 1, 2, 3, 6])
        hi = _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, max(1, min(256, 400000 // hi, 60000000 // (hi * H * S))))
        return dict(op=op, B=B, S=S, H=H, P=P, len_lo=max(1, hi // rng.choice([1, 2, 30])),
                    len_hi=hi)
    H = rng.choice([1, 2, 5, 8, 20, 32])
    hi = _log_int(rng, 16, 8192)
    new = _log_int(rng, 1, hi)
    B = _log_int(rng, 1, max(1, min(32, 16384 * 100000 // (hi * new * H))))
    return dict(op=op, B=B, H=H, new_lo=max(1, new // 2), new_hi=new, len_lo=new, len_hi=hi)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], spread evenly in a scattered order (the case's own, not
    the seed's, so that the work of a case is known); the first is hi."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lens(c):
    """(tokens of each request, new ones among them)."""
    if c["op"] == "gather":
        n = _spread(c["n_lo"], c["n_hi"], c["B"])
        return [x + f for x, f in zip(n, _firsts(c))], n
    lens = _spread(c["len_lo"], c["len_hi"], c["B"])
    if c["op"] == "decode":
        return lens, [c["S"]] * c["B"]
    return lens, [min(m, x) for m, x in zip(_spread(c["new_lo"], c["new_hi"], c["B"]), lens)]


def _firsts(c):
    return _spread(0, c["first_hi"], c["B"])


def work(case):
    c = case
    lens, news = _lens(c)
    if c["op"] in ("append", "gather"):
        # a token's bytes in bf16, and in its page
        wide = (C + R) * 2 if c["kind"] == "latent" else 2 * c["H_kv"] * D * 2
        page = wide // 2 if c["kind"] == "fp8" else wide
        return dict(bytes=sum(news) * (wide + page), flops=0)
    # pairs of a query token and a key that it sees
    pairs = sum(max(0, p + 1) for x, m in zip(lens, news) for p in range(x - m, x))
    rows = sum(news) * c["H"]
    if c["op"] == "decode":
        return dict(bytes=sum(lens) * (C + R) * 2 + rows * ((C + R) * 2 + C * 2 + 4),
                    flops=2 * (2 * C + R) * c["H"] * pairs)
    return dict(bytes=sum(lens) * (c["H"] * 2 * D + R) * 2 + rows * ((D + R) * 2 + D * 2 + 4),
                flops=2 * (2 * D + R) * c["H"] * pairs)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return _i32(out)


def _tables(lens, P, g, spare=3):
    """A block table of pages scattered over a pool: (table, pages in the pool)."""
    need = [-(-x // P) for x in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    c = case
    g = _gen(seed)
    s = dict(case=c, scratch=torch.empty(64 << 20, dtype=torch.uint8, device=DEV))
    lens, news = _lens(c)
    n = sum(news)
    s["lens"], s["start"], s["rows"] = _i32(lens), _starts(news), n
    if c["op"] == "prefill":
        s["q"] = _normal((n, c["H"], D + R), g)
        s["k_start"] = _starts(lens)
        kv = _normal((sum(lens), c["H"], 2 * D), g)  # as one product expands them
        s["k_nope"], s["v"] = kv[..., :D], kv[..., D:]
        s["k_rope"] = _normal((sum(lens), R), g)
        s["o"] = torch.empty((n, c["H"], D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(n, c["H"], device=DEV)
        return s
    s["table"], pool = _tables(lens, c["P"], g)
    if c["op"] == "decode":
        s["pages"] = _normal((pool, c["P"], C + R), g)
        s["max_len"] = c["len_hi"]
        s["q_c"] = _normal((n, c["H"], C), g)
        s["q_r"] = _normal((n, c["H"], R), g)
        s["o"] = torch.empty((n, c["H"], C), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(n, c["H"], device=DEV)
        return s
    if c["op"] == "gather":
        s["first"] = _i32(_firsts(c))
    if c["kind"] == "latent":
        s["pages"] = _normal((pool, c["P"], C + R), g)
        if c["op"] == "append":
            s["c_new"] = _normal((n, C), g)
            s["r_new"] = _normal((n, R), g)
        else:
            s["c_out"] = torch.empty((n, C), dtype=torch.bfloat16, device=DEV)
            s["r_out"] = torch.empty((n, R), dtype=torch.bfloat16, device=DEV)
        return s
    H = c["H_kv"]
    shape = (pool, c["P"], H, D)
    if c["op"] == "append":
        # K and V lie behind Q in the projection's rows
        s["qkv"] = _normal((n, 6 * H, D), g)
        s["k_new"], s["v_new"] = s["qkv"][:, 4 * H:5 * H], s["qkv"][:, 5 * H:]
    for name in ("k", "v"):
        if c["kind"] == "bf16":
            s[name] = _normal(shape, g)
            continue
        # channels of unequal size, with scales that a few values in a million leave
        size = torch.exp(0.5 * torch.randn(H, D, generator=g, device=DEV))
        if c["op"] == "append":
            s[name + "_new"].mul_(size.to(torch.bfloat16))
        s[name + "_scale"] = size * (4.5 / E4M3_MAX)
        if not c["per_channel"]:
            s[name + "_scale"] = s[name + "_scale"].amax().view(1)
        s[name] = (_normal(shape, g).float() * 96).to(torch.float8_e4m3fn).view(torch.uint8)
    if c["op"] == "gather":
        s["k_out"] = torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _pools(s):
    """The pools, FP8 ones as the values that their codes stand for."""
    if s["case"]["kind"] == "latent":
        return [s["pages"]]
    fp8 = s["case"]["kind"] == "fp8"
    return [s[n].view(torch.float8_e4m3fn) if fp8 else s[n] for n in ("k", "v")]


def _own(s):
    import cascade_paged_attention_gb300 as cpa
    c, ws = s["case"], s["scratch"]
    if c["op"] == "append":
        if c["kind"] == "latent":
            cpa.cpa_latent_append(s["c_new"], s["r_new"], s["pages"], s["table"], s["start"],
                                  s["lens"], workspace=ws)
        elif c["kind"] == "fp8":
            cpa.cpa_cache_append_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"],
                                     s["v_scale"], s["table"], s["start"], s["lens"], workspace=ws)
        else:
            cpa.cpa_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["start"],
                                 s["lens"], workspace=ws)
        return _pools(s)
    if c["op"] == "gather":
        if c["kind"] == "latent":
            return cpa.cpa_latent_gather(s["pages"], s["table"], s["start"], first=s["first"],
                                         c_out=s["c_out"], r_out=s["r_out"], workspace=ws)
        kw = dict(first=s["first"], k_out=s["k_out"], v_out=s["v_out"], workspace=ws)
        if c["kind"] == "fp8":
            return cpa.cpa_cache_gather_fp8(s["k"], s["v"], s["k_scale"], s["v_scale"],
                                            s["table"], s["start"], **kw)
        return cpa.cpa_cache_gather(s["k"], s["v"], s["table"], s["start"], **kw)
    if c["op"] == "decode":
        return cpa.cpa_latent_decode(s["q_c"], s["q_r"], s["pages"], s["table"], s["lens"],
                                     S=c["S"], max_seq_len=s["max_len"], o=s["o"], lse=s["lse"],
                                     workspace=ws)
    return cpa.cpa_latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["start"],
                                  s["k_start"], o=s["o"], lse=s["lse"], workspace=ws)


def _plain(s):
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode,
            "prefill": _plain_prefill}[s["case"]["op"]](s)


def _slots(s, first):
    """The slot of the pool of each token of the ragged rows, whose requests begin at
    positions `first`."""
    P = s["case"]["P"]
    start = s["start"].long()
    t = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1    # the request of each token
    pos = first.long()[b] + t - start[b]
    return s["table"][b, pos // P].long() * P + pos % P


def _plain_append(s):
    c = s["case"]
    start = s["start"]
    at = _slots(s, s["lens"] - (start[1:] - start[:-1]))
    if c["kind"] == "latent":
        s["pages"].view(-1, C + R)[at] = torch.cat([s["c_new"], s["r_new"]], 1)
        return _pools(s)
    for name in ("k", "v"):
        x = s[name + "_new"]
        if c["kind"] == "fp8":
            x = (x.float() / s[name + "_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
            x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name].view(-1, c["H_kv"], D)[at] = x
    return _pools(s)


def _plain_gather(s):
    c = s["case"]
    at = _slots(s, s["first"])
    if c["kind"] == "latent":
        x = s["pages"].view(-1, C + R)[at]
        s["c_out"].copy_(x[:, :C])
        s["r_out"].copy_(x[:, C:])
        return s["c_out"], s["r_out"]
    for name in ("k", "v"):
        x = s[name].view(-1, c["H_kv"], D)[at]
        if c["kind"] == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"]
        s[name + "_out"].copy_(x)
    return s["k_out"], s["v_out"]


def _softmax(x, seen):
    """Weights and log-sum-exp over the last axis where seen."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    t = e.sum(-1, keepdim=True)
    return e / torch.where(t == 0, torch.ones_like(t), t), (m + torch.log(t)).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, S, H, P = c["B"], c["S"], c["H"], c["P"]
    L = s["lens"].long()
    j = torch.arange(s["max_len"], device=DEV)[None]
    at = torch.minimum(j, L[:, None] - 1)
    k = s["pages"][torch.gather(s["table"].long(), 1, at // P), at % P].float()   # [B, L, C + R]
    q = torch.cat([s["q_c"], s["q_r"]], 2).float().view(B, S * H, C + R)
    x = (q @ k.transpose(1, 2)).view(B, S, H, -1) * SCALE
    last = L[:, None] - S + torch.arange(S, device=DEV)[None]       # the position of each token
    w, lse = _softmax(x, (j[:, None] <= last[..., None])[:, :, None])
    o = w.view(B, S * H, -1) @ k[..., :C]
    return o.view(B * S, H, C).to(torch.bfloat16), lse.view(B * S, H)


def _plain_prefill(s):
    c = s["case"]
    B, H, M = c["B"], c["H"], c["new_hi"]
    start, k_start, L = s["start"].long(), s["k_start"].long(), s["lens"].long()
    t = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1    # the request of each token
    i = t - start[b]
    q = torch.zeros(B, M, H, D + R, device=DEV)
    q[b, i] = s["q"].float()
    j = torch.arange(c["len_hi"], device=DEV)[None]
    at = k_start[:-1, None] + torch.minimum(j, L[:, None] - 1)
    k = torch.cat([s["k_nope"][at].float(), s["k_rope"][at].float()[:, :, None].expand(-1, -1, H, -1)], 3)
    x = (q.transpose(1, 2) @ k.permute(0, 2, 3, 1)) * SCALE         # [B, H, M, L]
    p = (L - (start[1:] - start[:-1]))[:, None] + torch.arange(M, device=DEV)[None]
    w, lse = _softmax(x, (j[:, None] <= p[..., None])[:, None])
    o = (w @ s["v"][at].float().transpose(1, 2)).transpose(1, 2)
    return o[b, i].to(torch.bfloat16), lse.transpose(1, 2)[b, i]


# ----------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    """Request by request.  Quantised values are what they would be before rounding; operators
    that move values compute none."""
    c = case
    if c["op"] in ("append", "gather") and c["kind"] != "fp8" or work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    lens, news = _lens(c)
    starts = s["start"].tolist()
    if c["op"] in ("append", "gather"):
        P, out = c["P"], []
        for name in ("k", "v"):
            codes = s[name].view(torch.float8_e4m3fn).double()
            scale = s[name + "_scale"].double()
            new = torch.empty((starts[-1], c["H_kv"], D), dtype=torch.float64, device=DEV)
            for b, (L, m) in enumerate(zip(lens, news)):
                pos = torch.arange(L - m, L, device=DEV)
                if c["op"] == "gather":
                    new[starts[b]:starts[b + 1]] = codes[s["table"][b][pos // P].long(), pos % P] * scale
                else:
                    x = s[name + "_new"][starts[b]:starts[b + 1]].double() / scale
                    codes[s["table"][b][pos // P].long(), pos % P] = x.clamp(-E4M3_MAX, E4M3_MAX)
            out.append(new if c["op"] == "gather" else codes)
        return out
    width = C if c["op"] == "decode" else D
    o = torch.empty((starts[-1] if c["op"] == "prefill" else c["B"] * c["S"], c["H"], width),
                    dtype=torch.float64, device=DEV)
    lse = torch.empty(o.shape[:2], dtype=torch.float64, device=DEV)
    k0 = 0
    for b, (L, m) in enumerate(zip(lens, news)):
        if c["op"] == "decode":
            n_pages = -(-L // c["P"])
            lat = s["pages"][s["table"][b, :n_pages].long()].double().reshape(-1, C + R)[:L]
        else:
            rope = s["k_rope"][k0:k0 + L].double()
            nope, val = (s[n][k0:k0 + L].double() for n in ("k_nope", "v"))
            k0 += L
        for i0 in range(0, m, 256):
            i1 = min(m, i0 + 256)
            rows = slice(starts[b] + i0, starts[b] + i1)
            p = torch.arange(L - m + i0, L - m + i1, device=DEV)
            top = max(0, L - m + i1)
            if c["op"] == "decode":
                x = torch.einsum("ihd,jd->hij", s["q_c"][rows].double(), lat[:top, :C])
                x += torch.einsum("ihd,jd->hij", s["q_r"][rows].double(), lat[:top, C:])
            else:
                q = s["q"][rows].double()
                x = torch.einsum("ihd,jhd->hij", q[..., :D], nope[:top])
                x += torch.einsum("ihd,jd->hij", q[..., D:], rope[:top])
            x /= math.sqrt(D + R)
            x.masked_fill_(torch.arange(top, device=DEV)[None] > p[:, None], -math.inf)
            z = torch.logsumexp(x, -1) if top else torch.full(x.shape[:2], -math.inf, device=DEV)
            lse[rows] = z.T
            x = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
            if c["op"] == "decode":
                o[rows] = torch.einsum("hij,jd->ihd", x, lat[:top, :C])
            else:
                o[rows] = torch.einsum("hij,jhd->ihd", x, val[:top])
    return o, lse
