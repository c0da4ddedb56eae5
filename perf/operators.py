"""Measured cases of the paged-cache operators: decode over a paged KV cache,
prefill of prompt chunks with a sliding window and sinks, and the page
operations of the cache that both read.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library's entry points.
"""
import math

import torch

own = False

D = 128          # head_dim of every call of the library
DEV = "cuda"


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one request in a chat window: the smallest call, latency is all of it
        dict(name="decode_single", op="decode", B=1, H_q=32, H_kv=8, P=16, len_lo=777, len_hi=777,
             window=0, sinks=0, fp8=False),
        # plain decode of the benchmark's batch (64 requests of 2000 tokens)
        dict(name="decode_batch", op="decode", B=64, H_q=32, H_kv=8, P=16, len_lo=2000,
             len_hi=2000, window=0, sinks=0, fp8=False),
        # long and very unequal contexts, wide groups (8 query heads a KV head)
        dict(name="decode_long_ragged", op="decode", B=16, H_q=64, H_kv=8, P=64, len_lo=1024,
             len_hi=32768, window=0, sinks=0, fp8=False),
        # a windowed layer of a long-context model: 4 sinks and the last 4096 tokens
        dict(name="decode_window", op="decode", B=48, H_q=32, H_kv=8, P=16, len_lo=500,
             len_hi=20000, window=4096, sinks=4, fp8=False),
        # the same cache held in FP8 with a scale for each KV head and channel
        dict(name="decode_fp8", op="decode", B=64, H_q=32, H_kv=8, P=16, len_lo=512, len_hi=8192,
             window=0, sinks=0, fp8=True),
        # a few tokens of a few requests (the end of a prompt, a tool's short answer)
        dict(name="prefill_few", op="prefill", B=3, H_q=32, H_kv=8, P=16, new_lo=5, new_hi=37,
             len_lo=100, len_hi=701, window=256, sinks=4),
        # chunked prefill: some hundred tokens of each request behind a long context
        dict(name="prefill_chunk", op="prefill", B=6, H_q=32, H_kv=8, P=16, new_lo=200,
             new_hi=640, len_lo=1000, len_hi=9001, window=4096, sinks=4),
        # whole prompts of the benchmark's prefill length through a windowed layer
        dict(name="prefill_long", op="prefill", B=2, H_q=32, H_kv=8, P=16, new_lo=8192,
             new_hi=8192, len_lo=8192, len_hi=8192, window=2048, sinks=16),
        # one conversation forked into four branches
        dict(name="fork_branches", op="fork", parents=1, fan=4, len_lo=777, len_hi=777, P=16,
             H_kv=8),
        # a batch forked: 64 requests of about 2000 tokens into four branches each
        dict(name="fork_batch", op="fork", parents=64, fan=4, len_lo=1801, len_hi=2199, P=16,
             H_kv=8),
        # accepted drafts of a verify step move behind the prefix (up to 6 of a tree's nodes)
        dict(name="compact_drafts", op="compact", B=64, keep_lo=1, keep_hi=6, span=20, P=16,
             H_kv=8, dst_lo=1500, dst_hi=2500),
        # a long history pruned: half of the tokens of 8 requests kept, on fresh pages
        dict(name="compact_history", op="compact", B=8, keep_lo=4000, keep_hi=8192, span=16384,
             P=64, H_kv=8, dst_lo=0, dst_hi=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "fork", "compact"])
    H_kv = rng.choice([1, 2, 4, 8])
    P = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "decode":
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        hi = _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, max(1, min(256, 270000 // hi)))
        return dict(op=op, B=B, H_q=H_kv * G, H_kv=H_kv, P=P, len_lo=max(1, hi // rng.choice([1, 2, 30])),
                    len_hi=hi, window=rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                    sinks=rng.choice([0, 1, 4, 130]), fp8=rng.random() < 0.3)
    if op == "prefill":
        G = rng.choice([1, 2, 4, 5, 8])
        hi = _log_int(rng, 16, 8192)
        new = _log_int(rng, 1, hi)
        B = _log_int(rng, 1, max(1, min(32, 16384 * 16384 // (hi * new * H_kv * G))))
        return dict(op=op, B=B, H_q=H_kv * G, H_kv=H_kv, P=P, new_lo=max(1, new // 2), new_hi=new,
                    len_lo=new, len_hi=hi, window=rng.choice([0, _log_int(rng, 16, 4096)]),
                    sinks=rng.choice([0, 4, 100]))
    if op == "fork":
        hi = _log_int(rng, 9, 8000)
        return dict(op=op, parents=_log_int(rng, 1, 64), fan=rng.randint(1, 8),
                    len_lo=max(1, hi // 2), len_hi=hi, P=P, H_kv=H_kv)
    span = _log_int(rng, 2, 16000)
    keep = _log_int(rng, 1, span // 2)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(64, 60000 // keep))), keep_lo=max(1, keep // 3),
                keep_hi=keep, span=span, P=P, H_kv=H_kv, dst_lo=0, dst_hi=rng.choice([0, 1000]))


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], spread evenly in a scattered order (the case's own, not
    the seed's, so that the work of a case is known); the first is hi."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _visible(pos, window, sinks):
    """How many keys a query at position pos sees."""
    if window == 0 or pos + 1 <= window:
        return pos + 1
    return min(sinks, pos + 1 - window) + window


def work(case):
    c = case
    if c["op"] == "decode":
        lens = _spread(c["len_lo"], c["len_hi"], c["B"])
        n = sum(_visible(x - 1, c["window"], c["sinks"]) for x in lens)
        kv = 2 * c["H_kv"] * D * (1 if c["fp8"] else 2)
        return dict(bytes=n * kv + c["B"] * c["H_q"] * (4 * D + 4), flops=4 * D * c["H_q"] * n)
    if c["op"] == "prefill":
        lens = _spread(c["len_lo"], c["len_hi"], c["B"])
        news = _spread(c["new_lo"], c["new_hi"], c["B"])
        pairs = keys = 0
        for x, m in zip(lens, news):
            m = min(m, x)
            pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(x - m, x))
            first = max(0, x - m + 1 - c["window"]) if c["window"] else 0
            keys += x - first + min(c["sinks"], first)
        rows = sum(min(m, x) for x, m in zip(lens, news)) * c["H_q"]
        return dict(bytes=keys * 4 * c["H_kv"] * D + rows * (4 * D + 4),
                    flops=4 * D * c["H_q"] * pairs)
    if c["op"] == "fork":
        lens = [x | 1 for x in _spread(c["len_lo"], c["len_hi"], c["parents"])]
        page = 2 * c["P"] * c["H_kv"] * D * 2
        entries = sum(-(-x // c["P"]) for x in lens) * c["fan"]
        n = c["parents"] * c["fan"]
        # the copied pages, the children's table rows and the counts of their pages
        return dict(bytes=2 * n * page + 8 * entries + 8 * entries, flops=0)
    keep = sum(_spread(c["keep_lo"], c["keep_hi"], c["B"]))
    return dict(bytes=2 * keep * 2 * c["H_kv"] * D * 2, flops=0)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


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
    if c["op"] in ("decode", "prefill"):
        lens = _spread(c["len_lo"], c["len_hi"], c["B"])
        s["table"], pool = _tables(lens, c["P"], g)
        s["lens"] = _i32(lens)
        s["max_len"] = c["len_hi"]
        shape = (pool, c["P"], c["H_kv"], D)
        if c.get("fp8"):
            for k in ("k", "v"):
                s[k] = torch.randn(shape, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
                s[k + "_scale"] = torch.rand(c["H_kv"], D, generator=g, device=DEV) * 0.5 + 0.5
        else:
            s["k"], s["v"] = _normal(shape, g), _normal(shape, g)
        if c["op"] == "decode":
            rows = c["B"]
        else:
            news = [min(m, x) for m, x in zip(_spread(c["new_lo"], c["new_hi"], c["B"]), lens)]
            start = [0]
            for m in news:
                start.append(start[-1] + m)
            s["q_start"] = _i32(start)
            rows = start[-1]
        s["q"] = _normal((rows, c["H_q"], D), g)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["H_q"], device=DEV)
    elif c["op"] == "fork":
        # parents in the first rows of the table; every child row still holds the branch of the
        # step before (a fork of the same parents), which the pass gives back first
        P, n = c["P"], c["parents"] * c["fan"]
        lens = [x | 1 for x in _spread(c["len_lo"], c["len_hi"], c["parents"])]  # inside a page
        table, pool = _tables(lens, P, g, spare=3 * n + 8)
        refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        s["parents"] = _i32([i % c["parents"] for i in range(n)])
        s["children"] = _i32([c["parents"] + i for i in range(n)])
        par = s["parents"].long()
        last = (torch.tensor(lens, device=DEV) - 1) // P
        free = torch.nonzero(refs == 0).view(-1)
        old = free[torch.randperm(free.numel(), generator=g, device=DEV)[:n]].to(torch.int32)
        rows = table[par].clone()
        whole = torch.arange(table.shape[1], device=DEV)[None] < last[par][:, None]
        refs.index_add_(0, rows[whole].long(), torch.ones_like(rows[whole]))
        rows[torch.arange(n, device=DEV), last[par]] = old
        refs[old.long()] = 1
        s["table"] = torch.cat([table, rows])
        s["lens"] = torch.cat([_i32(lens), _i32(lens)[par]])
        s["refs"] = refs
        s["first"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        s["last"] = torch.full((n,), table.shape[1], dtype=torch.int32, device=DEV)
        s["src"], s["dst"] = torch.empty_like(s["parents"]), torch.empty_like(s["parents"])
        s["k"] = _normal((pool, P, c["H_kv"], D), g)
        s["v"] = _normal((pool, P, c["H_kv"], D), g)
    else:
        P, B = c["P"], c["B"]
        keep = _spread(c["keep_lo"], c["keep_hi"], B)
        start = _spread(c["dst_lo"], c["dst_hi"], B)
        table, pool = _tables([c["span"]] * B + [a + k for a, k in zip(start, keep)], P, g)
        s["src_table"], s["dst_table"] = table[:B].contiguous(), table[B:].contiguous()
        pos = torch.zeros(B, c["keep_hi"], dtype=torch.int32, device=DEV)
        for b, k in enumerate(keep):
            pick = torch.randperm(c["span"], generator=g, device=DEV)[:k]
            pos[b, :k] = pick.sort().values.to(torch.int32)
        s["pos"], s["keep"], s["start"] = pos, _i32(keep), _i32(start)
        s["k"] = _normal((pool, P, c["H_kv"], D), g)
        s["v"] = _normal((pool, P, c["H_kv"], D), g)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import cascade_paged_attention_gb300 as cpa
    c = s["case"]
    if c["op"] == "decode":
        kw = dict(max_seq_len=s["max_len"], window=c["window"], sinks=c["sinks"], o=s["o"],
                  lse=s["lse"], workspace=s["scratch"])
        if c["fp8"]:
            return cpa.cpa_decode_fp8(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"],
                                      s["table"], s["lens"], **kw)
        return cpa.cpa_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], **kw)
    if c["op"] == "prefill":
        return cpa.cpa_window_prefill(s["q"], s["k"], s["v"], s["table"], s["q_start"], s["lens"],
                                      max_new=c["new_hi"], max_seq_len=s["max_len"],
                                      window=c["window"], sinks=c["sinks"], o=s["o"],
                                      lse=s["lse"], workspace=s["scratch"])
    if c["op"] == "fork":
        cpa.cpa_cache_free(s["table"], s["children"], s["first"], s["last"], s["refs"],
                           workspace=s["scratch"])
        cpa.cpa_cache_fork(s["table"], s["lens"], s["parents"], s["children"], s["refs"], c["P"],
                           copy_src=s["src"], copy_dst=s["dst"], workspace=s["scratch"])
        cpa.cpa_cache_copy_pages(s["k"], s["v"], s["src"], s["dst"], workspace=s["scratch"])
        return [s[k] for k in ("table", "lens", "refs", "src", "dst", "k", "v")]
    cpa.cpa_cache_compact(s["k"], s["v"], s["src_table"], s["pos"], s["keep"],
                          dst_page_table=s["dst_table"], dst_start=s["start"],
                          workspace=s["scratch"])
    return s["k"], s["v"]


def _plain(s):
    return {"decode": _plain_decode, "prefill": _plain_prefill, "fork": _plain_fork,
            "compact": _plain_compact}[s["case"]["op"]](s)


def _keys(s, table, pos):
    """K and V in 32 bits at positions pos [B, n] of each request: [B, H_kv, n, D]."""
    P = s["case"]["P"]
    page = torch.gather(table.long(), 1, (pos // P).clamp(0, table.shape[1] - 1)).clamp(min=0)
    out = []
    for name in ("k", "v"):
        x = s[name][page, pos % P]
        if name + "_scale" in s:
            x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"]
        out.append(x.float().transpose(1, 2))
    return out


def _softmax(x, seen):
    """Weights and log-sum-exp over the last axis where seen."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    t = e.sum(-1, keepdim=True)
    w = e / torch.where(t == 0, torch.ones_like(t), t)
    return w, (m + torch.log(t)).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, H_kv, G, W = c["B"], c["H_kv"], c["H_q"] // c["H_kv"], c["window"]
    L = s["lens"].long()[:, None]
    lo = (L - W).clamp(min=0) if W else torch.zeros_like(L)
    sink = lo.clamp(max=c["sinks"])
    most = min(s["max_len"], W + c["sinks"]) if W else s["max_len"]
    i = torch.arange(most, device=DEV)[None]
    pos = torch.where(i < sink, i, i - sink + lo)
    k, v = _keys(s, s["table"], torch.minimum(pos, L - 1))
    x = (s["q"].float().view(B, H_kv, G, D) @ k.transpose(2, 3)) * D ** -0.5
    w, lse = _softmax(x, (i < sink + L - lo)[:, None, None])
    return (w @ v).reshape(B, c["H_q"], D).to(torch.bfloat16), lse.reshape(B, c["H_q"])


def _plain_prefill(s):
    c = s["case"]
    B, H_kv, G, W, M = c["B"], c["H_kv"], c["H_q"] // c["H_kv"], c["window"], c["new_hi"]
    T = s["q"].shape[0]
    start = s["q_start"].long()
    L = s["lens"].long()
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1    # the request of each token
    i = t - start[b]
    q = torch.zeros(B, M, c["H_q"], D, device=DEV)
    q[b, i] = s["q"].float()
    j = torch.arange(s["max_len"], device=DEV)[None].expand(B, -1)
    k, v = _keys(s, s["table"], torch.minimum(j, L[:, None] - 1))
    m = start[1:] - start[:-1]
    p = (L - m)[:, None, None] + torch.arange(M, device=DEV)[None, :, None]
    j = j[:, None]
    seen = j <= p
    if W:
        seen = seen & ((j > p - W) | (j < c["sinks"]))
    q = q.view(B, M, H_kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * M, D)
    x = (q @ k.transpose(2, 3)).view(B, H_kv, G, M, -1) * D ** -0.5
    w, lse = _softmax(x, seen[:, None, None])
    o = (w.reshape(B, H_kv, G * M, -1) @ v).view(B, H_kv, G, M, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, c["H_q"], D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, M, c["H_q"])
    return o[b, i].to(torch.bfloat16), lse[b, i]


def _plain_fork(s):
    P, table, lens, refs = s["case"]["P"], s["table"], s["lens"], s["refs"]
    par, chi = s["parents"].long(), s["children"].long()
    col = torch.arange(table.shape[1], device=DEV)[None]
    # give back what the children's rows hold
    rows = table[chi]
    live = (col >= s["first"][:, None]) & (col < s["last"][:, None]) & (rows >= 0)
    refs.index_add_(0, rows.clamp(min=0).long().view(-1), -live.to(torch.int32).view(-1))
    table[chi] = torch.where(live, torch.full_like(rows, -1), rows)
    # whole pages are shared; the last, partly filled one becomes the lowest free page
    L = lens[par].long()
    whole, tail = (L // P)[:, None], L % P > 0
    rows = table[par]
    rank = torch.cumsum(tail.long(), 0)
    new = torch.searchsorted(torch.cumsum((refs == 0).long(), 0), rank).to(torch.int32)
    old = torch.gather(rows, 1, whole.clamp(max=table.shape[1] - 1)).squeeze(1)
    none = torch.full_like(rows, -1)
    shared = col < whole
    table[chi] = torch.where(shared, rows, torch.where((col == whole) & tail[:, None],
                                                       new[:, None], none))
    refs.index_add_(0, rows.clamp(min=0).long().view(-1), shared.to(torch.int32).view(-1))
    refs.index_add_(0, new.long(), tail.to(torch.int32))
    lens[chi] = lens[par]
    s["src"].copy_(torch.where(tail, old, torch.full_like(old, -1)))
    s["dst"].copy_(torch.where(tail, new, torch.full_like(new, -1)))
    # every prompt here ends inside a page, so every pair is a copy
    for name in ("k", "v"):
        s[name][s["dst"].long()] = s[name][s["src"].long()]
    return [table, lens, refs, s["src"], s["dst"], s["k"], s["v"]]


def _plain_compact(s):
    P = s["case"]["P"]
    i = torch.arange(s["pos"].shape[1], device=DEV)[None]
    # past a request's count the first token is moved again, which changes nothing
    i = torch.where(i < s["keep"][:, None], i, torch.zeros_like(i)).long()
    a = torch.gather(s["pos"].long(), 1, i)
    z = s["start"].long()[:, None] + i
    src = torch.gather(s["src_table"].long(), 1, a // P) * P + a % P
    dst = torch.gather(s["dst_table"].long(), 1, z // P) * P + z % P
    for name in ("k", "v"):
        rows = s[name].view(-1, s["case"]["H_kv"], D)
        rows[dst.view(-1)] = rows[src.view(-1)]
    return s["k"], s["v"]


# ----------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    """Request by request and block of queries by block: softmax(q K^T / sqrt d) V over the keys
    that a position sees.  The page operations move values and compute none."""
    c = case
    if c["op"] not in ("decode", "prefill"):
        return None
    if work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    G = c["H_q"] // c["H_kv"]
    lens = s["lens"].tolist()
    starts = s["q_start"].tolist() if "q_start" in s else list(range(c["B"] + 1))
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        dense = []
        for name in ("k", "v"):
            pages = s[name][s["table"][b, :-(-L // c["P"])].long()]
            if c.get("fp8"):
                x = pages.view(torch.float8_e4m3fn).double() * s[name + "_scale"].double()
            else:
                x = pages.double()
            dense.append(x.reshape(-1, c["H_kv"], D)[:L].repeat_interleave(G, 1))
        K, V = dense
        m = starts[b + 1] - starts[b]
        for i0 in range(0, m, 128):
            i1 = min(m, i0 + 128)
            p = torch.arange(L - m + i0, L - m + i1, device=DEV)
            top = L - m + i1
            bottom = max(0, L - m + i0 + 1 - c["window"]) if c["window"] else 0
            cols = torch.arange(top, device=DEV)
            cols = cols[(cols >= bottom) | (cols < c["sinks"])]
            ok = cols[None] <= p[:, None]
            if c["window"]:
                ok &= (p[:, None] - cols[None] < c["window"]) | (cols[None] < c["sinks"])
            q = s["q"][starts[b] + i0:starts[b] + i1].double()
            x = torch.einsum("ihd,jhd->hij", q, K[cols]) / math.sqrt(D)
            x.masked_fill_(~ok[None], -math.inf)
            z = torch.logsumexp(x, -1)
            o[starts[b] + i0:starts[b] + i1] = torch.einsum("hij,jhd->ihd", torch.exp(x - z[..., None]), V[cols])
            lse[starts[b] + i0:starts[b] + i1] = z.T
    return o, lse
