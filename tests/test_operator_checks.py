"""Refusals of decode, windowed prefill and the page operations that need no GPU:
the binding's tensor checks and the C entry points' argument checks."""
import ctypes

import pytest
import torch

import cascade_paged_attention_gb300 as cpa


@pytest.fixture(scope="module")
def L():
    cpa.build_library()
    return cpa.lib()


@pytest.fixture(scope="module")
def p():
    """An aligned pointer that no call may follow."""
    buf = (ctypes.c_uint8 * 4352)()
    ptr = ctypes.c_void_p((ctypes.addressof(buf) + 255) // 256 * 256)
    ptr.keep = buf
    return ptr


DECODE = dict(q=1, k=1, v=1, table=1, stride=4, lens=1, B=2, H_q=8, H_kv=2, d=128, P=16, pages=8,
              max_len=64, window=0, sinks=0, scale=0.088, o=1, lse=1, ws=1, nbytes=1 << 30)


def _args(base, p, kw):
    a = dict(base, **kw)
    ptrs = ("q", "k", "v", "ks", "vs", "table", "lens", "start", "o", "lse", "ws", "rows", "parents",
            "children", "refs", "src", "dst", "first", "last", "pos", "keep", "dst_start")
    return [(p if x == 1 else x) if n in ptrs else x for n, x in a.items()] + [None]


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(o=None), 1),
    (dict(lse=None), 1), (dict(B=0), 1), (dict(H_q=9), 1), (dict(H_kv=0), 1), (dict(max_len=-1), 1),
    (dict(stride=3), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(d=64), 2), (dict(P=12), 2),
    (dict(P=512), 2), (dict(pages=1 << 28), 2), (dict(ws=None), 3), (dict(nbytes=16), 3),
    (dict(pages=0), 1)])
def test_decode_refuses(L, p, kw, status):
    assert L.cpa_decode(*_args(DECODE, p, kw)) == status


def test_decode_fp8_refuses(L, p):
    base = dict(q=1, k=1, v=1, ks=1, vs=1, per=0, **{k: x for k, x in DECODE.items()
                                                     if k not in ("q", "k", "v")})
    assert L.cpa_decode_fp8(*_args(base, p, dict(ks=None))) == 1
    assert L.cpa_decode_fp8(*_args(base, p, dict(vs=None))) == 1
    assert L.cpa_decode_fp8(*_args(base, p, dict(d=64))) == 2


def test_unaligned_pointers_are_refused(L, p):
    odd = ctypes.c_void_p(p.value + 8)
    for n in ("q", "k", "v", "o", "ws"):
        assert L.cpa_decode(*_args(DECODE, p, {n: odd})) == 1
        assert L.cpa_window_prefill(*_args(PREFILL, p, {n: odd})) == 1


PREFILL = dict(q=1, k=1, v=1, table=1, stride=4, start=1, lens=1, B=2, T=10, H_q=8, H_kv=2, d=128,
               P=16, pages=8, max_new=8, max_len=64, window=0, sinks=0, scale=0.088, o=1, lse=1,
               ws=1, nbytes=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(start=None), 1), (dict(lens=None), 1), (dict(o=None), 1), (dict(B=0), 1),
    (dict(T=-1), 1), (dict(max_new=-1), 1), (dict(max_len=-1), 1), (dict(stride=3), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=-1.0), 1), (dict(H_q=7), 1),
    (dict(d=64), 2), (dict(P=4), 2), (dict(H_q=258), 2), (dict(ws=None), 3), (dict(nbytes=16), 3)])
def test_window_prefill_refuses(L, p, kw, status):
    assert L.cpa_window_prefill(*_args(PREFILL, p, kw)) == status


FORK = dict(table=1, stride=4, n_rows=4, lens=1, parents=1, children=1, n=2, refs=1, P=16, pages=8,
            src=1, dst=1, ws=1, nbytes=1 << 30)
FREE = dict(table=1, stride=4, n_rows=4, rows=1, first=1, last=1, n=2, refs=1, pages=8, ws=1,
            nbytes=256)
COPY = dict(k=1, v=1, src=1, dst=1, n=2, pages=8, page_bytes=4096, ws=1, nbytes=256)
COMPACT = dict(k=1, v=1, src=1, stride=4, n_rows=2, rows=None, pos=1, max_keep=3, keep=1, dst=1,
               dst_stride=4, dst_start=1, B=2, P=16, pages=8, token=256, ws=1, nbytes=256)


@pytest.mark.parametrize("fn,base,kw,status", [
    ("fork", FORK, dict(table=None), 1), ("fork", FORK, dict(parents=None), 1),
    ("fork", FORK, dict(n=-1), 1), ("fork", FORK, dict(stride=0), 1), ("fork", FORK, dict(P=3), 2),
    ("fork", FORK, dict(nbytes=256), 3), ("fork", FORK, dict(pages=0), 1),
    ("fork", FORK, dict(src=None), 1), ("fork", FORK, dict(pages=1 << 28), 2),
    ("free", FREE, dict(refs=None), 1), ("free", FREE, dict(rows=None), 1),
    ("free", FREE, dict(n_rows=0), 1), ("free", FREE, dict(nbytes=255), 3),
    ("free", FREE, dict(n=-1), 1),
    ("copy_pages", COPY, dict(k=None), 1), ("copy_pages", COPY, dict(page_bytes=24), 1),
    ("copy_pages", COPY, dict(page_bytes=0), 1), ("copy_pages", COPY, dict(dst=None), 1),
    ("copy_pages", COPY, dict(ws=None), 3), ("copy_pages", COPY, dict(n=-1), 1),
    ("compact", COMPACT, dict(v=None), 1), ("compact", COMPACT, dict(keep=None), 1),
    ("compact", COMPACT, dict(dst_start=None), 1), ("compact", COMPACT, dict(n_rows=1), 1),
    ("compact", COMPACT, dict(dst_stride=0), 1), ("compact", COMPACT, dict(token=24), 1),
    ("compact", COMPACT, dict(P=7), 2), ("compact", COMPACT, dict(nbytes=0), 3),
    ("compact", COMPACT, dict(max_keep=-1), 1), ("compact", COMPACT, dict(B=0), 1)])
def test_page_operations_refuse(L, p, fn, base, kw, status):
    assert getattr(L, "cpa_cache_" + fn)(*_args(base, p, kw)) == status


def test_workspace_sizes(L):
    assert cpa.cpa_decode_workspace_size(0, 8, 2, 128, 16) == 0
    assert cpa.cpa_decode_workspace_size(1, 9, 2, 128, 16) == 0
    assert cpa.cpa_decode_workspace_size(1, 8, 2, 64, 16) == 0
    assert cpa.cpa_decode_workspace_size(1, 8, 2, 128, 5) == 0
    assert cpa.cpa_window_prefill_workspace_size(0, 1, 8, 2, 128, 16, 1) == 0
    assert cpa.cpa_window_prefill_workspace_size(1, 1, 258, 2, 128, 16, 1) == 0
    assert cpa.cpa_cache_fork_workspace_size(0) == 0
    assert cpa.cpa_cache_fork_workspace_size(1) >= 256 + 4 + 512
    # 4 bytes for each 4096 pages, a bit a page
    assert cpa.cpa_cache_fork_workspace_size(4096 * 50) >= 256 + 50 * (4 + 512)


def test_new_status_codes_have_their_own_text(L):
    texts = {cpa.cpa_status_string(i) for i in range(13)}
    assert len(texts) == 13 and "unknown status" not in texts


def _cpu(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_types():
    kv, i2, i1 = _cpu((4, 16, 2, 128)), _cpu((2, 4), torch.int32), _cpu((2,), torch.int32)
    q = _cpu((2, 8, 128))
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_decode(q, kv, kv, i2, i1)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_window_prefill(q, kv, kv, i2, _cpu((3,), torch.int32), i1)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_cache_fork(i2, i1, i1, i1, i1, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_cache_free(i2, i1, i1, i1, i1)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_cache_copy_pages(kv, kv, i1, i1)
    with pytest.raises(ValueError, match="CUDA device"):
        cpa.cpa_cache_compact(kv, kv, i2, i2, i1, dst_start=i1)
    with pytest.raises(TypeError, match="bfloat16"):
        cpa.cpa_decode(q.half(), kv, kv, i2, i1)
    with pytest.raises(TypeError, match="torch.Tensor"):
        cpa.cpa_cache_copy_pages([0], kv, i1, i1)


def test_fork_workspace_holds_a_count_for_each_1024_pages(L):
    """The status word, a count of 4 bytes for each 1024 pages, a bit a page."""
    for chunks in (1, 200, 684):
        for pages in (1024 * chunks, 1024 * chunks - 1023):
            assert cpa.cpa_cache_fork_workspace_size(pages) >= 256 + chunks * (4 + 128)
