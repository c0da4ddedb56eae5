"""Refusals of writing rows to pages, reading them back and latent attention that need no
GPU: the C entry points' argument checks and the binding's tensor checks."""
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


PTR = object()
APPEND = dict(k=PTR, v=PTR, ks=4096, vs=4096, kp=PTR, vp=PTR, table=PTR, stride=4, start=PTR,
              lens=PTR, B=2, T=5, P=16, pages=8, token=2048, ws=PTR, nbytes=256)
APPEND_FP8 = dict(k=PTR, v=PTR, ks=4096, vs=4096, kp=PTR, vp=PTR, k_scale=PTR, v_scale=PTR, per=1,
                  table=PTR, stride=4, start=PTR, lens=PTR, B=2, T=5, channels=1024, P=16, pages=8,
                  ws=PTR, nbytes=256)
LATENT_APPEND = dict(c=PTR, r=PTR, cs=1024, rs=128, kp=PTR, table=PTR, stride=4, start=PTR,
                     lens=PTR, B=2, T=5, C=512, R=64, P=16, pages=8, ws=PTR, nbytes=256)
GATHER = dict(kp=PTR, vp=PTR, table=PTR, stride=4, start=PTR, first=None, B=2, T=5, P=16, pages=8,
              token=2048, k=PTR, v=PTR, ws=PTR, nbytes=256)
GATHER_FP8 = dict(kp=PTR, vp=PTR, k_scale=PTR, v_scale=PTR, per=1, table=PTR, stride=4, start=PTR,
                  first=None, B=2, T=5, channels=1024, P=16, pages=8, k=PTR, v=PTR, ws=PTR,
                  nbytes=256)
LATENT_GATHER = dict(kp=PTR, table=PTR, stride=4, start=PTR, first=None, B=2, T=5, C=512, R=64,
                     P=16, pages=8, c=PTR, r=PTR, ws=PTR, nbytes=256)
DECODE = dict(q_c=PTR, ct=4096, ch=512, q_r=PTR, rt=512, rh=64, kp=PTR, table=PTR, stride=4,
              lens=PTR, B=2, S=1, H=8, C=512, R=64, P=16, pages=8, max_len=64, scale=0.07, o=PTR,
              lse=PTR, ws=PTR, nbytes=1 << 30)
PREFILL = dict(q=PTR, k=PTR, kt=2048, kh=256, rope=PTR, rs=64, v=PTR, vt=2048, vh=256, start=PTR,
               k_start=PTR, B=2, T=5, T_k=9, H=8, nope=128, R=64, vd=128, scale=0.07, o=PTR,
               lse=PTR, ws=PTR, nbytes=1 << 30)
BASES = {"cache_append": APPEND, "cache_append_fp8": APPEND_FP8, "latent_append": LATENT_APPEND,
         "cache_gather": GATHER, "cache_gather_fp8": GATHER_FP8, "latent_gather": LATENT_GATHER,
         "latent_decode": DECODE, "latent_prefill": PREFILL}


def call(L, p, fn, **kw):
    a = dict(BASES[fn], **kw)
    return getattr(L, "cpa_" + fn)(*[p if x is PTR else x for x in a.values()], None)


@pytest.mark.parametrize("fn", sorted(BASES))
def test_null_and_unaligned_pointers_and_workspaces(L, p, fn):
    odd = ctypes.c_void_p(p.value + 8)
    for n, x in BASES[fn].items():
        if x is not PTR:
            continue
        if n == "ws":
            assert call(L, p, fn, ws=None) == 3
            continue
        assert call(L, p, fn, **{n: None}) == 1, n
        if n not in ("table", "start", "k_start", "lens", "lse", "k_scale", "v_scale"):
            assert call(L, p, fn, **{n: odd}) == 1, n
    assert call(L, p, fn, nbytes=255) == 3
    assert call(L, p, fn, ws=ctypes.c_void_p(p.value + 2)) == 1


@pytest.mark.parametrize("fn", sorted(BASES))
@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(pages=0), 1), (dict(stride=0), 1), (dict(P=12), 2),
    (dict(P=512), 2), (dict(pages=1 << 28), 2), (dict(token=24), 1), (dict(token=0), 1),
    (dict(token=1 << 21), 2), (dict(channels=24), 1), (dict(channels=0), 1),
    (dict(channels=1 << 20), 2), (dict(C=256), 2), (dict(R=32), 2), (dict(ks=2050), 1),
    (dict(vs=8), 1), (dict(cs=1032), 1), (dict(S=0), 1), (dict(H=0), 1), (dict(max_len=-1), 1),
    (dict(max_len=65), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1), (dict(ct=0), 1), (dict(ch=4), 1),
    (dict(rt=-512), 1), (dict(rh=0), 1), (dict(kt=0), 1), (dict(kh=12), 1), (dict(vt=-8), 1),
    (dict(vh=0), 1), (dict(T_k=-1), 1), (dict(nope=64), 2), (dict(vd=64), 2)])
def test_sizes_out_of_range(L, p, fn, kw, status):
    if set(kw) <= set(BASES[fn]):
        assert call(L, p, fn, **kw) == status


def test_row_limits(L, p):
    assert call(L, p, "cache_append", T=(1 << 30) + 1) == 2
    assert call(L, p, "cache_gather", T=(1 << 30) + 1) == 2
    assert call(L, p, "latent_prefill", T=1 << 22) == 2
    assert call(L, p, "latent_prefill", T_k=(1 << 30) + 1) == 2
    assert call(L, p, "latent_decode", B=1 << 20) == 2
    assert call(L, p, "latent_decode", S=65) == 2
    assert call(L, p, "latent_decode", max_len=(1 << 30) + 1, stride=1 << 27) == 2


@pytest.mark.parametrize("fn", ["cache_append", "cache_append_fp8", "cache_gather", "cache_gather_fp8"])
def test_more_rows_than_a_grid_has_blocks_for(L, p, fn):
    """Rows may overlap (a stride of 0), so their number is not bounded by memory alone."""
    wide = dict(channels=1 << 19) if "fp8" in fn else dict(token=1 << 20)
    small = dict(ks=0, vs=0) if "append" in fn else {}
    assert call(L, p, fn, T=1 << 30, **wide, **small) == 2


def test_workspace_sizes(L):
    for bad in ((0, 1, 8, 512, 64, 16), (1, 0, 8, 512, 64, 16), (1, 1, 0, 512, 64, 16),
                (1, 1, 8, 256, 64, 16), (1, 1, 8, 512, 32, 16), (1, 1, 8, 512, 64, 7),
                (1, 65, 8, 512, 64, 16)):
        assert L.cpa_latent_decode_workspace_size(*bad) == 0
    for bad in ((0, 1, 1, 8, 128, 64, 128), (1, -1, 1, 8, 128, 64, 128), (1, 1, -1, 8, 128, 64, 128),
                (1, 1, 1, 0, 128, 64, 128), (1, 1, 1, 8, 64, 64, 128), (1, 1, 1, 8, 128, 32, 128),
                (1, 1, 1, 8, 128, 64, 64)):
        assert L.cpa_latent_prefill_workspace_size(*bad) == 0


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_types():
    kv, new, lat = _cpu(4, 16, 2, 128), _cpu(3, 2, 128), _cpu(4, 16, 576)
    table, one = _cpu(2, 4, dtype=torch.int32), _cpu(2, dtype=torch.int32)
    start, scale = _cpu(3, dtype=torch.int32), _cpu(1, dtype=torch.float32)
    for call in (lambda: cpa.cpa_cache_append(new, new, kv, kv, table, start, one),
                 lambda: cpa.cpa_cache_append_fp8(new, new, kv.byte(), kv.byte(), scale, scale,
                                                  table, start, one),
                 lambda: cpa.cpa_cache_gather(kv, kv, table, start, T=3),
                 lambda: cpa.cpa_cache_gather_fp8(kv.byte(), kv.byte(), scale, scale, table, start, 3),
                 lambda: cpa.cpa_latent_append(_cpu(3, 512), _cpu(3, 64), lat, table, start, one),
                 lambda: cpa.cpa_latent_gather(lat, table, start, T=3),
                 lambda: cpa.cpa_latent_decode(_cpu(2, 8, 512), _cpu(2, 8, 64), lat, table, one),
                 lambda: cpa.cpa_latent_prefill(_cpu(3, 8, 192), _cpu(5, 8, 128), _cpu(5, 64),
                                                _cpu(5, 8, 128), start, start)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError, match="bfloat16"):
        cpa.cpa_latent_gather(lat.half(), table, start, T=3)
    with pytest.raises(TypeError, match="torch.Tensor"):
        cpa.cpa_latent_prefill([0], new, new, new, start, start)
