"""Python binding of libcpa.so, the cascade paged-attention library for sm_103a.

Argument marshalling only: every function here checks tensor dtypes, shapes
and devices, allocates outputs / workspace with PyTorch when the caller does
not pass them, and calls the C entry point of the same name on PyTorch's
current CUDA stream.  All arithmetic runs in the library's CUDA kernels; there
is no fallback path, and a missing library raises ``RuntimeError``.

Every call that takes a workspace (and the static-scratch call) accepts
``check=True``: after the launch it reads the device status word
(synchronising the stream) and raises ``CpaError`` when the GPU recorded a bad
page id, a bad length, a bad tree parent or a pipeline timeout, or a bad row, a
bad count or a lack of free pages in a page operation.  The outputs of such a
call are undefined unless include/cpa.h says what they are.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

__all__ = [
    "CpaError",
    "lib",
    "build_library",
    "cpa_status_string",
    "cpa_version",
    "cpa_cascade_verify_workspace_size",
    "cpa_prefill_hit_workspace_size",
    "cpa_status_workspace_size",
    "cpa_cascade_verify",
    "cpa_cascade_verify_noalloc",
    "cpa_cascade_verify_fp8",
    "cpa_cascade_pass_a_fp8",
    "cpa_naive_expand_verify",
    "cpa_cascade_pass_a",
    "cpa_cascade_pass_b",
    "cpa_merge_state",
    "cpa_prefill_hit",
    "cpa_cascade_verify_shared_workspace_size",
    "cpa_cascade_verify_shared",
    "cpa_tree_verify_workspace_size",
    "cpa_tree_verify",
    "cpa_tree_pass_b",
    "cpa_decode_workspace_size",
    "cpa_decode",
    "cpa_decode_fp8",
    "cpa_window_prefill_workspace_size",
    "cpa_window_prefill",
    "cpa_cache_fork_workspace_size",
    "cpa_cache_fork",
    "cpa_cache_free",
    "cpa_cache_copy_pages",
    "cpa_cache_compact",
    "cpa_get_device_status",
    "cpa_noalloc_device_status",
    "cpa_debug_wait_timeout",
    "cpa_plan_partition",
    "declared_functions",
    "PREFILL_FULL",
    "PREFILL_RECT",
    "PREFILL_TRI",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcpa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "cpa.h")

PREFILL_FULL, PREFILL_RECT, PREFILL_TRI = 0, 1, 2
_STATUS = {0: "CPA_OK", 1: "CPA_ERR_INVALID_ARG", 2: "CPA_ERR_UNSUPPORTED",
           3: "CPA_ERR_WORKSPACE", 4: "CPA_ERR_LAUNCH", 5: "CPA_ERR_BAD_PAGE",
           6: "CPA_ERR_TIMEOUT", 7: "CPA_ERR_CUDA", 8: "CPA_ERR_BAD_LENGTH",
           9: "CPA_ERR_BAD_TREE", 10: "CPA_ERR_BAD_ROW", 11: "CPA_ERR_NO_PAGE",
           12: "CPA_ERR_BAD_COUNT"}


class CpaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {_STATUS.get(status, status)}: "
                         f"{cpa_status_string(status)}")


_lib: Optional[ctypes.CDLL] = None
_STATUS_BYTES = 256  # cpa_status_workspace_size()


def build_library(force: bool = False) -> str:
    """Compile libcpa.so in-tree (nvcc, sm_103a)."""
    import importlib
    return importlib.import_module(__name__ + ".build").build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded library: libcpa.so, or the build that $CPA_LIBRARY names (the
    diagnostic trace build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = os.environ.get("CPA_LIBRARY") or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m cascade_paged_attention_gb300.build`")
    L = ctypes.CDLL(path)
    P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                        ctypes.c_size_t)
    verify_args = [P, P, P, P, I, P, I, P, I, I, I, I, I, I, I, I, I, F, P, P, P, SZ, P]
    sig = {
        "cpa_status_string": (ctypes.c_char_p, [I]),
        "cpa_version": (I, []),
        "cpa_status_workspace_size": (SZ, []),
        "cpa_cascade_verify_workspace_size": (SZ, [I, I, I, I, I, I, I]),
        "cpa_prefill_hit_workspace_size": (SZ, [I, I, I, I, I, I, I]),
        "cpa_cascade_verify": (I, verify_args),
        "cpa_naive_expand_verify": (I, verify_args),
        "cpa_cascade_verify_noalloc": (I, verify_args[:20] + [P]),
        "cpa_cascade_verify_fp8": (I, verify_args[:3] + [P, P, I] + verify_args[3:]),
        "cpa_cascade_pass_a_fp8": (I, [P, P, P, P, P, I, P, I, P, I, I, I, I, I, I, I, I, I, F, P,
                                       P, P, SZ, P]),
        "cpa_cascade_pass_a": (I, [P, P, P, P, I, P, I, I, I, I, I, I, I, I, I, F, P, P, P, SZ,
                                   P]),
        "cpa_cascade_pass_b": (I, [P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, P, P, SZ, P]),
        "cpa_merge_state": (I, [P, P, P, P, I, I, I, P, P, P]),
        "cpa_prefill_hit": (I, [P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, P, P, SZ, P]),
        "cpa_cascade_verify_shared_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
        "cpa_cascade_verify_shared": (I, [P, P, P, P, I, I, I, P, I, P, I, P, I, I, I, I, I, I,
                                          I, I, I, F, P, P, P, SZ, P]),
        "cpa_tree_verify_workspace_size": (SZ, [I, I, I, I, I, I]),
        "cpa_tree_verify": (I, [P, P, P, P, I, P, I, P, P, I, I, I, I, I, I, I, I, F, P, P, P, SZ,
                                P]),
        "cpa_tree_pass_b": (I, [P, P, P, P, I, P, I, I, I, I, I, I, I, F, P, P, P, SZ, P]),
        "cpa_decode_workspace_size": (SZ, [I, I, I, I, I]),
        "cpa_decode": (I, [P, P, P, P, I, P, I, I, I, I, I, I, I, I, I, F, P, P, P, SZ, P]),
        "cpa_decode_fp8": (I, [P, P, P, P, P, I, P, I, P, I, I, I, I, I, I, I, I, I, F, P, P, P,
                               SZ, P]),
        "cpa_window_prefill_workspace_size": (SZ, [I, I, I, I, I, I, I]),
        "cpa_window_prefill": (I, [P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, I, I, I, F, P, P,
                                   P, SZ, P]),
        "cpa_cache_fork_workspace_size": (SZ, [I]),
        "cpa_cache_fork": (I, [P, I, I, P, P, P, I, P, I, I, P, P, P, SZ, P]),
        "cpa_cache_free": (I, [P, I, I, P, P, P, I, P, I, P, SZ, P]),
        "cpa_cache_copy_pages": (I, [P, P, P, P, I, I, SZ, P, SZ, P]),
        "cpa_cache_compact": (I, [P, P, P, I, I, P, P, I, P, P, I, P, I, I, I, SZ, P, SZ, P]),
        "cpa_get_device_status": (I, [P, ctypes.POINTER(ctypes.c_uint32), P]),
        "cpa_noalloc_device_status": (I, [ctypes.POINTER(ctypes.c_uint32), P]),
        "cpa_debug_wait_timeout": (I, [P, SZ, I, P]),
        "cpa_plan_partition": (I, [I64, I, I, I64, ctypes.POINTER(ctypes.c_int64),
                                   ctypes.POINTER(ctypes.c_int64)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def declared_functions() -> list[str]:
    """Names of the functions include/cpa.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(cpa_[a-z0-9_]+)\s*\(", text)))


def cpa_status_string(status: int) -> str:
    return lib().cpa_status_string(int(status)).decode()


def cpa_version() -> int:
    return lib().cpa_version()


def cpa_status_workspace_size() -> int:
    return lib().cpa_status_workspace_size()


def cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, head_dim, page_size) -> int:
    return lib().cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, head_dim, page_size)


def cpa_prefill_hit_workspace_size(B, N, H_hit, H_q, H_kv, head_dim, page_size) -> int:
    return lib().cpa_prefill_hit_workspace_size(B, N, H_hit, H_q, H_kv, head_dim, page_size)


# ---------------------------------------------------------------- marshalling helpers
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, ndim: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")


_ws_cache: dict = {}


def _workspace(nbytes: int, device: torch.device, workspace: Optional[torch.Tensor]):
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        return workspace
    key = (device.index, nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _ws_cache.clear()
        _ws_cache[key] = ws
    return ws


def _check(fn: str, status: int):
    if status != 0:
        raise CpaError(fn, status)


def _check_device(fn: str, workspace: torch.Tensor, stream):
    """Raise if the device status word of `workspace` has any bit set (synchronises)."""
    st, word = cpa_get_device_status(workspace, stream)
    if st != 0:
        raise CpaError(f"{fn} (device status word {word:#x})", st)


def _verify_shapes(q, k_pages, v_pages, prefix_page_table, prefix_lens, topk, S):
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(prefix_page_table, "prefix_page_table", torch.int32, 2)
    _need(prefix_lens, "prefix_lens", torch.int32, 1)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, page_size, H_kv, d = k_pages.shape
    B = prefix_lens.numel()
    T, H_q, dq = q.shape
    if dq != d or T != B * topk * S or prefix_page_table.shape[0] != B:
        raise ValueError("inconsistent verify shapes")
    return B, H_q, H_kv, d, page_size, num_pages


def _verify_call(name, q, k_pages, v_pages, prefix_page_table, draft_page_table, prefix_lens,
                 topk, S, max_prefix_len, sm_scale, o, lse, workspace, stream, check=False):
    B, H_q, H_kv, d, P, num_pages = _verify_shapes(q, k_pages, v_pages, prefix_page_table,
                                                    prefix_lens, topk, S)
    _need(draft_page_table, "draft_page_table", torch.int32, 2)
    if draft_page_table.shape[0] != B * topk:
        raise ValueError("draft_page_table must have B*topk rows")
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o, "o", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    nbytes = cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, d, P)
    ws = _workspace(nbytes, q.device, workspace)
    st = getattr(lib(), name)(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(draft_page_table), draft_page_table.shape[1],
        _ptr(prefix_lens), B, topk, S, H_q, H_kv, d, P, num_pages, int(max_prefix_len),
        float(sm_scale), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(name, st)
    if check:
        _check_device(name, ws, stream)
    return o, lse


# ---------------------------------------------------------------- entry points
def cpa_cascade_verify(q, k_pages, v_pages, prefix_page_table, draft_page_table, prefix_lens,
                       topk: int, S: int, max_prefix_len: Optional[int] = None,
                       sm_scale: Optional[float] = None, o=None, lse=None, workspace=None,
                       stream=None, check: bool = False):
    """Cascade verify attention (Pass A + Pass B + merge).  Returns (o bf16, lse fp32)."""
    return _verify_call("cpa_cascade_verify", q, k_pages, v_pages, prefix_page_table,
                        draft_page_table, prefix_lens, topk, S, max_prefix_len, sm_scale, o, lse,
                        workspace, stream, check)


def cpa_cascade_verify_noalloc(q, k_pages, v_pages, prefix_page_table, draft_page_table,
                               prefix_lens, topk: int, S: int, o, lse,
                               max_prefix_len: Optional[int] = None,
                               sm_scale: Optional[float] = None, stream=None,
                               check: bool = False):
    """Cascade verify without a workspace, for callers that cannot allocate device memory.

    The library keeps its scratch in a fixed-size array it owns on every GPU,
    and this path allocates nothing: the caller passes preallocated `o`
    (bf16, shaped like q) and `lse` (fp32 [T, H_q]).  Returns (o, lse).
    """
    B, H_q, H_kv, d, P, num_pages = _verify_shapes(q, k_pages, v_pages, prefix_page_table,
                                                    prefix_lens, topk, S)
    _need(draft_page_table, "draft_page_table", torch.int32, 2)
    _need(o, "o", torch.bfloat16, 3)
    _need(lse, "lse", torch.float32, 2)
    if draft_page_table.shape[0] != B * topk or o.shape != q.shape or \
            lse.shape != (q.shape[0], H_q):
        raise ValueError("inconsistent verify shapes")
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    st = lib().cpa_cascade_verify_noalloc(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(draft_page_table), draft_page_table.shape[1],
        _ptr(prefix_lens), B, topk, S, H_q, H_kv, d, P, num_pages, int(max_prefix_len),
        float(sm_scale), _ptr(o), _ptr(lse), _stream(stream))
    _check("cpa_cascade_verify_noalloc", st)
    if check:
        st, word = cpa_noalloc_device_status(stream)
        if st != 0:
            raise CpaError(f"cpa_cascade_verify_noalloc (device status word {word:#x})", st)
    return o, lse


def _fp8_pools(q, k_pages, v_pages, k_scale, v_scale, prefix_page_table, prefix_lens, topk, S):
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.uint8, 4)
    _need(v_pages, "v_pages", torch.uint8, 4)
    _need(k_scale, "k_scale", torch.float32)
    _need(v_scale, "v_scale", torch.float32)
    _need(prefix_page_table, "prefix_page_table", torch.int32, 2)
    _need(prefix_lens, "prefix_lens", torch.int32, 1)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, P, H_kv, d = k_pages.shape
    B = prefix_lens.numel()
    T, H_q, dq = q.shape
    if dq != d or T != B * topk * S or prefix_page_table.shape[0] != B:
        raise ValueError("inconsistent verify shapes")
    n = k_scale.numel()
    if v_scale.numel() != n or n not in (1, H_kv * d):
        raise ValueError("k_scale / v_scale must hold 1 or H_kv * head_dim values each")
    return B, H_q, H_kv, d, P, num_pages, int(n > 1)


def cpa_cascade_verify_fp8(q, k_pages, v_pages, k_scale, v_scale, prefix_page_table,
                           draft_page_table, prefix_lens, topk: int, S: int,
                           max_prefix_len: Optional[int] = None, sm_scale: Optional[float] = None,
                           o=None, lse=None, workspace=None, stream=None, check: bool = False):
    """Cascade verify over FP8 E4M3 KV pages.  Returns (o bf16, lse fp32).

    ``k_pages`` / ``v_pages`` are uint8 E4M3 codes; ``k_scale`` / ``v_scale``
    fp32 with one value each (per tensor) or ``[H_kv, head_dim]`` (per channel).
    """
    B, H_q, H_kv, d, P, num_pages, per_ch = _fp8_pools(q, k_pages, v_pages, k_scale, v_scale,
                                                       prefix_page_table, prefix_lens, topk, S)
    _need(draft_page_table, "draft_page_table", torch.int32, 2)
    if draft_page_table.shape[0] != B * topk:
        raise ValueError("draft_page_table must have B*topk rows")
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o, "o", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    ws = _workspace(cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, d, P), q.device,
                    workspace)
    st = lib().cpa_cascade_verify_fp8(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), per_ch,
        _ptr(prefix_page_table), prefix_page_table.shape[1], _ptr(draft_page_table),
        draft_page_table.shape[1], _ptr(prefix_lens), B, topk, S, H_q, H_kv, d, P, num_pages,
        int(max_prefix_len), float(sm_scale), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
        _stream(stream))
    _check("cpa_cascade_verify_fp8", st)
    if check:
        _check_device("cpa_cascade_verify_fp8", ws, stream)
    return o, lse


def cpa_cascade_pass_a_fp8(q, k_pages, v_pages, k_scale, v_scale, prefix_page_table,
                           prefix_lens, topk: int, S: int, max_prefix_len: Optional[int] = None,
                           sm_scale: Optional[float] = None, o_a=None, lse_a=None,
                           workspace=None, stream=None, check: bool = False):
    """Pass A alone over FP8 E4M3 KV pages.  Returns (o_a fp32, lse_a fp32)."""
    B, H_q, H_kv, d, P, num_pages, per_ch = _fp8_pools(q, k_pages, v_pages, k_scale, v_scale,
                                                       prefix_page_table, prefix_lens, topk, S)
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o_a is None:
        o_a = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse_a is None:
        lse_a = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o_a, "o_a", torch.float32)
    _need(lse_a, "lse_a", torch.float32)
    ws = _workspace(cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, d, P), q.device,
                    workspace)
    st = lib().cpa_cascade_pass_a_fp8(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), per_ch,
        _ptr(prefix_page_table), prefix_page_table.shape[1], _ptr(prefix_lens), B, topk, S, H_q,
        H_kv, d, P, num_pages, int(max_prefix_len), float(sm_scale), _ptr(o_a), _ptr(lse_a),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("cpa_cascade_pass_a_fp8", st)
    if check:
        _check_device("cpa_cascade_pass_a_fp8", ws, stream)
    return o_a, lse_a


def cpa_naive_expand_verify(q, k_pages, v_pages, prefix_page_table, draft_page_table,
                            prefix_lens, topk: int, S: int, max_prefix_len: Optional[int] = None,
                            sm_scale: Optional[float] = None, o=None, lse=None, workspace=None,
                            stream=None, check: bool = False):
    """Naive-expand verify (the baseline).  Returns (o bf16, lse fp32)."""
    return _verify_call("cpa_naive_expand_verify", q, k_pages, v_pages, prefix_page_table,
                        draft_page_table, prefix_lens, topk, S, max_prefix_len, sm_scale, o, lse,
                        workspace, stream, check)


def cpa_cascade_pass_a(q, k_pages, v_pages, prefix_page_table, prefix_lens, topk: int, S: int,
                       max_prefix_len: Optional[int] = None, sm_scale: Optional[float] = None,
                       o_a=None, lse_a=None, workspace=None, stream=None, check: bool = False):
    """Pass A alone.  Returns (o_a fp32, lse_a fp32)."""
    B, H_q, H_kv, d, P, num_pages = _verify_shapes(q, k_pages, v_pages, prefix_page_table,
                                                    prefix_lens, topk, S)
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o_a is None:
        o_a = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse_a is None:
        lse_a = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o_a, "o_a", torch.float32)
    _need(lse_a, "lse_a", torch.float32)
    nbytes = cpa_cascade_verify_workspace_size(B, topk, S, H_q, H_kv, d, P)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().cpa_cascade_pass_a(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(prefix_lens), B, topk, S, H_q, H_kv, d, P, num_pages,
        int(max_prefix_len), float(sm_scale), _ptr(o_a), _ptr(lse_a), _ptr(ws), ws.numel(),
        _stream(stream))
    _check("cpa_cascade_pass_a", st)
    if check:
        _check_device("cpa_cascade_pass_a", ws, stream)
    return o_a, lse_a


def cpa_cascade_pass_b(q, k_pages, v_pages, draft_page_table, B: int, topk: int, S: int,
                       sm_scale: Optional[float] = None, o_b=None, lse_b=None, workspace=None,
                       stream=None, check: bool = False):
    """Pass B alone (warp-level draft kernel).  Returns (o_b fp32, lse_b fp32)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(draft_page_table, "draft_page_table", torch.int32, 2)
    num_pages, P, H_kv, d = k_pages.shape
    T, H_q, _ = q.shape
    if T != B * topk * S or draft_page_table.shape[0] != B * topk:
        raise ValueError("inconsistent Pass B shapes")
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o_b is None:
        o_b = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse_b is None:
        lse_b = torch.empty(T, H_q, dtype=torch.float32, device=q.device)
    ws = _workspace(cpa_status_workspace_size(), q.device, workspace)
    st = lib().cpa_cascade_pass_b(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(draft_page_table), draft_page_table.shape[1],
        B, topk, S, H_q, H_kv, d, P, num_pages, float(sm_scale), _ptr(o_b), _ptr(lse_b),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("cpa_cascade_pass_b", st)
    if check:
        _check_device("cpa_cascade_pass_b", ws, stream)
    return o_b, lse_b


def cpa_merge_state(o_a, lse_a, o_b, lse_b, o_out=None, lse_out=None, stream=None):
    """merge_state of two fp32 partial attentions -> (o bf16, lse fp32)."""
    for t, n in ((o_a, "o_a"), (o_b, "o_b")):
        _need(t, n, torch.float32, 3)
    for t, n in ((lse_a, "lse_a"), (lse_b, "lse_b")):
        _need(t, n, torch.float32, 2)
    n_tokens, H, d = o_a.shape
    if o_b.shape != o_a.shape or lse_a.shape != (n_tokens, H) or lse_b.shape != (n_tokens, H):
        raise ValueError("inconsistent merge_state shapes")
    if o_out is None:
        o_out = torch.empty(o_a.shape, dtype=torch.bfloat16, device=o_a.device)
    if lse_out is None:
        lse_out = torch.empty_like(lse_a)
    st = lib().cpa_merge_state(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), n_tokens, H, d,
                               _ptr(o_out), _ptr(lse_out), _stream(stream))
    _check("cpa_merge_state", st)
    return o_out, lse_out


def cpa_prefill_hit(q, k_pages, v_pages, page_table, B: int, N: int, H_hit: int,
                    part: int = PREFILL_FULL, sm_scale: Optional[float] = None, o=None, lse=None,
                    workspace=None, stream=None, check: bool = False):
    """Prefix-hit prefill.  Returns (o, lse); o is bf16 for PREFILL_FULL, fp32 otherwise."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(page_table, "page_table", torch.int32, 2)
    num_pages, P, H_kv, d = k_pages.shape
    T, H_q, _ = q.shape
    if T != B * (N - H_hit) or page_table.shape[0] != B:
        raise ValueError("inconsistent prefill shapes")
    if sm_scale is None:
        sm_scale = d ** -0.5
    odt = torch.bfloat16 if part == PREFILL_FULL else torch.float32
    if o is None:
        o = torch.empty(q.shape, dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty(T, H_q, dtype=torch.float32, device=q.device)
    _need(o, "o", odt)
    nbytes = cpa_prefill_hit_workspace_size(B, N, H_hit, H_q, H_kv, d, P)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().cpa_prefill_hit(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), page_table.shape[1], B, N,
        H_hit, H_q, H_kv, d, P, num_pages, float(sm_scale), int(part), _ptr(o), _ptr(lse),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("cpa_prefill_hit", st)
    if check:
        _check_device("cpa_prefill_hit", ws, stream)
    return o, lse


def cpa_cascade_verify_shared_workspace_size(B, n_groups, topk, S, H_q, H_kv, head_dim,
                                            page_size) -> int:
    return lib().cpa_cascade_verify_shared_workspace_size(B, n_groups, topk, S, H_q, H_kv,
                                                          head_dim, page_size)


def cpa_cascade_verify_shared(q, k_pages, v_pages, shared_page_table, shared_len: int,
                              prefix_page_table, draft_page_table, prefix_lens, topk: int, S: int,
                              max_prefix_len: Optional[int] = None,
                              sm_scale: Optional[float] = None, o=None, lse=None, workspace=None,
                              stream=None, check: bool = False):
    """Multi-level cascade verify.  Returns (o bf16, lse fp32).

    ``shared_page_table`` int32 [n_groups, stride]: one shared prefix of
    ``shared_len`` tokens per group of ``B // n_groups`` consecutive requests;
    ``prefix_page_table`` / ``prefix_lens`` describe each request's own prefix.
    """
    B, H_q, H_kv, d, P, num_pages = _verify_shapes(q, k_pages, v_pages, prefix_page_table,
                                                    prefix_lens, topk, S)
    _need(shared_page_table, "shared_page_table", torch.int32, 2)
    _need(draft_page_table, "draft_page_table", torch.int32, 2)
    n_groups = shared_page_table.shape[0]
    if draft_page_table.shape[0] != B * topk or n_groups < 1 or B % n_groups:
        raise ValueError("inconsistent multi-level verify shapes")
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o, "o", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    nbytes = cpa_cascade_verify_shared_workspace_size(B, n_groups, topk, S, H_q, H_kv, d, P)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().cpa_cascade_verify_shared(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(shared_page_table),
        shared_page_table.shape[1], n_groups, int(shared_len), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(draft_page_table), draft_page_table.shape[1],
        _ptr(prefix_lens), B, topk, S, H_q, H_kv, d, P, num_pages, int(max_prefix_len),
        float(sm_scale), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check("cpa_cascade_verify_shared", st)
    if check:
        _check_device("cpa_cascade_verify_shared", ws, stream)
    return o, lse


def cpa_tree_verify_workspace_size(B, N, H_q, H_kv, head_dim, page_size) -> int:
    return lib().cpa_tree_verify_workspace_size(B, N, H_q, H_kv, head_dim, page_size)


def _tree_shapes(q, k_pages, v_pages, tree_page_table, tree_parents):
    _need(q, "q", torch.bfloat16, 3)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(tree_page_table, "tree_page_table", torch.int32, 2)
    _need(tree_parents, "tree_parents", torch.int32, 2)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, P, H_kv, d = k_pages.shape
    B, N = tree_parents.shape
    T, H_q, dq = q.shape
    if dq != d or T != B * N or tree_page_table.shape[0] != B:
        raise ValueError("inconsistent tree verify shapes")
    return B, N, H_q, H_kv, d, P, num_pages


def cpa_tree_verify(q, k_pages, v_pages, prefix_page_table, tree_page_table, prefix_lens,
                    tree_parents, max_prefix_len: Optional[int] = None,
                    sm_scale: Optional[float] = None, o=None, lse=None, workspace=None,
                    stream=None, check: bool = False):
    """Verify over draft trees (prefix pass + tree pass + merge).  Returns (o bf16, lse fp32).

    ``tree_parents`` int32 [B, N]: parent BFS index of each node, -1 for a root.
    """
    B, N, H_q, H_kv, d, P, num_pages = _tree_shapes(q, k_pages, v_pages, tree_page_table,
                                                     tree_parents)
    _need(prefix_page_table, "prefix_page_table", torch.int32, 2)
    _need(prefix_lens, "prefix_lens", torch.int32, 1)
    if prefix_lens.numel() != B or prefix_page_table.shape[0] != B:
        raise ValueError("inconsistent tree verify shapes")
    if max_prefix_len is None:
        max_prefix_len = prefix_page_table.shape[1] * P
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o, "o", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    nbytes = cpa_tree_verify_workspace_size(B, N, H_q, H_kv, d, P)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().cpa_tree_verify(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(tree_page_table), tree_page_table.shape[1],
        _ptr(prefix_lens), _ptr(tree_parents), B, N, H_q, H_kv, d, P, num_pages,
        int(max_prefix_len), float(sm_scale), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
        _stream(stream))
    _check("cpa_tree_verify", st)
    if check:
        _check_device("cpa_tree_verify", ws, stream)
    return o, lse


def cpa_tree_pass_b(q, k_pages, v_pages, tree_page_table, tree_parents,
                    sm_scale: Optional[float] = None, o_b=None, lse_b=None, workspace=None,
                    stream=None, check: bool = False):
    """The tree part alone (each node against its ancestor-or-self nodes).  Returns fp32 (o_b, lse_b)."""
    B, N, H_q, H_kv, d, P, num_pages = _tree_shapes(q, k_pages, v_pages, tree_page_table,
                                                     tree_parents)
    if sm_scale is None:
        sm_scale = d ** -0.5
    if o_b is None:
        o_b = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if lse_b is None:
        lse_b = torch.empty(q.shape[0], H_q, dtype=torch.float32, device=q.device)
    _need(o_b, "o_b", torch.float32)
    _need(lse_b, "lse_b", torch.float32)
    ws = _workspace(cpa_status_workspace_size(), q.device, workspace)
    st = lib().cpa_tree_pass_b(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(tree_page_table), tree_page_table.shape[1],
        _ptr(tree_parents), B, N, H_q, H_kv, d, P, num_pages, float(sm_scale), _ptr(o_b),
        _ptr(lse_b), _ptr(ws), ws.numel(), _stream(stream))
    _check("cpa_tree_pass_b", st)
    if check:
        _check_device("cpa_tree_pass_b", ws, stream)
    return o_b, lse_b


# ---------------------------------------------------------------- decode, windowed prefill, page operations
def _want(t, name: str, dtype, ndim: int, dev: int):
    """`_need`, and on device `dev`.  (The calls below are a few microseconds of GPU work at their
    smallest: one pass over what nearly every call gets right, the messages apart.)"""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim
            and t.get_device() == dev and t.is_contiguous()):
        return
    _need(t, name, dtype, ndim)
    raise ValueError(f"{name} is on {t.device}: the call's tensors must be on one device")


def _device(t, name: str, dtype=None) -> int:
    """The device of the call: that of its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


def _shape(t: torch.Tensor, name: str, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _int(x, name: str) -> int:
    """A whole number for the C entry points, whose ints have 32 bits (ctypes would cut it)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits: {x}")
    return x


def _max_len(max_seq_len, columns: int, page_size: int) -> int:
    """max_seq_len, by default all that a table of so many columns holds."""
    if max_seq_len is None:
        return min(columns * page_size, 1 << 30)  # (the longest sequence that the calls take)
    return _int(max_seq_len, "max_seq_len")


def _new(shape, dtype, dev: int, stream):
    """An output that the caller did not give, from PyTorch's allocator on the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


# PyTorch's current stream of a device as an integer (the first without making a Stream of it)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(name: str, args, dev: int, stream, workspace, nbytes, check: bool):
    """Call entry point `name` with `args`, workspace and stream on device `dev`.  Without a
    workspace from the caller each call gets its own (`nbytes()` of it), from PyTorch's
    allocator on the call's stream: calls on several streams, or in several captured graphs,
    then share nothing."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(name, args, dev, stream, workspace, nbytes, check)
    if workspace is None:
        workspace = _new(nbytes(), torch.uint8, dev, stream)
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8
              and workspace.get_device() == dev and workspace.is_contiguous()):
        _need(workspace, "workspace", torch.uint8)
        raise ValueError("workspace is on another device than the call's tensors")
    raw = _current_stream(dev) if stream is None else stream.cuda_stream
    st = getattr(_lib or lib(), name)(*args, workspace.data_ptr(), workspace.numel(), raw)
    if st != 0:
        raise CpaError(name, st)
    if check:
        _check_device(name, workspace, stream)


def cpa_decode_workspace_size(B, H_q, H_kv, head_dim, page_size) -> int:
    return lib().cpa_decode_workspace_size(B, H_q, H_kv, head_dim, page_size)


def _decode(name, q, k_pages, v_pages, scales, page_table, seq_lens, max_seq_len, window, sinks,
            sm_scale, o, lse, workspace, stream, check):
    dev = _device(q, "q", torch.bfloat16)
    kv = torch.uint8 if scales else torch.bfloat16
    _want(q, "q", torch.bfloat16, 3, dev)
    _want(k_pages, "k_pages", kv, 4, dev)
    _want(v_pages, "v_pages", kv, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(seq_lens, "seq_lens", torch.int32, 1, dev)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, P, H_kv, d = k_pages.shape
    B, H_q, dq = q.shape
    rows, stride = page_table.shape
    if dq != d or seq_lens.shape[0] != B or rows != B:
        raise ValueError("inconsistent decode shapes")
    sc = ()
    if scales:
        n = scales[0].numel() if isinstance(scales[0], torch.Tensor) else 0
        for t, nm in zip(scales, ("k_scale", "v_scale")):
            _want(t, nm, torch.float32, t.dim() if isinstance(t, torch.Tensor) else 1, dev)
            if t.numel() != n or n not in (1, H_kv * d):
                raise ValueError("k_scale / v_scale must hold 1 or H_kv * head_dim values each")
        sc = (scales[0].data_ptr(), scales[1].data_ptr(), int(n > 1))
    if o is None:
        o = _new(q.shape, torch.bfloat16, dev, stream)
    if lse is None:
        lse = _new((B, H_q), torch.float32, dev, stream)
    _want(o, "o", torch.bfloat16, 3, dev)
    _want(lse, "lse", torch.float32, 2, dev)
    _shape(o, "o", q.shape)
    _shape(lse, "lse", (B, H_q))
    args = (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), *sc, page_table.data_ptr(),
            stride, seq_lens.data_ptr(), B, H_q, H_kv, d, P, num_pages,
            _max_len(max_seq_len, stride, P), _int(window, "window"), _int(sinks, "sinks"),
            d ** -0.5 if sm_scale is None else float(sm_scale), o.data_ptr(), lse.data_ptr())
    _launch(name, args, dev, stream, workspace,
            lambda: cpa_decode_workspace_size(B, H_q, H_kv, d, P), check)
    return o, lse


def cpa_decode(q, k_pages, v_pages, page_table, seq_lens, max_seq_len: Optional[int] = None,
               window: int = 0, sinks: int = 0, sm_scale: Optional[float] = None, o=None,
               lse=None, workspace=None, stream=None, check: bool = False):
    """Attention of one new token per request.  Returns (o bf16, lse fp32).

    Row b of ``q`` [B, H_q, 128] is the token at position ``seq_lens[b] - 1``; it
    sees every key, or with ``window`` > 0 the last ``window`` (itself among
    them) and the first ``sinks``.
    """
    return _decode("cpa_decode", q, k_pages, v_pages, (), page_table, seq_lens, max_seq_len,
                   window, sinks, sm_scale, o, lse, workspace, stream, check)


def cpa_decode_fp8(q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens,
                   max_seq_len: Optional[int] = None, window: int = 0, sinks: int = 0,
                   sm_scale: Optional[float] = None, o=None, lse=None, workspace=None,
                   stream=None, check: bool = False):
    """cpa_decode over FP8 E4M3 pages (pools and scales as for cpa_cascade_verify_fp8)."""
    return _decode("cpa_decode_fp8", q, k_pages, v_pages, (k_scale, v_scale), page_table,
                   seq_lens, max_seq_len, window, sinks, sm_scale, o, lse, workspace, stream,
                   check)


def cpa_window_prefill_workspace_size(B, T, H_q, H_kv, head_dim, page_size, max_new) -> int:
    return lib().cpa_window_prefill_workspace_size(B, T, H_q, H_kv, head_dim, page_size, max_new)


def cpa_window_prefill(q, k_pages, v_pages, page_table, q_start, seq_lens,
                       max_new: Optional[int] = None, max_seq_len: Optional[int] = None,
                       window: int = 0, sinks: int = 0, sm_scale: Optional[float] = None, o=None,
                       lse=None, workspace=None, stream=None, check: bool = False):
    """Causal prefill of ragged prompt chunks, with a sliding window and sinks.

    Request b has the new tokens ``q_start[b] .. q_start[b+1]-1`` of ``q``
    [T, H_q, 128], the last ones of its ``seq_lens[b]`` tokens.  Returns (o bf16,
    lse fp32); rows that belong to no request are not written.
    """
    dev = _device(q, "q", torch.bfloat16)
    _want(q, "q", torch.bfloat16, 3, dev)
    _want(k_pages, "k_pages", torch.bfloat16, 4, dev)
    _want(v_pages, "v_pages", torch.bfloat16, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(q_start, "q_start", torch.int32, 1, dev)
    _want(seq_lens, "seq_lens", torch.int32, 1, dev)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, P, H_kv, d = k_pages.shape
    T, H_q, dq = q.shape
    B = seq_lens.shape[0]
    rows, stride = page_table.shape
    if dq != d or q_start.shape[0] != B + 1 or rows != B:
        raise ValueError("inconsistent prefill shapes")
    max_new = T if max_new is None else _int(max_new, "max_new")
    if o is None:
        o = _new(q.shape, torch.bfloat16, dev, stream)
    if lse is None:
        lse = _new((T, H_q), torch.float32, dev, stream)
    _want(o, "o", torch.bfloat16, 3, dev)
    _want(lse, "lse", torch.float32, 2, dev)
    _shape(o, "o", q.shape)
    _shape(lse, "lse", (T, H_q))
    args = (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), stride,
            q_start.data_ptr(), seq_lens.data_ptr(), B, T, H_q, H_kv, d, P, num_pages, max_new,
            _max_len(max_seq_len, stride, P), _int(window, "window"), _int(sinks, "sinks"),
            d ** -0.5 if sm_scale is None else float(sm_scale), o.data_ptr(), lse.data_ptr())
    _launch("cpa_window_prefill", args, dev, stream, workspace,
            lambda: cpa_window_prefill_workspace_size(B, T, H_q, H_kv, d, P, max_new), check)
    return o, lse


def cpa_cache_fork_workspace_size(num_pages) -> int:
    return lib().cpa_cache_fork_workspace_size(num_pages)


def cpa_cache_fork(page_table, seq_lens, parents, children, refcounts, page_size: int,
                   copy_src=None, copy_dst=None, workspace=None, stream=None,
                   check: bool = False):
    """Row ``children[i]`` of ``page_table`` becomes a copy of row ``parents[i]``: whole pages
    shared, a partly filled last one replaced by a free page (count 0 in ``refcounts``).

    Returns (copy_src, copy_dst), the page pairs for ``cpa_cache_copy_pages`` (-1, -1 where
    there is none).  ``page_table``, ``seq_lens`` and ``refcounts`` change in place.
    """
    dev = _device(page_table, "page_table", torch.int32)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(seq_lens, "seq_lens", torch.int32, 1, dev)
    _want(parents, "parents", torch.int32, 1, dev)
    _want(children, "children", torch.int32, 1, dev)
    _want(refcounts, "refcounts", torch.int32, 1, dev)
    n_rows, stride = page_table.shape
    n, num_pages = parents.shape[0], refcounts.shape[0]
    _shape(seq_lens, "seq_lens", (n_rows,))
    _shape(children, "children", (n,))
    if copy_src is None:
        copy_src = _new((n,), torch.int32, dev, stream)
    if copy_dst is None:
        copy_dst = _new((n,), torch.int32, dev, stream)
    _want(copy_src, "copy_src", torch.int32, 1, dev)
    _want(copy_dst, "copy_dst", torch.int32, 1, dev)
    _shape(copy_src, "copy_src", (n,))
    _shape(copy_dst, "copy_dst", (n,))
    args = (page_table.data_ptr(), stride, n_rows, seq_lens.data_ptr(), parents.data_ptr(),
            children.data_ptr(), n, refcounts.data_ptr(), _int(page_size, "page_size"), num_pages,
            copy_src.data_ptr(), copy_dst.data_ptr())
    _launch("cpa_cache_fork", args, dev, stream, workspace,
            lambda: cpa_cache_fork_workspace_size(num_pages), check)
    return copy_src, copy_dst


def cpa_cache_free(page_table, rows, first, last, refcounts, workspace=None, stream=None,
                   check: bool = False) -> None:
    """Give back entries ``first[i] .. last[i]-1`` of row ``rows[i]``: the pages' counts are
    lowered and the entries become -1."""
    dev = _device(page_table, "page_table", torch.int32)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(rows, "rows", torch.int32, 1, dev)
    _want(first, "first", torch.int32, 1, dev)
    _want(last, "last", torch.int32, 1, dev)
    _want(refcounts, "refcounts", torch.int32, 1, dev)
    n_rows, stride = page_table.shape
    n = rows.shape[0]
    _shape(first, "first", (n,))
    _shape(last, "last", (n,))
    args = (page_table.data_ptr(), stride, n_rows, rows.data_ptr(), first.data_ptr(),
            last.data_ptr(), n, refcounts.data_ptr(), refcounts.shape[0])
    _launch("cpa_cache_free", args, dev, stream, workspace, lambda: _STATUS_BYTES, check)


def _any_pools(k_pages, v_pages):
    """K and V pools of any element type; returns (device, num_pages, page_size, bytes of a token)."""
    dev = _device(k_pages, "k_pages")
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _want(t, n, k_pages.dtype, 4, dev)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    num_pages, P, H_kv, d = k_pages.shape
    return dev, num_pages, P, H_kv * d * k_pages.element_size()


def cpa_cache_copy_pages(k_pages, v_pages, copy_src, copy_dst, workspace=None, stream=None,
                         check: bool = False) -> None:
    """Page ``copy_dst[i]`` of both pools becomes a copy of page ``copy_src[i]``; pairs of two
    -1 are passed over."""
    dev, num_pages, P, token = _any_pools(k_pages, v_pages)
    _want(copy_src, "copy_src", torch.int32, 1, dev)
    _want(copy_dst, "copy_dst", torch.int32, 1, dev)
    _shape(copy_dst, "copy_dst", copy_src.shape)
    args = (k_pages.data_ptr(), v_pages.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(),
            copy_src.shape[0], num_pages, P * token)
    _launch("cpa_cache_copy_pages", args, dev, stream, workspace, lambda: _STATUS_BYTES, check)


def cpa_cache_compact(k_pages, v_pages, src_page_table, src_pos, n_keep, dst_page_table=None,
                      dst_start=None, src_rows=None, workspace=None, stream=None,
                      check: bool = False) -> None:
    """Move the kept tokens of each request together: position ``src_pos[b, i]`` of row
    ``src_rows[b]`` (default b) of ``src_page_table`` goes to position ``dst_start[b] + i`` of row
    b of ``dst_page_table``, for i < ``n_keep[b]``.  Without ``dst_page_table`` the move is within
    the source row, whose positions ascend."""
    dev, num_pages, P, token = _any_pools(k_pages, v_pages)
    _want(src_page_table, "src_page_table", torch.int32, 2, dev)
    _want(src_pos, "src_pos", torch.int32, 2, dev)
    _want(n_keep, "n_keep", torch.int32, 1, dev)
    _want(dst_start, "dst_start", torch.int32, 1, dev)
    B, max_keep = src_pos.shape
    _shape(n_keep, "n_keep", (B,))
    _shape(dst_start, "dst_start", (B,))
    if src_rows is not None:
        _want(src_rows, "src_rows", torch.int32, 1, dev)
        _shape(src_rows, "src_rows", (B,))
    dst, dst_stride = None, 0
    if dst_page_table is not None:
        _want(dst_page_table, "dst_page_table", torch.int32, 2, dev)
        if dst_page_table.shape[0] != B:
            raise ValueError("dst_page_table must have a row for each request")
        dst, dst_stride = dst_page_table.data_ptr(), dst_page_table.shape[1]
    args = (k_pages.data_ptr(), v_pages.data_ptr(), src_page_table.data_ptr(),
            src_page_table.shape[1], src_page_table.shape[0],
            None if src_rows is None else src_rows.data_ptr(), src_pos.data_ptr(), max_keep,
            n_keep.data_ptr(), dst, dst_stride, dst_start.data_ptr(), B, P, num_pages, token)
    _launch("cpa_cache_compact", args, dev, stream, workspace, lambda: _STATUS_BYTES, check)


def cpa_get_device_status(workspace: torch.Tensor, stream=None) -> tuple[int, int]:
    """(status code, raw device status word) of the last call on `workspace` (synchronises)."""
    word = ctypes.c_uint32(0)
    st = lib().cpa_get_device_status(_ptr(workspace), ctypes.byref(word), _stream(stream))
    return st, word.value


def cpa_noalloc_device_status(stream=None) -> tuple[int, int]:
    """(status code, raw word) of the static scratch of the current device (synchronises)."""
    word = ctypes.c_uint32(0)
    st = lib().cpa_noalloc_device_status(ctypes.byref(word), _stream(stream))
    return st, word.value


def cpa_debug_wait_timeout(workspace: torch.Tensor, limit_us: int, stream=None) -> None:
    st = lib().cpa_debug_wait_timeout(_ptr(workspace), workspace.numel(), int(limit_us),
                                      _stream(stream))
    _check("cpa_debug_wait_timeout", st)


def cpa_plan_partition(total: int, n_ctas: int, cta: int, tile: int):
    """(owner of `tile`, begin, end of `cta`) of the kernels' work partition (host-side)."""
    b = ctypes.c_int64(0)
    e = ctypes.c_int64(0)
    owner = lib().cpa_plan_partition(total, n_ctas, cta, tile, ctypes.byref(b), ctypes.byref(e))
    return owner, b.value, e.value
