// cpa_window.cu -- prefill of ragged prompt chunks over the paged cache, causal,
// with an optional sliding window and sinks.
#include <cmath>

#include "cpa_checks.h"
#include "cpa_rows.cuh"

using namespace cpa;

extern "C" {

size_t cpa_window_prefill_workspace_size(int B, int T, int H_q, int H_kv, int head_dim,
                                         int page_size, int max_new) {
    if (B < 1 || T < 0 || max_new < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv ||
        H_q / H_kv > 128 || head_dim != 128 || !page_size_ok(page_size))
        return 0;
    return kStatusBytes;
}

cpa_status cpa_window_prefill(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* page_table, int pt_stride, const int32_t* q_start,
                              const int32_t* seq_lens, int B, int T, int H_q, int H_kv,
                              int head_dim, int page_size, int num_pages, int max_new,
                              int max_seq_len, int window, int sinks, float sm_scale, void* o,
                              float* lse, void* workspace, size_t workspace_bytes,
                              cpa_stream_t stream) {
    if (!k_pages || !v_pages || !page_table || !q_start || !seq_lens) return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !o || !lse)) return CPA_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv || num_pages < 1 || max_new < 0 ||
        max_seq_len < 0 || window < 0 || sinks < 0)
        return CPA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o))
        return CPA_ERR_INVALID_ARG;
    if (head_dim != 128 || !page_size_ok(page_size) || H_q / H_kv > 128)
        return CPA_ERR_UNSUPPORTED;
    if (pt_stride < 1 || pt_stride < ((long long)max_seq_len + page_size - 1) / page_size)
        return CPA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    if ((long long)T * H_q > (1ll << 31) / 128) return CPA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(workspace, 0, 4, s) != cudaSuccess) return CPA_ERR_CUDA;
    if (T == 0) return CPA_OK;
    RowParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.table = page_table;
    p.q_start = q_start;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(workspace);
    p.stride = pt_stride;
    p.B = B;
    p.T = T;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_new = max_new;
    p.max_len = max_seq_len;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    rows_kernel<false><<<(unsigned)(((long long)T * H_q + 7) / 8), 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

}  // extern "C"
