// cpa_decode.cu -- attention of one new token per request over the paged cache.
#include <cmath>

#include "cpa_checks.h"
#include "cpa_rows.cuh"

namespace cpa {
namespace {

cpa_status decode_common(const void* q, const void* k_pages, const void* v_pages,
                         const float* k_scale, const float* v_scale, int per_channel, bool fp8,
                         const int32_t* page_table, int pt_stride, const int32_t* seq_lens, int B,
                         int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                         int max_seq_len, int window, int sinks, float sm_scale, void* o,
                         float* lse, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream) {
    if (!q || !k_pages || !v_pages || !page_table || !seq_lens || !o || !lse)
        return CPA_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale)) return CPA_ERR_INVALID_ARG;
    if (B < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv || num_pages < 1 || max_seq_len < 0 ||
        window < 0 || sinks < 0)
        return CPA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o))
        return CPA_ERR_INVALID_ARG;
    if (head_dim != 128 || !page_size_ok(page_size)) return CPA_ERR_UNSUPPORTED;
    if (pt_stride < 1 || pt_stride < ((long long)max_seq_len + page_size - 1) / page_size)
        return CPA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    if ((long long)B * H_q > (1ll << 31) / 128) return CPA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    RowParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.per_channel = per_channel;
    p.table = page_table;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(workspace);
    p.stride = pt_stride;
    p.B = B;
    p.T = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_len = max_seq_len;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    if (cudaMemsetAsync(workspace, 0, 4, stream) != cudaSuccess) return CPA_ERR_CUDA;
    const unsigned blocks = (unsigned)(((long long)B * H_q + 7) / 8);
    if (fp8) rows_kernel<true><<<blocks, 256, 0, stream>>>(p);
    else rows_kernel<false><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_decode_workspace_size(int B, int H_q, int H_kv, int head_dim, int page_size) {
    if (B < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv || head_dim != 128 || !page_size_ok(page_size))
        return 0;
    return kStatusBytes;
}

cpa_status cpa_decode(const void* q, const void* k_pages, const void* v_pages,
                      const int32_t* page_table, int pt_stride, const int32_t* seq_lens, int B,
                      int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                      int max_seq_len, int window, int sinks, float sm_scale, void* o, float* lse,
                      void* workspace, size_t workspace_bytes, cpa_stream_t stream) {
    return decode_common(q, k_pages, v_pages, nullptr, nullptr, 0, false, page_table, pt_stride,
                         seq_lens, B, H_q, H_kv, head_dim, page_size, num_pages, max_seq_len,
                         window, sinks, sm_scale, o, lse, workspace, workspace_bytes,
                         reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_decode_fp8(const void* q, const void* k_pages, const void* v_pages,
                          const float* k_scale, const float* v_scale, int scale_per_channel,
                          const int32_t* page_table, int pt_stride, const int32_t* seq_lens,
                          int B, int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                          int max_seq_len, int window, int sinks, float sm_scale, void* o,
                          float* lse, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream) {
    return decode_common(q, k_pages, v_pages, k_scale, v_scale, scale_per_channel ? 1 : 0, true,
                         page_table, pt_stride, seq_lens, B, H_q, H_kv, head_dim, page_size,
                         num_pages, max_seq_len, window, sinks, sm_scale, o, lse, workspace,
                         workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
