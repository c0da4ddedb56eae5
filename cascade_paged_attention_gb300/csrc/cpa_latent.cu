// cpa_latent.cu -- decode over a paged cache of latents, in the absorbed form: every
// head's keys and values come from one vector of 512 + 64 elements a token, all of
// it the key, the first 512 the value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_launch.cuh"

namespace cpa {
namespace {

constexpr int kC = 512, kR = 64, kSlot = kC + kR;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct LatentParams {
    const __nv_bfloat16* q_c;
    const __nv_bfloat16* q_r;
    const __nv_bfloat16* pages;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    size_t qc_token, qc_head, qr_token, qr_head;  // strides in elements
    int stride, B, S, H, lp, num_pages, max_len;
    float scale_log2;
};

__device__ __forceinline__ float ninf_f() { return __int_as_float(0xff800000); }

// One row against keys [k0, k1) of its request, by a whole warp, key by key: lane l
// holds elements 64 i + 2 l, 64 i + 2 l + 1 of every 64 columns i.  Returns the
// log-sum-exp in log2 units.
__device__ __forceinline__ float latent_row(const LatentParams& p, int b, int s, int h, int k0,
                                           int k1, float (&o)[16], uint32_t& bad) {
    const int lane = threadIdx.x & 31;
    float q[18];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const size_t t = (size_t)b * p.S + s;
        const __nv_bfloat16* src = i < 8 ? p.q_c + t * p.qc_token + h * p.qc_head + 64 * i
                                         : p.q_r + t * p.qr_token + h * p.qr_head;
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
        q[2 * i] = __uint_as_float(w << 16);
        q[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
    float m = ninf_f(), l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    for (int key = k0; key < k1; ++key) {
        const int pg = __ldg(p.table + (size_t)b * p.stride + (key >> p.lp));
        if (pg < 0 || pg >= p.num_pages) {
            bad |= CPA_DEV_BAD_PAGE;
            continue;
        }
        const size_t slot = ((size_t)pg << p.lp) + (key & ((1 << p.lp) - 1));
        float x[18], d = 0.f;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const uint32_t w =
                __ldg(reinterpret_cast<const uint32_t*>(p.pages + slot * kSlot) + 32 * i + lane);
            x[2 * i] = __uint_as_float(w << 16);
            x[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
            d += q[2 * i] * x[2 * i] + q[2 * i + 1] * x[2 * i + 1];
        }
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
        d *= p.scale_log2;
        const float mn = fmaxf(m, d), r = mn == ninf_f() ? 0.f : mn;
        const float f = ex2(m - r), e = ex2(d - r);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * x[i];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= inv;
    return l == 0.f ? ninf_f() : m + lg2(l);
}

__global__ void __launch_bounds__(256) latent_rows_kernel(const __grid_constant__ LatentParams p) {
    wait_for_clear();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.B * p.S * p.H) return;
    const int h = (int)(row % p.H), t = (int)(row / p.H), b = t / p.S, s = t % p.S;
    int L = __ldg(p.lens + b);
    uint32_t bad = 0;
    if (L < 0 || L > p.max_len) {
        bad |= CPA_DEV_BAD_LENGTH;
        L = 0;
    }
    float o[16];
    const float z = latent_row(p, b, s, h, 0, L - p.S + 1 + s, o, bad);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint32_t*>(p.o + (size_t)row * kC)[32 * i + lane] =
            pack_bf16x2(o[2 * i], o[2 * i + 1]);
    if (lane == 0) {
        p.lse[row] = z == ninf_f() ? z : z * kLn2;
        if (bad) flag(p.status, bad);
    }
}

bool strides_ok(int64_t token, int64_t head, int tokens, int heads) {
    return (tokens <= 1 || (token > 0 && token % 8 == 0)) &&
           (heads <= 1 || (head > 0 && head % 8 == 0));
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_latent_decode_workspace_size(int B, int S, int H, int latent_dim, int rope_dim,
                                        int page_size) {
    if (B < 1 || S < 1 || H < 1 || latent_dim != kC || rope_dim != kR || !page_size_ok(page_size))
        return 0;
    return kStatusBytes;
}

cpa_status cpa_latent_decode(const void* q_c, int64_t qc_token_stride, int64_t qc_head_stride,
                             const void* q_r, int64_t qr_token_stride, int64_t qr_head_stride,
                             const void* pages, const int32_t* page_table, int pt_stride,
                             const int32_t* seq_lens, int B, int S, int H, int latent_dim,
                             int rope_dim, int page_size, int num_pages, int max_seq_len,
                             float sm_scale, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, cpa_stream_t stream) {
    if (!q_c || !q_r || !pages || !page_table || !seq_lens || !o || !lse) return CPA_ERR_INVALID_ARG;
    if (B < 1 || S < 1 || H < 1 || num_pages < 1 || max_seq_len < 0) return CPA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(q_c) || !aligned16(q_r) || !aligned16(pages) || !aligned32(o))
        return CPA_ERR_INVALID_ARG;
    if (latent_dim != kC || rope_dim != kR || !page_size_ok(page_size)) return CPA_ERR_UNSUPPORTED;
    if (pt_stride < 1 || pt_stride < ((long long)max_seq_len + page_size - 1) / page_size)
        return CPA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > (1ll << 31) || max_seq_len > kMaxLength)
        return CPA_ERR_UNSUPPORTED;
    if ((long long)B * S > (1ll << 22) || (long long)B * S * H > (1ll << 22))
        return CPA_ERR_UNSUPPORTED;
    if (!strides_ok(qc_token_stride, qc_head_stride, B * S, H) ||
        !strides_ok(qr_token_stride, qr_head_stride, B * S, H))
        return CPA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    LatentParams p = {};
    p.q_c = static_cast<const __nv_bfloat16*>(q_c);
    p.q_r = static_cast<const __nv_bfloat16*>(q_r);
    p.pages = static_cast<const __nv_bfloat16*>(pages);
    p.table = page_table;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(workspace);
    p.qc_token = (size_t)qc_token_stride;
    p.qc_head = (size_t)qc_head_stride;
    p.qr_token = (size_t)qr_token_stride;
    p.qr_head = (size_t)qr_head_stride;
    p.stride = pt_stride;
    p.B = B;
    p.S = S;
    p.H = H;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_len = max_seq_len;
    p.scale_log2 = sm_scale * kLog2e;
    const long long rows = (long long)B * S * H;
    return launch_cleared(latent_rows_kernel, dim3((unsigned)((rows + 7) / 8)), 256,
                          reinterpret_cast<cudaStream_t>(stream), p.status, p);
}

}  // extern "C"
