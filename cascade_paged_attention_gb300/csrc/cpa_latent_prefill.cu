// cpa_latent_prefill.cu -- causal prefill of ragged prompt chunks over expanded
// latents: a head's key is its own 128 elements and 64 that all heads share, its
// value 128.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_launch.cuh"
#include "cpa_mma.cuh"

namespace cpa {
namespace {

constexpr int kNope = 128, kRope = 64, kQk = kNope + kRope, kV = 128;

struct ExpandedParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_nope;
    const __nv_bfloat16* k_rope;
    const __nv_bfloat16* v;
    const int32_t* q_start;
    const int32_t* k_start;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    size_t k_token, k_head, r_token, v_token, v_head;  // strides in elements
    int B, T, T_k, H;
    float scale_log2;
};

// One request: its new tokens and its keys; m = 0 where nothing is to be done.
struct Request {
    int t0, m, k0, L;
};
__device__ __forceinline__ Request request_of(const ExpandedParams& p, int b, uint32_t& bad) {
    const int s0 = __ldg(p.q_start + b), s1 = __ldg(p.q_start + b + 1);
    const int k0 = __ldg(p.k_start + b), k1 = __ldg(p.k_start + b + 1);
    Request r = {s0, 0, k0, 0};
    if (s0 < 0 || s1 < s0 || s1 > p.T || k0 < 0 || k1 < k0 || k1 > p.T_k || s1 - s0 > k1 - k0) {
        bad |= CPA_DEV_BAD_LENGTH;
    } else {
        r.m = s1 - s0;
        r.L = k1 - k0;
    }
    return r;
}

// One row against keys [k0, k1) (rows of k and v), by a whole warp, key by key: lane l
// holds elements 2 l, 2 l + 1 of every 64 columns.  Returns the log-sum-exp in log2 units.
__device__ __forceinline__ float expanded_row(const ExpandedParams& p, size_t row, int h, int k0,
                                             int k1, float (&o)[4]) {
    const int lane = threadIdx.x & 31;
    float q[6];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.q + row * kQk) + 32 * i + lane);
        q[2 * i] = __uint_as_float(w << 16);
        q[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
    float m = ninf_f(), l = 0.f;
    o[0] = o[1] = o[2] = o[3] = 0.f;
    for (int key = k0; key < k1; ++key) {
        const uint32_t* kn = reinterpret_cast<const uint32_t*>(p.k_nope + key * p.k_token + h * p.k_head);
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(p.k_rope + key * p.r_token);
        const uint32_t* vr = reinterpret_cast<const uint32_t*>(p.v + key * p.v_token + h * p.v_head);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t w = __ldg((i < 2 ? kn + 32 * i : kr) + lane);
            d += q[2 * i] * __uint_as_float(w << 16) + q[2 * i + 1] * __uint_as_float(w & 0xFFFF0000u);
        }
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
        d *= p.scale_log2;
        const float mn = fmaxf(m, d), r = mn == ninf_f() ? 0.f : mn;
        const float f = ex2(m - r), e = ex2(d - r);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = __ldg(vr + 32 * i + lane);
            o[2 * i] = o[2 * i] * f + e * __uint_as_float(w << 16);
            o[2 * i + 1] = o[2 * i + 1] * f + e * __uint_as_float(w & 0xFFFF0000u);
        }
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    return l == 0.f ? ninf_f() : m + lg2(l);
}

__global__ void __launch_bounds__(256) expanded_rows_kernel(const __grid_constant__ ExpandedParams p) {
    wait_for_clear();
    const int lane = threadIdx.x & 31;
    uint32_t bad = 0;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += 256) request_of(p, b, bad);
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w < (long long)p.T * p.H) {
        const int t = (int)(w / p.H), h = (int)(w % p.H);
        for (int b = 0; b < p.B; ++b) {
            uint32_t none = 0;
            const Request r = request_of(p, b, none);
            if (t < r.t0 || t >= r.t0 + r.m) continue;
            float o[4];
            const float z = expanded_row(p, (size_t)w, h, r.k0, r.k0 + r.L - r.m + (t - r.t0) + 1, o);
            uint32_t* out = reinterpret_cast<uint32_t*>(p.o + (size_t)w * kV);
            out[lane] = pack_bf16x2(o[0], o[1]);
            out[32 + lane] = pack_bf16x2(o[2], o[3]);
            if (lane == 0) p.lse[w] = z == ninf_f() ? z : z * kLn2;
        }
    }
    if (bad) flag(p.status, bad);
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_latent_prefill_workspace_size(int B, int T, int T_k, int H, int nope_dim, int rope_dim,
                                         int v_dim) {
    if (B < 1 || T < 0 || T_k < 0 || H < 1 || nope_dim != kNope || rope_dim != kRope || v_dim != kV)
        return 0;
    return kStatusBytes;
}

cpa_status cpa_latent_prefill(const void* q, const void* k_nope, int64_t k_token_stride,
                              int64_t k_head_stride, const void* k_rope, int64_t rope_token_stride,
                              const void* v, int64_t v_token_stride, int64_t v_head_stride,
                              const int32_t* q_start, const int32_t* k_start, int B, int T, int T_k,
                              int H, int nope_dim, int rope_dim, int v_dim, float sm_scale, void* o,
                              float* lse, void* workspace, size_t workspace_bytes,
                              cpa_stream_t stream) {
    if (!q_start || !k_start || B < 1 || T < 0 || T_k < 0 || H < 1) return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !o || !lse)) return CPA_ERR_INVALID_ARG;
    if (T_k > 0 && (!k_nope || !k_rope || !v)) return CPA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_nope) || !aligned16(k_rope) || !aligned16(v) || !aligned32(o))
        return CPA_ERR_INVALID_ARG;
    if (nope_dim != kNope || rope_dim != kRope || v_dim != kV) return CPA_ERR_UNSUPPORTED;
    if ((long long)T * H > (1ll << 24) || T_k > kMaxLength) return CPA_ERR_UNSUPPORTED;
    if (!strides_ok(k_token_stride, k_head_stride, T_k, H) ||
        !strides_ok(v_token_stride, v_head_stride, T_k, H) ||
        !strides_ok(rope_token_stride, 0, T_k, 1))
        return CPA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return clear_status(workspace, s);
    ExpandedParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_nope = static_cast<const __nv_bfloat16*>(k_nope);
    p.k_rope = static_cast<const __nv_bfloat16*>(k_rope);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_start = q_start;
    p.k_start = k_start;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(workspace);
    p.k_token = (size_t)k_token_stride;
    p.k_head = (size_t)k_head_stride;
    p.r_token = (size_t)rope_token_stride;
    p.v_token = (size_t)v_token_stride;
    p.v_head = (size_t)v_head_stride;
    p.B = B;
    p.T = T;
    p.T_k = T_k;
    p.H = H;
    p.scale_log2 = sm_scale * kLog2e;
    const long long rows = (long long)T * H;
    return launch_cleared(expanded_rows_kernel, dim3((unsigned)((rows + 7) / 8)), 256, s, p.status, p);
}

}  // extern "C"
