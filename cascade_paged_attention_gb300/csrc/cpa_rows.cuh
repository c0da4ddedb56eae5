// cpa_rows.cuh -- attention of one row at a time: a warp per (query token, query
// head), the visible keys in ascending order, a warp-level online softmax.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpa_device.cuh"

namespace cpa {

struct RowParams {
    const __nv_bfloat16* q;
    const void* k_pages;
    const void* v_pages;
    const float* k_scale;  // FP8 pools
    const float* v_scale;
    int per_channel;
    const int32_t* table;
    const int32_t* q_start;  // null: one token per request
    const int32_t* lens;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    int stride, B, T, H_q, H_kv, lp, num_pages, max_new, max_len, window, sinks;
    float scale_log2;
};

template <bool FP8>
__global__ void __launch_bounds__(256) rows_kernel(RowParams p) {
    const float ninf = __int_as_float(0xff800000);
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (id >= (long long)p.T * p.H_q) return;
    const int t = (int)(id / p.H_q), h = (int)(id % p.H_q);
    const int hk = h / (p.H_q / p.H_kv);
    int b = t, m = 1, i = 0;
    if (p.q_start) {
        int a = 0, z = p.B;  // the last request that starts at or before t
        while (z - a > 1) {
            const int mid = (a + z) / 2;
            if (__ldg(p.q_start + mid) <= t) a = mid;
            else z = mid;
        }
        b = a;
        const int s0 = __ldg(p.q_start + b), s1 = __ldg(p.q_start + b + 1);
        if (s0 < 0 || s1 > p.T || s1 < s0) {
            if (lane == 0) atomicOr(p.status, CPA_DEV_BAD_LENGTH);
            return;
        }
        m = s1 - s0;
        i = t - s0;
        if (i < 0 || i >= m) return;  // before the first request or past the last
    }
    const int L = __ldg(p.lens + b);
    const bool bad_len = L < 0 || L > p.max_len || (p.q_start && (m > p.max_new || m > L));
    if (bad_len) {
        if (lane == 0) atomicOr(p.status, CPA_DEV_BAD_LENGTH);
        return;
    }
    const int pos = L - m + i;
    const int lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    const int sink = min(p.sinks, lo);
    float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint2 qr = __ldg(reinterpret_cast<const uint2*>(p.q + id * 128) + lane);
    q[0] = __uint_as_float(qr.x << 16);
    q[1] = __uint_as_float(qr.x & 0xFFFF0000u);
    q[2] = __uint_as_float(qr.y << 16);
    q[3] = __uint_as_float(qr.y & 0xFFFF0000u);
    float vs[4] = {1.f, 1.f, 1.f, 1.f};
    if (FP8)
        for (int c = 0; c < 4; ++c) {
            const int at = p.per_channel ? hk * 128 + lane * 4 + c : 0;
            q[c] *= __ldg(p.k_scale + at);
            vs[c] = __ldg(p.v_scale + at);
        }
    float mx = ninf, l = 0.f;
    const int32_t* trow = p.table + (size_t)b * p.stride;
    for (int j = sink > 0 ? 0 : lo; j <= pos; j = (j + 1 == sink) ? lo : j + 1) {
        const int pg = __ldg(trow + (j >> p.lp));
        if (pg < 0 || pg >= p.num_pages) {
            if (lane == 0) atomicOr(p.status, CPA_DEV_BAD_PAGE);
            continue;
        }
        const size_t off =
            ((((size_t)pg << p.lp) + (j & ((1 << p.lp) - 1))) * p.H_kv + hk) * 128 + lane * 4;
        float k[4], v[4];
        if (FP8) {
            const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(
                static_cast<const uint8_t*>(p.k_pages) + off));
            const uint32_t vw = __ldg(reinterpret_cast<const uint32_t*>(
                static_cast<const uint8_t*>(p.v_pages) + off));
            for (int c = 0; c < 2; ++c) {
                const uint32_t a = e4m3x2_to_f16x2(kw, c), e = e4m3x2_to_f16x2(vw, c);
                const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
                const float2 fe = __half22float2(*reinterpret_cast<const __half2*>(&e));
                k[2 * c] = fa.x;
                k[2 * c + 1] = fa.y;
                v[2 * c] = fe.x;
                v[2 * c + 1] = fe.y;
            }
        } else {
            const uint2 kr = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p.k_pages) + off));
            const uint2 vr = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p.v_pages) + off));
            k[0] = __uint_as_float(kr.x << 16);
            k[1] = __uint_as_float(kr.x & 0xFFFF0000u);
            k[2] = __uint_as_float(kr.y << 16);
            k[3] = __uint_as_float(kr.y & 0xFFFF0000u);
            v[0] = __uint_as_float(vr.x << 16);
            v[1] = __uint_as_float(vr.x & 0xFFFF0000u);
            v[2] = __uint_as_float(vr.y << 16);
            v[3] = __uint_as_float(vr.y & 0xFFFF0000u);
        }
        float dot = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = dot * p.scale_log2;
        const float m_new = fmaxf(mx, x);
        const float c = ex2(mx - m_new), e = ex2(x - m_new);
        l = l * c + e;
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = acc[u] * c + e * v[u];
        mx = m_new;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint2*>(p.o + id * 128)[lane] =
        make_uint2(pack_bf16x2(acc[0] * inv * vs[0], acc[1] * inv * vs[1]),
                   pack_bf16x2(acc[2] * inv * vs[2], acc[3] * inv * vs[3]));
    if (lane == 0) p.lse[id] = l > 0.f ? (mx + lg2(l)) * 0.6931471805599453f : ninf;
}

}  // namespace cpa
