// cpa_decode.cu -- attention of one new token per request over the paged cache,
// bf16 or FP8 E4M3 pages, with an optional sliding window and sinks.
//
// Mathematics.  Per (request, KV head) the G query heads of the group meet the
// same visible keys: s = scale * K q, one pass with a running maximum m and sum
// l per head, o = V^T p / l with p = 2^(s - m).  Keys that the window hides are
// never visited: visible key v is position v for v < n_sink, v + shift after.
//
// What bounds it.  2 G flops a byte of bf16 pages (4 G of FP8): HBM, for any G
// the tensor cores need not be fast for.  So the kernel is built around the
// loads.  The library's verify kernel brings pages by TMA boxes (one head's rows
// of a page: 2 KB) and measured 5.0-5.5 TB/s at that; plain loads into registers
// reach the copy rate over the same pages.  Here every lane loads 32 bytes of a
// row straight into the registers that the warp's mma.sync reads as operands
// (which dimension stands in which place of a fragment is free, as long as Q and
// K, or V and the output, agree), so no byte passes through shared memory.
// mma.sync and not tcgen05: with 8 heads as N = 8 and 16 keys as M = 16 nothing
// is padded for G = 8 and the operands are the loaded registers themselves; the
// 128-row tile of tcgen05 would have to be fed through shared memory or TMEM.
// Whole calls: 64 requests of 2000 tokens (32/8 heads, 525 MB) 85.2 us, 0.91 of the
// measured copy rate; 16 of 1024 to 32768 (64/8 heads, 1.2 GB) 186 us, 0.96; FP8
// pages, 64 of 512 to 8192 (572 MB) 103 us, 0.82.
//
// Split.  The tiles (64 or 128 keys) of all units (request, KV head, up to 8 or
// 16 of its query heads) are laid end to end and cut into equal ranges, one per
// block, so unequal lengths cost nothing; a unit cut by a range's end is joined
// by a second kernel in the order of its parts, which does not depend on which
// block ran first.  That kernel is launched while the first runs
// (programmatic dependent launch) and waits for it on the device.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"

namespace cpa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Fewest tiles of a block.  One request of 777 tokens, 8 KV heads (104 tiles): 9.5 us with 1,
// 8.9 with 2 (half the parts to join), 9.2 with 3, 9.8 with 4; a call with two tiles or more
// for every block does not come to it.
constexpr int kMinTiles = 2;
// O is rescaled when a maximum grew by more than 2^8 (FP8: 2^7, which with the lift leaves f16
// a factor of 4 for maxima so large that subtracting the lift rounds).
constexpr float kRescale = 8.0f, kRescaleFp8 = 7.0f;
// FP8: weights meet V in f16, so they are taken 2^7 times as large: f16 then holds a weight to
// 2^-11 of itself down to 2^-21 of the largest, and to 2^-32 of that below (2^-14 and 2^-25
// without: behind one strong key the flat rest of a long row lost part of its share).
constexpr float kLiftFp8 = 7.0f;
constexpr float kLeast = 1.17549435e-38f;  // 2^-126, the least normal bf16

struct DecodeParams {
    const __nv_bfloat16* q;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* k_scale;  // FP8 pools
    const float* v_scale;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    uint32_t* bad;    // [n_cta] what each block found wrong
    int2* desc;       // [n_cta] unit that starts in block c and goes on past it, and its parts
    float* part_lse;  // [2 n_cta][heads of a unit], log2 units
    float* part_o;    // [2 n_cta][heads of a unit][128]
    int stride, B, H_q, H_kv, G, chunks, lp, num_pages, max_len, window, sinks, n_cta;
    int per_channel;
    int wh;  // KV heads of a unit (the first kernel's WH)
    float scale_log2;
};

template <bool FP8, int NG>
struct Cfg {
    static constexpr int kHeads = 8 * NG;            // query heads of a unit
    static constexpr int kBlocks = FP8 ? 2 : 1;      // 16-key blocks of a warp's step
    static constexpr int kKeys = 16 * kBlocks;       // keys of a warp's step: 8 KB of K and V
    static constexpr int kRowBytes = FP8 ? 128 : 256;
    static constexpr int kKWords = kRowBytes / 16;   // 32-bit words of a K row in one lane
    static constexpr int kVWords = kRowBytes / 32;   // of a V row
    static constexpr int kPerSm = NG == 1 ? 3 : 2;   // resident blocks (by registers)
    static constexpr float kLift = FP8 ? kLiftFp8 : 0.f;
    static constexpr float kGrow = FP8 ? kRescaleFp8 : kRescale;
};

// What a request's token sees: keys [0, n_sink) and [n_sink + shift, L).
struct Seen {
    int n, n_sink, shift;
};
__device__ __forceinline__ Seen seen_of(const DecodeParams& p, int L) {
    Seen s;
    L = L < 0 ? 0 : (L > p.max_len ? p.max_len : L);
    const int lo = p.window > 0 && L > p.window ? L - p.window : 0;
    s.n_sink = min(p.sinks, lo);
    s.shift = lo - s.n_sink;
    s.n = L - s.shift;
    return s;
}

__device__ __forceinline__ void load32(const uint8_t* ptr, uint32_t* r) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "l"(ptr));
}
__device__ __forceinline__ void load16(const uint8_t* ptr, uint32_t* r, uint64_t policy) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.b32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(ptr), "l"(policy));
}

// d += a (16x16) * b (16x8), fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8x8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ninf_f() { return __int_as_float(0xff800000); }

// Exclusive prefix sum over the block's kThreads threads, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long* ws, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    long long base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += ws[w];
        total += ws[w];
    }
    __syncthreads();
    return base + x - v;
}

template <bool FP8, int NG, int WH>
__global__ void __launch_bounds__(kThreads, Cfg<FP8, NG>::kPerSm) decode_kernel(DecodeParams p) {
    using C = Cfg<FP8, NG>;
    constexpr int KB = C::kBlocks, KW = C::kKWords, VW = C::kVWords;
    __shared__ __align__(16) float sm_o[kWarps][C::kHeads][132];  // (read as float4 and uint4)
    __shared__ float sm_m[kWarps][C::kHeads], sm_l[kWarps][C::kHeads];
    __shared__ long long scan[kWarps];
    __shared__ long long s_off;
    __shared__ int s_b;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int wa = warp % WH, wb = warp / WH;          // this warp's head, and its place in the keys
    constexpr int tile = C::kKeys * (kWarps / WH);    // keys of a block's step
    const int U = p.H_kv / WH * p.chunks;             // units of a request
    uint32_t bad = 0;
    const uint64_t once = FP8 ? l2_policy_evict_first() : 0;  // K and V are read once

    // ---- this block's range of tiles
    auto unit_tiles = [&](int b) -> int {
        const int n = seen_of(p, __ldg(p.lens + b)).n;
        return n <= tile ? 1 : (n + tile - 1) / tile;
    };
    // each thread sums a run of requests; one scan over the block follows
    const int per_thread = (p.B + kThreads - 1) / kThreads, b0 = tid * per_thread;
    long long mine = 0, total;
#pragma unroll 4
    for (int i = 0; i < per_thread; ++i)
        if (b0 + i < p.B) {
            const int L = __ldg(p.lens + b0 + i);
            if (L < 0 || L > p.max_len) bad |= CPA_DEV_BAD_LENGTH;
            mine += (long long)U * unit_tiles(b0 + i);
        }
    long long before = block_scan(mine, scan, total);
    long long per = (total + p.n_cta - 1) / p.n_cta;
    if (per < kMinTiles) per = kMinTiles;
    const long long t0 = per * blockIdx.x;
    long long left = t0 < total ? min(per, total - t0) : 0;
    int2 desc = make_int2(-1, 0);
    if (left > 0) {
        if (before <= t0 && t0 < before + mine) {
            int b = b0;
            for (;; ++b) {
                const long long v = (long long)U * unit_tiles(b);
                if (t0 < before + v) break;
                before += v;
            }
            s_b = b;
            s_off = t0 - before;
        }
        __syncthreads();
        int b = s_b;
        int nt = unit_tiles(b);
        int u = (int)(s_off / nt), j = (int)(s_off % nt);

        while (left > 0) {
            const Seen see = seen_of(p, __ldg(p.lens + b));
            nt = unit_tiles(b);
            const int j1 = (int)min((long long)nt, (long long)j + left);
            const int chunk = u % p.chunks, hk = u / p.chunks * WH + wa;
            const int h0 = chunk * C::kHeads;           // first head of the unit in its group
            const int nh = min(C::kHeads, p.G - h0);    // its heads
            const size_t row0 = (size_t)b * p.H_q + (size_t)hk * p.G + h0;
            const int32_t* trow = p.table + (size_t)b * p.stride;
            const size_t row_bytes = (size_t)p.H_kv * C::kRowBytes;
            const uint8_t* kbase = p.k_pages + (size_t)hk * C::kRowBytes + c * 32;
            const uint8_t* vbase = p.v_pages + (size_t)hk * C::kRowBytes + g * (C::kRowBytes / 8);

            // Q: head g (and g + 8) of the unit, the dimensions of this lane's K words
            // (FP8: q x k_scale as two f16 terms, because one alone would leave 2^-12 of
            // every product in the scores; the second waits in this warp's part of sm_o,
            // which is free until the output)
            uint32_t qf[NG][16];
            uint4* q_low = reinterpret_cast<uint4*>(&sm_o[warp][0][0]) + lane;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const bool on = n * 8 + g < nh;
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + (row0 + (on ? n * 8 + g : 0)) * 128);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // bf16: 16 dimensions at 16 c and at 64 + 16 c; FP8: 32 at 32 c
                    const int at = FP8 ? 4 * c + i : (i >> 1) * 8 + 2 * c + (i & 1);
                    const uint4 w = on ? __ldg(src + at) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                    uint32_t low[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t x = ww[e];
                        if (FP8) {
                            const int d = at * 8 + 2 * e + (p.per_channel ? hk * 128 : 0);
                            const float x0 = __uint_as_float(x << 16) *
                                             __ldg(p.k_scale + (p.per_channel ? d : 0));
                            const float x1 = __uint_as_float(x & 0xFFFF0000u) *
                                             __ldg(p.k_scale + (p.per_channel ? d + 1 : 0));
                            const __half2 hi = __floats2half2_rn(x0, x1);
                            x = *reinterpret_cast<const uint32_t*>(&hi);
                            low[e] = pack_f16x2(x0 - __low2float(hi), x1 - __high2float(hi));
                        }
                        qf[n][4 * i + e] = x;
                    }
                    if (FP8) q_low[(n * 4 + i) * 32] = make_uint4(low[0], low[1], low[2], low[3]);
                }
            }

            float of[NG][8][4], m[NG][2], l[NG][2];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) of[n][e][i] = 0.f;
                m[n][0] = m[n][1] = ninf_f();
                l[n][0] = l[n][1] = 0.f;
            }

            // lane l < kKeys follows key l of the warp's step: its table entry one
            // step ahead of its row, its row one step ahead of its products
            const int n_it = j1 - j;
            const int v_base = j * tile + wb * C::kKeys + lane;
            auto entry = [&](int it, int& pos) -> int {
                const int v = v_base + it * tile;
                pos = v < see.n_sink ? v : v + see.shift;
                return (lane < C::kKeys && it < n_it && v < see.n) ? __ldg(trow + (pos >> p.lp))
                                                                  : -1;
            };
            auto to_row = [&](int it, int e, int pos) -> int {
                const int v = v_base + it * tile;
                if (!(lane < C::kKeys && it < n_it && v < see.n)) return -1;
                if (e < 0 || e >= p.num_pages) {
                    bad |= CPA_DEV_BAD_PAGE;
                    return -1;
                }
                return (int)(((uint32_t)e << p.lp) + (uint32_t)(pos & ((1 << p.lp) - 1)));
            };
            uint32_t kr[KB][2][KW], vr[KB][4][VW];
            auto load_k = [&](int row) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = max(0, __shfl_sync(0xffffffffu, row, kb * 16 + i * 8 + g));
                        const uint8_t* src = kbase + (size_t)r * row_bytes;
#pragma unroll
                        for (int w = 0; w < KW; w += 8) load32(src + w * 16, kr[kb][i] + w);
                    }
            };
            auto load_v = [&](int row) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = kb * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
                        const int r = max(0, __shfl_sync(0xffffffffu, row, key));
                        const uint8_t* src = vbase + (size_t)r * row_bytes;
                        if (FP8) load16(src, vr[kb][i], once);
                        else load32(src, vr[kb][i]);
                    }
            };
            int pos;
            int e0 = entry(0, pos);
            int row = to_row(0, e0, pos);
            e0 = entry(1, pos);
            load_k(row);
            load_v(row);
            for (int it = 0; it < n_it; ++it) {
                const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
                const bool whole = there == (C::kKeys == 32 ? 0xffffffffu : 0xffffu);
                // S^T = K Q^T: keys are the rows, heads the columns (FP8: the second
                // terms of Q in sums of their own, because products into one sum wait for
                // one another: 104 -> 102 us)
                float s[KB][NG][4], s_low[KB][NG][4];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[kb][n][i] = s_low[kb][n][i] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        uint32_t a0, a1, a2, a3;
                        if (FP8) {
                            a0 = e4m3x2_to_f16x2(kr[kb][0][ks], false);
                            a1 = e4m3x2_to_f16x2(kr[kb][1][ks], false);
                            a2 = e4m3x2_to_f16x2(kr[kb][0][ks], true);
                            a3 = e4m3x2_to_f16x2(kr[kb][1][ks], true);
                        } else {
                            a0 = kr[kb][0][(2 * ks) % KW];
                            a1 = kr[kb][1][(2 * ks) % KW];
                            a2 = kr[kb][0][(2 * ks + 1) % KW];
                            a3 = kr[kb][1][(2 * ks + 1) % KW];
                        }
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            mma<FP8>(s[kb][n], a0, a1, a2, a3, qf[n][2 * ks], qf[n][2 * ks + 1]);
                            if (FP8) {
                                const uint2 ql = reinterpret_cast<const uint2*>(
                                    q_low + (n * 4 + ks / 2) * 32)[ks & 1];
                                mma<FP8>(s_low[kb][n], a0, a1, a2, a3, ql.x, ql.y);
                            }
                        }
                    }
                }
                // the next step's rows, and its K into the registers just read
                const int row_next = to_row(it + 1, e0, pos);
                e0 = entry(it + 2, pos);
                if (it + 1 < n_it) load_k(row_next);

                bool grow = false;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = s[kb][n][i];
                            if (FP8) x += s_low[kb][n][i];
                            x *= p.scale_log2;
                            if (!whole && !(there >> (kb * 16 + g + (i >> 1) * 8) & 1u)) x = ninf_f();
                            s[kb][n][i] = x;
                            grow |= x > m[n][i & 1] + C::kGrow;
                        }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float mx = m[n][h];
#pragma unroll
                            for (int kb = 0; kb < KB; ++kb)
                                mx = fmaxf(mx, fmaxf(s[kb][n][h], s[kb][n][2 + h]));
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            const float f = m[n][h] == ninf_f() ? 0.f : ex2(m[n][h] - mx);
                            m[n][h] = mx;
                            l[n][h] *= f;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                of[n][e][h] *= f;
                                of[n][e][2 + h] *= f;
                            }
                        }
                }
                // P^T, 16 keys by 8 heads: the weights of a score fragment, packed by
                // pairs of heads and transposed into an operand fragment
                uint32_t ph[KB][NG][2], pl[KB][NG][2];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        const float r0 = m[n][0] == ninf_f() ? 0.f : m[n][0] - C::kLift;
                        const float r1 = m[n][1] == ninf_f() ? 0.f : m[n][1] - C::kLift;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float w0 = ex2(s[kb][n][2 * i] - r0);
                            const float w1 = ex2(s[kb][n][2 * i + 1] - r1);
                            l[n][0] += w0;
                            l[n][1] += w1;
                            if (FP8) {
                                ph[kb][n][i] = transpose8(pack_f16x2(w0, w1));
                            } else {
                                // a weight as two bf16 terms (15 bits): a second pass of
                                // the tensor cores, which have the time, in place of
                                // 2^-8 of every weight.  The first is cut off, not rounded,
                                // and the second is never 0: both then have the weight's
                                // sign, and an infinity in V stays one
                                const uint32_t x0 = __float_as_uint(w0), x1 = __float_as_uint(w1);
                                ph[kb][n][i] = transpose8(__byte_perm(x0, x1, 0x7632u));
                                pl[kb][n][i] = transpose8(pack_bf16x2(
                                    fmaxf(w0 - __uint_as_float(x0 & 0xFFFF0000u), kLeast),
                                    fmaxf(w1 - __uint_as_float(x1 & 0xFFFF0000u), kLeast)));
                            }
                        }
                    }
                if (!whole) {  // what is not there must not meet a weight of 0 as NaN
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(there >> (kb * 16 + 2 * c + (i & 1) + (i >> 1) * 8) & 1u)) {
#pragma unroll
                                for (int w = 0; w < VW; ++w) vr[kb][i][w] = 0u;
                            }
                }
                // O^T += V^T P^T: dimensions are the rows, heads the columns
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t a0, a1, a2, a3;
                        if (FP8) {
                            const uint32_t sel = (e & 1) ? 0x7362u : 0x5140u;
                            const uint32_t x = __byte_perm(vr[kb][0][e >> 1], vr[kb][1][e >> 1], sel);
                            const uint32_t y = __byte_perm(vr[kb][2][e >> 1], vr[kb][3][e >> 1], sel);
                            a0 = e4m3x2_to_f16x2(x, false);
                            a1 = e4m3x2_to_f16x2(x, true);
                            a2 = e4m3x2_to_f16x2(y, false);
                            a3 = e4m3x2_to_f16x2(y, true);
                        } else {
                            a0 = __byte_perm(vr[kb][0][e % VW], vr[kb][1][e % VW], 0x5410u);
                            a1 = __byte_perm(vr[kb][0][e % VW], vr[kb][1][e % VW], 0x7632u);
                            a2 = __byte_perm(vr[kb][2][e % VW], vr[kb][3][e % VW], 0x5410u);
                            a3 = __byte_perm(vr[kb][2][e % VW], vr[kb][3][e % VW], 0x7632u);
                        }
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            mma<FP8>(of[n][e], a0, a1, a2, a3, ph[kb][n][0], ph[kb][n][1]);
                            if (!FP8)
                                mma<FP8>(of[n][e], a0, a1, a2, a3, pl[kb][n][0], pl[kb][n][1]);
                        }
                    }
                if (it + 1 < n_it) load_v(row_next);
                row = row_next;
            }

            // ---- the block's four warps joined
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = l[n][h];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    const int head = n * 8 + 2 * c + h;
                    if (g == 0) {
                        sm_m[warp][head] = m[n][h] - C::kLift;  // what O and the sum refer to
                        sm_l[warp][head] = x;
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        *reinterpret_cast<float4*>(&sm_o[warp][head][g * 16 + 2 * e]) =
                            make_float4(of[n][e][h], of[n][e][2 + h], of[n][e + 1][h],
                                        of[n][e + 1][2 + h]);
                }
            __syncthreads();
            const bool split = j > 0 || j1 < nt;
            const size_t slot = 2 * (size_t)blockIdx.x + (j > 0 ? 0 : 1);
            for (int x = tid; x < WH * C::kHeads * 16; x += kThreads) {
                const int a = x / (C::kHeads * 16), head = (x >> 4) % C::kHeads, d = (x & 15) * 8;
                if (head >= nh) continue;
                const int hka = u / p.chunks * WH + a;
                const size_t row = (size_t)b * p.H_q + (size_t)hka * p.G + h0 + head;
                float mx = ninf_f();
#pragma unroll
                for (int w = a; w < kWarps; w += WH) mx = fmaxf(mx, sm_m[w][head]);
                float sum = 0.f, acc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
                for (int w = a; w < kWarps; w += WH) {
                    const float mw = sm_m[w][head];
                    const float f = mw == ninf_f() ? 0.f : ex2(mw - mx);
                    sum += f * sm_l[w][head];
                    const float4 a = *reinterpret_cast<const float4*>(&sm_o[w][head][d]);
                    const float4 z = *reinterpret_cast<const float4*>(&sm_o[w][head][d + 4]);
                    acc[0] += f * a.x;
                    acc[1] += f * a.y;
                    acc[2] += f * a.z;
                    acc[3] += f * a.w;
                    acc[4] += f * z.x;
                    acc[5] += f * z.y;
                    acc[6] += f * z.z;
                    acc[7] += f * z.w;
                }
                // (a sum of NaN stays NaN; a row that sees nothing has o = 0)
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const float lse2 = sum == 0.f ? ninf_f() : mx + lg2(sum);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] *= inv;
                    if (FP8) acc[i] *= __ldg(p.v_scale + (p.per_channel ? hka * 128 + d + i : 0));
                }
                if (split) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + ((slot * WH + a) * C::kHeads + head) * 128 + d);
                    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    if (d == 0) p.part_lse[(slot * WH + a) * C::kHeads + head] = lse2;
                } else {
                    *reinterpret_cast<uint4*>(p.o + row * 128 + d) =
                        make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                   pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
                    if (d == 0) p.lse[row] = lse2 == ninf_f() ? lse2 : lse2 * kLn2;
                }
            }
            __syncthreads();
            if (j == 0 && j1 < nt) {
                // the unit's first tile is `left` before this block's end; its last is in
                // the block of that tile
                const long long first = t0 + per - left;
                desc = make_int2(b * U + u, (int)((first + nt - 1) / per - blockIdx.x) + 1);
            }
            left -= j1 - j;
            j = 0;
            if (++u == U) {
                u = 0;
                ++b;
            }
        }
    }
    uint32_t all = __syncthreads_or((int)(bad & CPA_DEV_BAD_PAGE)) ? CPA_DEV_BAD_PAGE : 0u;
    if (__syncthreads_or((int)(bad & CPA_DEV_BAD_LENGTH))) all |= CPA_DEV_BAD_LENGTH;
    if (tid == 0) {
        p.desc[blockIdx.x] = desc;
        p.bad[blockIdx.x] = all;
    }
}

// Joins the unit that starts in block c's range and goes on past its end: its
// parts are block c's second slot and the first slots of the blocks after it.
// grid (blocks, heads of a unit / 8), a warp per head, a lane per 4 dimensions.
// The last block, whose range nothing follows, gathers what the first kernel's
// blocks found wrong into the status word, which therefore needs no clearing.
template <int NG>
__global__ void __launch_bounds__(256) join_kernel(DecodeParams p) {
    constexpr int NH = 8 * NG;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y > 0) return;
        uint32_t bad = 0;
        for (int i = threadIdx.x; i < p.n_cta; i += 256) bad |= __ldcg(p.bad + i);
        uint32_t all = __syncthreads_or((int)(bad & CPA_DEV_BAD_PAGE)) ? CPA_DEV_BAD_PAGE : 0u;
        if (__syncthreads_or((int)(bad & CPA_DEV_BAD_LENGTH))) all |= CPA_DEV_BAD_LENGTH;
        if (threadIdx.x == 0) *p.status = all;
        return;
    }
    const int2 desc = __ldcg(p.desc + blockIdx.x);
    if (desc.x < 0) return;
    const int U = p.H_kv / p.wh * p.chunks;
    const int b = desc.x / U, u = desc.x % U, np = desc.y;
    const int h0 = (u % p.chunks) * NH;
    const int lane = threadIdx.x & 31;
    const int x = blockIdx.y * 8 + (threadIdx.x >> 5), nw = p.wh * NH;  // head of the slot
    const int a = x / NH, head = x % NH;
    if (head >= p.G - h0) return;
    // row of part i: block c's second slot for the first, the first slots of the
    // blocks after it for the others
    const size_t base = 2 * (size_t)blockIdx.x;
    auto row_of = [&](int i) -> size_t { return (i ? base + 2 * i : base + 1) * nw + x; };
    float m = ninf_f(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < np; i0 += 8) {  // eight parts' loads in flight at a time
        float4 y[8];
        float z[8], mx = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t at = row_of(min(i0 + i, np - 1));
            y[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * 128) + lane);
            z[i] = __ldcg(p.part_lse + at);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i >= np) z[i] = ninf_f();
            mx = fmaxf(mx, z[i]);
        }
        const float r = mx == ninf_f() ? 0.f : mx, f = ex2(m - r);
        sum *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i >= np) break;
            const float w = ex2(z[i] - r);
            sum += w;
            acc.x += w * y[i].x;
            acc.y += w * y[i].y;
            acc.z += w * y[i].z;
            acc.w += w * y[i].w;
        }
        m = mx;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t row = (size_t)b * p.H_q + (size_t)(u / p.chunks * p.wh + a) * p.G + h0 + head;
    reinterpret_cast<uint2*>(p.o + row * 128)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0)
        p.lse[row] = sum == 0.f ? ninf_f() : ((m == ninf_f() ? 0.f : m) + lg2(sum)) * kLn2;
}

// Groups of up to 8 query heads fill one operand of N = 8; wider ones take two
// at a time, so K and V are read ceil(G / 16) times.
int groups_of(int G) { return G <= 8 ? 1 : 2; }

// KV heads that a block's warps take side by side.  A row of one head is 128 bytes
// in FP8 pages: two heads together read 256 contiguous bytes (109 -> 101 us for 64
// requests of 512 to 8192 tokens; four heads: 102).  In bf16 pages a row is 256 bytes
// by itself, and two heads only mean more parts to join (84.6 -> 85.7 us).
int heads_of(bool fp8, int H_kv) { return fp8 && H_kv % 2 == 0 ? 2 : 1; }

int blocks_of(int G, int n_sm) { return n_sm * (groups_of(G) == 1 ? 3 : 2); }

struct DecodeWs {
    size_t bad, desc, part_lse, part_o, total;
};
DecodeWs decode_ws(int G, int wh, int n_cta) {
    const size_t slots = 2 * (size_t)n_cta * wh * 8 * groups_of(G);
    DecodeWs w;
    w.bad = kStatusBytes;
    w.desc = align_up(w.bad + (size_t)n_cta * 4, 256);
    w.part_lse = align_up(w.desc + (size_t)n_cta * 8, 256);
    w.part_o = align_up(w.part_lse + slots * 4, 256);
    w.total = align_up(w.part_o + slots * 128 * 4, 256);
    return w;
}

template <bool FP8, int NG, int WH>
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
    decode_kernel<FP8, NG, WH><<<p.n_cta, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.n_cta, (unsigned)(p.wh * NG));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_kernel<NG>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

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
    if (!aligned16(q) || !aligned32(k_pages) || !aligned32(v_pages) || !aligned16(o))
        return CPA_ERR_INVALID_ARG;
    if (head_dim != 128 || !page_size_ok(page_size)) return CPA_ERR_UNSUPPORTED;
    if (pt_stride < 1 || pt_stride < ((long long)max_seq_len + page_size - 1) / page_size)
        return CPA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    if ((long long)B * H_q > (1ll << 31) / 128) return CPA_ERR_UNSUPPORTED;
    if (max_seq_len > kMaxLength) return CPA_ERR_UNSUPPORTED;
    if (!workspace) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    const int G = H_q / H_kv;
    const int n_sm = sm_count();
    if (workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (n_sm <= 0) return CPA_ERR_CUDA;
    DecodeParams p = {};
    p.n_cta = blocks_of(G, n_sm);
    p.wh = heads_of(fp8, H_kv);
    const DecodeWs w = decode_ws(G, p.wh, p.n_cta);
    if (workspace_bytes < w.total) return CPA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.bad = reinterpret_cast<uint32_t*>(ws + w.bad);
    p.desc = reinterpret_cast<int2*>(ws + w.desc);
    p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    p.part_o = reinterpret_cast<float*>(ws + w.part_o);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = static_cast<const uint8_t*>(k_pages);
    p.v_pages = static_cast<const uint8_t*>(v_pages);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.per_channel = per_channel;
    p.table = page_table;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.stride = pt_stride;
    p.B = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.G = G;
    p.chunks = (G + 8 * groups_of(G) - 1) / (8 * groups_of(G));
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_len = max_seq_len;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = sm_scale * kLog2e;
    const bool one = groups_of(G) == 1;
    cudaError_t e;
    if (!fp8)
        e = one ? launch_decode<false, 1, 1>(p, stream) : launch_decode<false, 2, 1>(p, stream);
    else if (p.wh == 2)
        e = one ? launch_decode<true, 1, 2>(p, stream) : launch_decode<true, 2, 2>(p, stream);
    else
        e = one ? launch_decode<true, 1, 1>(p, stream) : launch_decode<true, 2, 1>(p, stream);
    return e == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_decode_workspace_size(int B, int H_q, int H_kv, int head_dim, int page_size) {
    if (B < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv || head_dim != 128 || !page_size_ok(page_size))
        return 0;
    const int n_sm = sm_count();
    if (n_sm <= 0) return 0;
    const int G = H_q / H_kv;
    return decode_ws(G, heads_of(true, H_kv), blocks_of(G, n_sm)).total;  // (either call's)
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
