// cpa_rows.cu -- rows of new tokens written to the pages of a cache, and rows of a
// cache read back: bf16 as it is, FP8 E4M3 quantised on the way in and widened on
// the way out, latents (two rows of unequal width that share a slot).
//
// A code is e4m3(x / scale), the quotient in 32 bits, rounded to the nearest with
// ties to even, cut at +-448; what is read back is bf16(code * scale), the product
// in 32 bits.
//
// What bounds it: HBM for prompts, where a row is read once and written once (128k tokens of 8 heads
// of 128, bf16: 1.05 GB in 156 us, 0.99 of the copy rate; to FP8 pages 0.79 GB in 134 us, 0.87, from
// them in 120 us, 0.97), latency for the tokens of a decode step (4.4 us).
//
// A warp takes up to 32 tokens and a segment of a row, up to 32 pieces (a piece is eight
// elements: 16 bytes of a row in bf16, 8 codes in an FP8 page).  Its lanes first look up the slots of the
// tokens, one each, all at once; then each moves its piece of one token after the other, several
// of them in flight, so that the scales of its channels stay in registers.  A segment narrower
// than a warp (128 bytes in a latent's row, whose nine are then alike) shares it with the next
// tokens.  There are more blocks than run at a time: the lookups of those that begin hide behind
// the rows of the others.
//
// A lane's registers hold few rows, so a warp first asks the rows that it will read into L2: an
// append before its lookups, which rows need none of.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_launch.cuh"

namespace cpa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
// Tokens in flight a lane, blocks an SM (their registers).  (41k tokens to FP8 pages: 4, 3 49.5 us;
// 4, 4 57.0; 2, 3 58.8; 8, 3 57.8.  74k tokens of FP8 pages to rows: 8, 3 75.9; 8, 4 76.5; 4, 3
// 76.9.  Copies of 41k tokens: 4, 3 55.9; 2, 3 56.7; 8, 3 56.8; 8, 2 58.9.  A loop over runs in as
// many blocks as run at a time: 1.2 to 1.5 times as long.)
constexpr int unroll_of(bool fp8, bool gather) { return fp8 && gather ? 8 : 4; }
// Tokens of a warp in a call with many, by rows side by side in it, and how many of them are asked
// into L2 ahead of their load.  (To FP8 pages 32 and 6 49.5 us, 4 49.1, 8 50.4, 12 53.1, all 61.4,
// none 59.4; 16 and all 56.1; 128k tokens 32 and 6 133.7, 4 134.0, none 164.  From them 16 and all
// 75.9, 32 and 8 77.4, none 83.5.  Copies 8 and all 55.9, 4 57.0, 16 58.0, 32 63.3, none 61.4;
// latents read back 32 and all 17.3, 16 17.9, 8 23.0, none 19.5.)
CPA_HD int tokens_of(bool fp8, bool gather, int sub) {
    const int n = (fp8 ? (gather ? 16 : 32) : 8) * sub;
    return n < 32 ? n : 32;
}
CPA_HD int ahead_of(bool fp8, bool gather, int sub) { return fp8 && !gather ? 6 * sub : 32; }
constexpr int kMinBlocks = 3;
constexpr int kLatentC = 512, kLatentR = 64;  // elements of a latent's two parts

struct RowParams {
    uint8_t* rows[2];       // ragged rows (of new tokens, or the output)
    uint8_t* pages[2];      // the pool, from the first byte that the part has of a slot
    size_t row_bytes[2];    // from one row to the next
    size_t slot_bytes[2];   // from one slot of the pool to the next
    const float* scale[2];
    int pieces[2];          // of a row
    int log_lanes[2];       // lanes that a row takes of a warp (8, 16 or 32)
    int segments[2];
    const int32_t* table;
    const int32_t* start;
    const int32_t* lens;    // of the sequences (append), or first positions (gather; may be null)
    uint32_t* status;
    int stride, B, T, lp, num_pages, per_channel;
    int tokens;             // of a warp
    long long max_len;      // positions that a row of the table holds
    int status_block;       // 1: the first block looks the call over and writes the status word
};

// What a request asks for: its rows [s0, s1) and the position of the first.
struct RowRequest {
    int s0, s1;
    long long pos;
    bool ok;
};
template <bool GATHER>
__device__ __forceinline__ RowRequest row_request(const RowParams& p, int b) {
    RowRequest r;
    r.s0 = __ldg(p.start + b);
    r.s1 = __ldg(p.start + b + 1);
    const long long x = p.lens ? __ldg(p.lens + b) : 0, m = (long long)r.s1 - r.s0;
    r.pos = GATHER ? x : x - m;
    r.ok = r.s0 >= 0 && m >= 0 && r.s1 <= p.T && r.pos >= 0 && r.pos + m <= p.max_len;
    return r;
}

// The slot of token t of a warp's run t0 .. t0 + n - 1 (lane i: token t0 + i), or -1
// where there is nothing to move.  Every lane takes part.
template <bool GATHER>
__device__ __forceinline__ int slot_of_token(const RowParams& p, int t0, int n, uint32_t& bad) {
    const int lane = threadIdx.x & 31;
    // the last request that starts at or before t0: 32 probes at a time
    int lo = 0, hi = p.B;  // it is in [lo, hi)
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) >> 5;
        const int b = lo + lane * step;
        const uint32_t le = __ballot_sync(0xffffffffu, b < hi && __ldg(p.start + b) <= t0);
        const int k = le ? 31 - __clz((int)le) : 0;
        hi = min(hi, lo + (k + 1) * step);
        lo += k * step;
    }
    // each token's request: those of the 32 starts behind lo that are at or before it
    const int t = t0 + lane;
    int b = lo;
    for (int base = lo;; base += 32) {
        const int s = base + 1 + lane < p.B ? __ldg(p.start + base + 1 + lane) : 0x7fffffff;
        int k = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (__shfl_sync(0xffffffffu, s, k + o - 1) <= t) k += o;
        k += __shfl_sync(0xffffffffu, s, k) <= t ? 1 : 0;
        if (b == base) b = base + k;
        if (!__any_sync(0xffffffffu, lane < n && b == base + 32)) break;
    }
    if (lane >= n || b >= p.B) return -1;
    const RowRequest r = row_request<GATHER>(p, b);
    if (!r.ok || t < r.s0 || t >= r.s1) return -1;
    const long long pos = r.pos + (t - r.s0);
    const int pg = __ldg(p.table + (size_t)b * p.stride + (pos >> p.lp));
    if (pg < 0 || pg >= p.num_pages) {
        bad |= CPA_DEV_BAD_PAGE;
        return -1;
    }
    return (int)(((uint32_t)pg << p.lp) + ((uint32_t)pos & ((1u << p.lp) - 1u)));
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A value is quantised by its channel's reciprocal.  The quotient in 32 bits, and x * (1 / scale)
// with its own two roundings, are both within 3 * 2^-24 of x / scale: where the product less and
// more 2^-21 of itself round to one code, that is the quotient's too.  Elsewhere (one value in
// 10^5, and ties of scales of few bits) it is divided.  Scales that are powers of two have exact
// reciprocals and need no margin; one far from 1 is always divided by.  (Every value divided:
// 106 us in place of 79 for 41k tokens.)
struct Reciprocals {
    float inv[8], more;  // the reciprocals less the margin, and the factor to the other side
    bool divide;
    template <class F>
    __device__ __forceinline__ Reciprocals(F scale_of) {
        bool exact = true;
        divide = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = scale_of(i);
            inv[i] = 1.f / s;
            divide |= !(fabsf(s) > 0x1p-100f && fabsf(s) < 0x1p100f);
            exact = exact && fmaf(inv[i], s, -1.f) == 0.f;
        }
        more = exact ? 1.f : 1.f + 0x1p-20f;
#pragma unroll
        for (int i = 0; i < 8; ++i) inv[i] *= exact ? 1.f : 1.f - 0x1p-21f;
    }
};

// Every row of every request that is right, request by request, by one block.  The search above takes
// starts to be ascending; where one is not it may pass over requests that are, and this block moves
// their rows.  (Rows that the search did find get the same bytes twice.)  Slow: one SM copies.
template <bool FP8, bool GATHER>
__device__ __noinline__ uint32_t move_request_by_request(const RowParams& p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t bad = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        RowRequest mine = {0, 0, 0, false};
        if (b0 + lane < p.B) mine = row_request<GATHER>(p, b0 + lane);
        for (uint32_t todo = __ballot_sync(0xffffffffu, mine.ok && mine.s1 > mine.s0); todo; todo &= todo - 1) {
            const int src = __ffs((int)todo) - 1;
            const int s0 = __shfl_sync(0xffffffffu, mine.s0, src), s1 = __shfl_sync(0xffffffffu, mine.s1, src);
            const int first = (int)__shfl_sync(0xffffffffu, mine.pos, src);
            const int32_t* const table = p.table + (size_t)(b0 + src) * p.stride;
            for (int t = s0 + ((warp - src) & (kRowWarps - 1)); t < s1; t += kRowWarps) {
                const int pos = first + (t - s0), pg = __ldg(table + (pos >> p.lp));
                if (pg < 0 || pg >= p.num_pages) {
                    bad |= CPA_DEV_BAD_PAGE;
                    continue;
                }
                const size_t slot = ((size_t)pg << p.lp) + (pos & ((1 << p.lp) - 1));
                for (int part = 0; part < 2; ++part) {
                    for (int piece = lane; piece < p.pieces[part]; piece += 32) {
                        uint4* const row = reinterpret_cast<uint4*>(
                            p.rows[part] + (size_t)t * p.row_bytes[part] + (size_t)piece * 16);
                        uint8_t* const page = p.pages[part] + slot * p.slot_bytes[part] + (size_t)piece * (FP8 ? 8 : 16);
                        if (!FP8) {
                            if (GATHER)
                                *row = *reinterpret_cast<const uint4*>(page);
                            else
                                *reinterpret_cast<uint4*>(page) = *row;
                            continue;
                        }
                        const float* const scale = p.scale[part] + (p.per_channel ? piece * 8 : 0);
                        const int step = p.per_channel ? 1 : 0;
                        if (GATHER) {
                            const uint2 c = *reinterpret_cast<const uint2*>(page);
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t h = e4m3x2_to_f16x2(k < 2 ? c.x : c.y, k & 1);
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                                o[k] = pack_bf16x2(f.x * __ldg(scale + 2 * k * step),
                                                   f.y * __ldg(scale + (2 * k + 1) * step));
                            }
                            *row = make_uint4(o[0], o[1], o[2], o[3]);
                        } else {
                            float f[8];
                            bf16x8_to_f32(*row, f);
                            uint32_t c[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                c[k] = e4m3x2(f[2 * k] / __ldg(scale + 2 * k * step),
                                              f[2 * k + 1] / __ldg(scale + (2 * k + 1) * step));
                            *reinterpret_cast<uint2*>(page) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                        }
                    }
                }
            }
        }
    }
    return bad;
}

// What is wrong with a call, by one block: every request, and every page that it names.
template <bool FP8, bool GATHER>
__device__ void look_over(const RowParams& p) {
    const int lane = threadIdx.x & 31;
    uint32_t bad = 0;
    bool descends = false;
    // up to 32 requests to a warp at a time, fewer so that all warps have some: a request for
    // each lane, then the pages of each by the warp
    const int chunk = min(32, (p.B + kRowWarps - 1) / kRowWarps);
    for (int b0 = (threadIdx.x >> 5) * chunk; b0 < p.B; b0 += kRowWarps * chunk) {
        int first = 0, n = 0;
        if (lane < chunk && b0 + lane < p.B) {
            const RowRequest r = row_request<GATHER>(p, b0 + lane);
            descends |= r.s1 < r.s0;
            if (!r.ok) {
                bad |= CPA_DEV_BAD_LENGTH;
            } else if (r.s1 > r.s0) {
                first = (int)(r.pos >> p.lp);
                n = (int)((r.pos + (r.s1 - r.s0) - 1) >> p.lp) - first + 1;
            }
        }
        auto look = [&](int b, int entry) {
            const int pg = __ldg(p.table + (size_t)b * p.stride + entry);
            if (pg < 0 || pg >= p.num_pages) bad |= CPA_DEV_BAD_PAGE;
        };
        if (n > 0) look(b0 + lane, first);
        __syncwarp();
        for (uint32_t m = __ballot_sync(0xffffffffu, n > 1); m; m &= m - 1) {
            const int src = __ffs((int)m) - 1;
            const int f = __shfl_sync(0xffffffffu, first, src), k = __shfl_sync(0xffffffffu, n, src);
#pragma unroll 4
            for (int e = 1 + lane; e < k; e += 32) look(b0 + src, f + e);
        }
    }
    const bool page = __syncthreads_or((int)(bad & CPA_DEV_BAD_PAGE));
    const bool len = __syncthreads_or((int)(bad & CPA_DEV_BAD_LENGTH));
    if (threadIdx.x == 0)
        *p.status = (page ? CPA_DEV_BAD_PAGE : 0u) | (len ? CPA_DEV_BAD_LENGTH : 0u);
    if (len && __syncthreads_or((int)descends)) move_request_by_request<FP8, GATHER>(p);
}

template <bool FP8, bool GATHER>
__global__ void __launch_bounds__(kRowThreads, kMinBlocks) rows_kernel(const __grid_constant__ RowParams p) {
    constexpr int kUnroll = unroll_of(FP8, GATHER);
    const int lane = threadIdx.x & 31;
    uint32_t bad = 0;
    if (p.status_block && blockIdx.x == 0) {
        look_over<FP8, GATHER>(p);
        return;
    }
    const int block = (int)blockIdx.x - p.status_block;
    const int per_group = p.segments[0] + p.segments[1];
    const long long w = (long long)block * kRowWarps + (threadIdx.x >> 5);
    int seg = (int)(w % per_group);
    const int part = seg >= p.segments[0] ? 1 : 0;
    if (part) seg -= p.segments[0];
    const long long t0 = w / per_group * p.tokens;
    if (!p.status_block) {
        wait_for_clear();
        if (block == 0) {
            bool descends = false;
            for (int b = threadIdx.x; b < p.B; b += kRowThreads) {
                const RowRequest r = row_request<GATHER>(p, b);
                descends |= r.s1 < r.s0;
                if (!r.ok) bad |= CPA_DEV_BAD_LENGTH;
            }
            if (__syncthreads_or((int)descends)) bad |= move_request_by_request<FP8, GATHER>(p);
        }
    }
    if (t0 < p.T) {
        const int log_lanes = p.log_lanes[part], sub = 32 >> log_lanes;
        const int piece = (seg << log_lanes) + (lane & ((1 << log_lanes) - 1)), mine = lane >> log_lanes;
        const bool inside = piece < p.pieces[part];
        const float* const scales = FP8 ? p.scale[part] + (p.per_channel && inside ? piece * 8 : 0) : nullptr;
        auto scale_of = [&](int i) { return FP8 ? __ldg(scales + (p.per_channel ? i : 0)) : 1.f; };
        const Reciprocals r(scale_of);  // (in the kernels that quantise; the others use none of it)
        float scale[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) scale[i] = scale_of(i);
        uint8_t* const rows = p.rows[part] + (size_t)piece * 16;
        uint8_t* const pages = p.pages[part] + (size_t)piece * (FP8 ? 8 : 16);
        const size_t row_bytes = p.row_bytes[part], slot_bytes = p.slot_bytes[part];
        const int n = min(p.tokens, p.T - (int)t0);
        // asks tokens i and on, 32 >> log_lines of them, into L2
        const int width = min(p.pieces[part] - (seg << log_lanes), 1 << log_lanes) * (GATHER && FP8 ? 8 : 16);
        const int log_lines = max(log_lanes - (GATHER && FP8 ? 4 : 3), 0);
        const int line = (lane & ((1 << log_lines) - 1)) * 128;
        const uint8_t* const first = (GATHER ? p.pages[part] : p.rows[part]) +
                                     (size_t)(seg << log_lanes) * (GATHER && FP8 ? 8 : 16) + line;
        auto ask = [&](int i, int end, int slot) {
            i += lane >> log_lines;
            const int at = GATHER ? __shfl_sync(0xffffffffu, slot, i & 31) : 0;
            if (i < end && at >= 0 && line < width)
                prefetch_l2(first + (GATHER ? (size_t)at * slot_bytes : (size_t)(t0 + i) * row_bytes));
        };
        const int asked = 32 >> log_lines, ahead = ahead_of(FP8, GATHER, sub);
        const int begin = min(n, ahead);
        if (!GATHER)
            for (int i = 0; i < begin; i += asked) ask(i, begin, 0);
        const int slot = slot_of_token<GATHER>(p, (int)t0, n, bad);
        if (GATHER)
            for (int i = 0; i < begin; i += asked) ask(i, begin, slot);
        for (int i0 = 0; i0 < n; i0 += sub * kUnroll) {
            if (FP8 && !GATHER) {
                const int end = min(n, i0 + ahead + sub * kUnroll);
                for (int i = i0 + ahead; i < end; i += asked) ask(i, end, 0);
            }
            uint4 x[kUnroll];
            int at[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * sub + mine;
                at[u] = __shfl_sync(0xffffffffu, slot, i & 31);
                if (i >= n || !inside) at[u] = -1;
                if (at[u] < 0) continue;
                const uint8_t* const from =
                    GATHER ? pages + (size_t)at[u] * slot_bytes : rows + (size_t)(t0 + i) * row_bytes;
                if (GATHER && FP8) {
                    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(from));
                    x[u].x = c.x;
                    x[u].y = c.y;
                } else {
                    x[u] = __ldcs(reinterpret_cast<const uint4*>(from));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (at[u] < 0) continue;
                uint4* const row = reinterpret_cast<uint4*>(rows + (size_t)(t0 + i0 + u * sub + mine) * row_bytes);
                uint8_t* const page = pages + (size_t)at[u] * slot_bytes;
                if (GATHER && FP8) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t h = e4m3x2_to_f16x2(k < 2 ? x[u].x : x[u].y, k & 1);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        o[k] = pack_bf16x2(f.x * scale[2 * k], f.y * scale[2 * k + 1]);
                    }
                    *row = make_uint4(o[0], o[1], o[2], o[3]);
                } else if (GATHER) {
                    *row = x[u];
                } else if (FP8) {
                    float f[8];
                    bf16x8_to_f32(x[u], f);
                    uint32_t c[4], differ = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float y0 = f[2 * k] * r.inv[2 * k], y1 = f[2 * k + 1] * r.inv[2 * k + 1];
                        c[k] = e4m3x2(y0, y1);
                        differ |= c[k] ^ e4m3x2(y0 * r.more, y1 * r.more);
                    }
                    if (differ || r.divide)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            c[k] = e4m3x2(f[2 * k] / scale_of(2 * k), f[2 * k + 1] / scale_of(2 * k + 1));
                    *reinterpret_cast<uint2*>(page) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                } else {
                    *reinterpret_cast<uint4*>(page) = x[u];
                }
            }
        }
    }
    if (bad && !p.status_block) flag(p.status, bad);
}

// One part of a row: `bytes` of it in bf16.
void set_part(RowParams& p, int i, const void* rows, size_t row_bytes, void* pages,
              size_t slot_bytes, size_t bytes, const float* scale) {
    p.rows[i] = static_cast<uint8_t*>(const_cast<void*>(rows));
    p.pages[i] = static_cast<uint8_t*>(pages);
    p.row_bytes[i] = row_bytes;
    p.slot_bytes[i] = slot_bytes;
    p.scale[i] = scale;
    p.pieces[i] = (int)(bytes / 16);
    p.log_lanes[i] = p.pieces[i] > 16 ? 5 : p.pieces[i] > 8 ? 4 : 3;
    p.segments[i] = (p.pieces[i] + 31) / 32;
}
// A latent's row: segments of eight pieces in both parts.
void set_latent(RowParams& p, const void* c, size_t c_bytes, const void* r, size_t r_bytes, void* pages) {
    constexpr size_t slot = (kLatentC + kLatentR) * 2;
    set_part(p, 0, c, c_bytes, pages, slot, kLatentC * 2, nullptr);
    set_part(p, 1, r, r_bytes, static_cast<uint8_t*>(pages) + kLatentC * 2, slot, kLatentR * 2, nullptr);
    p.log_lanes[0] = 3;
    p.segments[0] = p.pieces[0] / 8;
}

// Checks that every call shares; parts are set when it returns CPA_OK.
cpa_status rows_ready(RowParams& p, const int32_t* table, int stride, const int32_t* start,
                      const int32_t* lens, int B, int T, int page_size, int num_pages,
                      void* workspace, size_t workspace_bytes) {
    if (!table || !start || B < 1 || T < 0 || num_pages < 1 || stride < 1)
        return CPA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size)) return CPA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > (1ll << 31) || T > kMaxLength)
        return CPA_ERR_UNSUPPORTED;
    const cpa_status st = status_ws(workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    p.table = table;
    p.start = start;
    p.lens = lens;
    p.status = static_cast<uint32_t*>(workspace);
    p.stride = stride;
    p.B = B;
    p.T = T;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_len = (long long)stride * page_size;
    if (p.max_len > kMaxLength) p.max_len = kMaxLength;
    return CPA_OK;
}

template <bool FP8, bool GATHER>
cpa_status launch_rows(RowParams& p, cudaStream_t s) {
    const long long per_group = p.segments[0] + p.segments[1];
    p.tokens = tokens_of(FP8, GATHER, 32 >> p.log_lanes[0]);
    // (a grid has no more blocks than that)
    if ((p.T / p.tokens + 1) * per_group / kRowWarps >= 0x7ffffffe) return CPA_ERR_UNSUPPORTED;
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    // few tokens: fewer to a warp, so that all SMs take part
    while (p.tokens > 4 && p.T / p.tokens * per_group < (long long)n_sm * 16) p.tokens /= 2;
    const long long warps = ((long long)p.T + p.tokens - 1) / p.tokens * per_group;
    const long long blocks = (warps + kRowWarps - 1) / kRowWarps;
    // One block more looks a call over while the others move rows; where it would take longer
    // than they do, every warp reports into a cleared word.
    p.status_block = p.B <= 8192 && (p.T >> p.lp) <= 16384 ? 1 : 0;
    // (a call without rows has one block all the same, for its starts and lengths)
    const dim3 grid((unsigned)(blocks > 0 ? blocks + p.status_block : 1));
    if (!p.status_block)
        return launch_cleared(rows_kernel<FP8, GATHER>, grid, kRowThreads, s, p.status, p);
    rows_kernel<FP8, GATHER><<<grid, kRowThreads, 0, s>>>(p);
    return launched();
}

bool stride_ok(size_t stride, int T) { return T <= 1 || stride % 16 == 0; }

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

cpa_status cpa_cache_append(const void* k_new, const void* v_new, size_t k_stride_bytes,
                            size_t v_stride_bytes, void* k_pages, void* v_pages,
                            const int32_t* page_table, int pt_stride, const int32_t* new_start,
                            const int32_t* seq_lens, int B, int T, int page_size, int num_pages,
                            size_t token_bytes, void* workspace, size_t workspace_bytes,
                            cpa_stream_t stream) {
    if (!k_pages || !v_pages || !seq_lens || token_bytes < 16 || token_bytes % 16)
        return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!k_new || !v_new)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_new) || !aligned16(v_new) ||
        !stride_ok(k_stride_bytes, T) || !stride_ok(v_stride_bytes, T))
        return CPA_ERR_INVALID_ARG;
    if (token_bytes > ((size_t)1 << 20)) return CPA_ERR_UNSUPPORTED;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, new_start, seq_lens, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    set_part(p, 0, k_new, k_stride_bytes, k_pages, token_bytes, token_bytes, nullptr);
    set_part(p, 1, v_new, v_stride_bytes, v_pages, token_bytes, token_bytes, nullptr);
    return launch_rows<false, false>(p, reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_cache_append_fp8(const void* k_new, const void* v_new, size_t k_stride_bytes,
                                size_t v_stride_bytes, void* k_pages, void* v_pages,
                                const float* k_scale, const float* v_scale, int scale_per_channel,
                                const int32_t* page_table, int pt_stride,
                                const int32_t* new_start, const int32_t* seq_lens, int B, int T,
                                int channels, int page_size, int num_pages, void* workspace,
                                size_t workspace_bytes, cpa_stream_t stream) {
    if (!k_pages || !v_pages || !k_scale || !v_scale || !seq_lens || channels < 16 || channels % 16)
        return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!k_new || !v_new)) return CPA_ERR_INVALID_ARG;
    const size_t bytes = (size_t)channels * 2;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_new) || !aligned16(v_new) ||
        !stride_ok(k_stride_bytes, T) || !stride_ok(v_stride_bytes, T))
        return CPA_ERR_INVALID_ARG;
    if (channels > (1 << 19)) return CPA_ERR_UNSUPPORTED;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, new_start, seq_lens, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    p.per_channel = scale_per_channel ? 1 : 0;
    set_part(p, 0, k_new, k_stride_bytes, k_pages, (size_t)channels, bytes, k_scale);
    set_part(p, 1, v_new, v_stride_bytes, v_pages, (size_t)channels, bytes, v_scale);
    return launch_rows<true, false>(p, reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_latent_append(const void* c_new, const void* r_new, size_t c_stride_bytes,
                             size_t r_stride_bytes, void* pages, const int32_t* page_table,
                             int pt_stride, const int32_t* new_start, const int32_t* seq_lens,
                             int B, int T, int latent_dim, int rope_dim, int page_size,
                             int num_pages, void* workspace, size_t workspace_bytes,
                             cpa_stream_t stream) {
    if (!pages || !seq_lens) return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!c_new || !r_new)) return CPA_ERR_INVALID_ARG;
    if (latent_dim != kLatentC || rope_dim != kLatentR) return CPA_ERR_UNSUPPORTED;
    if (!aligned16(pages) || !aligned16(c_new) || !aligned16(r_new) ||
        !stride_ok(c_stride_bytes, T) || !stride_ok(r_stride_bytes, T))
        return CPA_ERR_INVALID_ARG;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, new_start, seq_lens, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    set_latent(p, c_new, c_stride_bytes, r_new, r_stride_bytes, pages);
    return launch_rows<false, false>(p, reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_cache_gather(const void* k_pages, const void* v_pages, const int32_t* page_table,
                            int pt_stride, const int32_t* out_start, const int32_t* first, int B,
                            int T, int page_size, int num_pages, size_t token_bytes, void* k_out,
                            void* v_out, void* workspace, size_t workspace_bytes,
                            cpa_stream_t stream) {
    if (!k_pages || !v_pages || token_bytes < 16 || token_bytes % 16) return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!k_out || !v_out)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out))
        return CPA_ERR_INVALID_ARG;
    if (token_bytes > ((size_t)1 << 20)) return CPA_ERR_UNSUPPORTED;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, out_start, first, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    set_part(p, 0, k_out, token_bytes, const_cast<void*>(k_pages), token_bytes, token_bytes, nullptr);
    set_part(p, 1, v_out, token_bytes, const_cast<void*>(v_pages), token_bytes, token_bytes, nullptr);
    return launch_rows<false, true>(p, reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_cache_gather_fp8(const void* k_pages, const void* v_pages, const float* k_scale,
                                const float* v_scale, int scale_per_channel,
                                const int32_t* page_table, int pt_stride,
                                const int32_t* out_start, const int32_t* first, int B, int T,
                                int channels, int page_size, int num_pages, void* k_out,
                                void* v_out, void* workspace, size_t workspace_bytes,
                                cpa_stream_t stream) {
    if (!k_pages || !v_pages || !k_scale || !v_scale || channels < 16 || channels % 16)
        return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!k_out || !v_out)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out))
        return CPA_ERR_INVALID_ARG;
    if (channels > (1 << 19)) return CPA_ERR_UNSUPPORTED;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, out_start, first, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    p.per_channel = scale_per_channel ? 1 : 0;
    const size_t bytes = (size_t)channels * 2;
    set_part(p, 0, k_out, bytes, const_cast<void*>(k_pages), (size_t)channels, bytes, k_scale);
    set_part(p, 1, v_out, bytes, const_cast<void*>(v_pages), (size_t)channels, bytes, v_scale);
    return launch_rows<true, true>(p, reinterpret_cast<cudaStream_t>(stream));
}

cpa_status cpa_latent_gather(const void* pages, const int32_t* page_table, int pt_stride,
                             const int32_t* out_start, const int32_t* first, int B, int T,
                             int latent_dim, int rope_dim, int page_size, int num_pages,
                             void* c_out, void* r_out, void* workspace, size_t workspace_bytes,
                             cpa_stream_t stream) {
    if (!pages) return CPA_ERR_INVALID_ARG;
    if (T > 0 && (!c_out || !r_out)) return CPA_ERR_INVALID_ARG;
    if (latent_dim != kLatentC || rope_dim != kLatentR) return CPA_ERR_UNSUPPORTED;
    if (!aligned16(pages) || !aligned16(c_out) || !aligned16(r_out)) return CPA_ERR_INVALID_ARG;
    RowParams p = {};
    const cpa_status st = rows_ready(p, page_table, pt_stride, out_start, first, B, T, page_size,
                                     num_pages, workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    set_latent(p, c_out, kLatentC * 2, r_out, kLatentR * 2, const_cast<void*>(pages));
    return launch_rows<false, true>(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
