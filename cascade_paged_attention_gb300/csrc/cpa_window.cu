// cpa_window.cu -- prefill of ragged prompt chunks over the paged cache, causal,
// with an optional sliding window and sinks, on the tensor cores (tcgen05).
//
// Unit: two tiles of up to 128 query rows of one request and KV head (a row is a
// (token, head of the group) pair), against the key tiles (128 keys) that any of
// its rows sees: the tiles of the sinks, then those from the first row's window
// to the last row's position.  Tiles between are not visited.
//
// Both query tiles meet each K/V tile while it is in shared memory, and take
// turns on the tensor cores: while one's scores go through the softmax, the
// other's products run.  The order of the products is
//     PV0(i-1) S0(i) PV1(i-1) S1(i)   for key tile i,
// S and its weights P share TMEM (P overwrites the scores that it came from, and
// S(i+1) is issued after PV(i)), so S0, S1, O0 and O1 fill the 512 columns.
//
// The order goes on from a unit into the next, so that the first scores of a unit
// run while the last weights of the one before are still being made.
//
// Warps (12): 0-3 softmax and output of query tile 0, 4-7 of tile 1 (one thread a
// row: its 128 scores in registers, no exchange between threads), 8 loads K, 9
// loads Q and V, 10 issues the products of query tile 0, 11 those of tile 1.  Two
// issuing warps, because a warp that has issued products goes on only when they
// have left its queue: the other one waits for its weights and loads meanwhile,
// and hands the turn on as soon as it has issued (one warp alone left the tensor
// cores idle for 0.3 of the time).
//
// What bounds it: the tensor cores for long chunks (4 H_q d flops a visible
// pair); the chain softmax -> PV -> S -> softmax of one query tile when the
// softmax takes longer than the other tile's products.
//
// 2 x 8192 tokens, 32/8 heads: 650 us causal, 1690 TFLOP/s of visible pairs, 0.89 of
// the measured bf16 rate; 349 us with a window of 2048, 1390 TFLOP/s, where units are
// 17 tiles long and their ends weigh more (the output's stores alone take 15 us of it).
// Of a tile's 2630 cycles the products are 2048 at the nominal rate and about 2500 as
// measured without a softmax: S reads Q and K from shared memory at all that it gives.
//
// Split.  As in decode the key tiles of all units lie end to end and every block
// takes a range of equal cost, so unequal requests, causal triangles and short
// batches over long caches are balanced alike; a unit cut by a range's end is joined
// by a second kernel in the order of its parts.
//
// Values that are not numbers.  A masked key has weight 0, but 0 times a NaN in V
// is a NaN in a matrix product.  A row whose weights are finite and whose result is
// not is therefore done again, key by key over what it sees, by its warp: exact,
// slow (hundreds of times when every row of a call is: the waits of the other warps
// know of it), and never taken by finite caches.  (Slots past a sequence's end may hold
// anything: their V rows are cleared in shared memory.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_host.h"

namespace cpa {
namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 256;       // rows of a unit
constexpr int kKStages = 3, kVStages = 2;
constexpr uint32_t kHalf = 128u * 128u;    // 64 columns of a 128-row tile: 16 KB
constexpr uint32_t kTileBytes = 2 * kHalf; // 128 rows of 256 bytes
constexpr uint32_t kOffQ = 1024;
constexpr uint32_t kOffK = kOffQ + 2 * kTileBytes;
constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
constexpr uint32_t kSmem = kOffV + kVStages * kTileBytes + 1024;  // (aligned up inside)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// What a unit costs besides its tiles, in tiles: its first scores, masked edge
// tiles and output.  Ranges are cut by this cost (equal numbers of tiles alone left
// the median block waiting 10 % of the time for those with many short units).  Where
// there are no more than two tiles a block a unit costs nothing and no block takes more
// than two: such a call lasts as long as its longest chain of tiles (88 tiles 19.3 ->
// 16.7 us, 160 tiles 21.3 -> 19.4, 296 tiles in 64 units 20.1 -> 17.5, 256 in 8 units
// 23.1 -> 23.3; the same rule up to three tiles: 432 tiles 19.5 -> 21.4).
constexpr int kUnitCost = 3;
constexpr int kMinTiles = 2;  // fewest tiles of a block where units have a cost
constexpr float kRescale = 8.0f;  // O is rescaled when a row's maximum grew by more than 2^8
static_assert(kSmem <= 232448, "shared memory of one block");

struct WindowParams {
    CUtensorMap qmap, kmap, vmap;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pages;
    const __nv_bfloat16* v_pages;
    const int32_t* table;
    const int32_t* q_start;
    const int32_t* lens;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    uint32_t* bad;    // [n_cta] what each block found wrong
    int4* desc;       // [n_cta] (first token, tokens, KV head, parts) of the unit that starts
                      // in the block's range and goes on past it; first token -1: none
    float* part_lse;  // [2 n_cta][kRows], log2 units
    float4* part_o;   // [2 n_cta][32 groups of 4 columns][kRows]
    int stride, B, T, H_q, H_kv, G, TSB, lp, boxr, num_pages, max_new, max_len, window, sinks;
    int n_cta;
    float scale_log2;
};

__device__ __forceinline__ float ninf_f() { return __int_as_float(0xff800000); }

// One request: its new tokens and their place; m = 0 where nothing is to be done.
struct Request {
    int t0, m, L;
};
__device__ __forceinline__ Request request_of(const WindowParams& p, int b, uint32_t& bad) {
    Request r;
    const int s0 = __ldg(p.q_start + b), s1 = __ldg(p.q_start + b + 1);
    r.L = __ldg(p.lens + b);
    r.t0 = s0;
    r.m = 0;
    if (s0 < 0 || s1 < s0 || s1 > p.T || r.L < 0 || r.L > p.max_len || s1 - s0 > p.max_new ||
        s1 - s0 > r.L)
        bad |= CPA_DEV_BAD_LENGTH;
    else
        r.m = s1 - s0;
    return r;
}

struct Unit {
    int b, hk, qt;
    int t0, ntok;       // first query token (row of q) and tokens of the unit
    int p0;             // position of the first token
    int L;
    int lo, sink;       // keys [0, sink) and [lo, p0 + ntok) are seen by some row
    int n_sink, w0;     // tiles 0 .. n_sink-1 are key tiles 0 ..; then key tiles w0 ..
    int n_tiles;
};

__device__ __forceinline__ void unit_tiles(const WindowParams& p, const Request& r, int qt, Unit& x) {
    const int TS = 2 * p.TSB;
    x.ntok = min(TS, r.m - qt * TS);
    x.p0 = r.L - r.m + qt * TS;
    x.lo = p.window > 0 && x.p0 + 1 > p.window ? x.p0 + 1 - p.window : 0;
    x.sink = min(p.sinks, x.lo);
    const int st = (x.sink + 127) >> 7, end = (x.p0 + x.ntok + 127) >> 7;
    x.w0 = x.lo >> 7;
    x.n_sink = st;
    if (x.w0 <= st) x.w0 = x.n_sink = 0;  // one run of tiles from 0
    x.n_tiles = x.n_sink + end - x.w0;
}

__device__ __forceinline__ Unit unit_of(const WindowParams& p, const Request& r, int b, int hk,
                                       int qt) {
    Unit x;
    unit_tiles(p, r, qt, x);
    x.b = b;
    x.hk = hk;
    x.qt = qt;
    x.t0 = r.t0 + qt * 2 * p.TSB;
    x.L = r.L;
    return x;
}

__device__ __forceinline__ int key0_of(const Unit& x, int j) {
    return (j < x.n_sink ? j : j - x.n_sink + x.w0) << 7;
}

struct Ctrl {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[kVStages], v_empty[kVStages];
    uint64_t s_full[2], p_full[2][2], o_full[2];  // p_full: weights of keys 0..63, 64..127
    uint64_t turn[2];   // the issuing warps' turns
    uint64_t mma_done;
    volatile uint64_t redo_ns;  // when a row that is done again last began a key tile
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
    uint32_t bad;
    int unit_cost;            // kUnitCost, or 0 where no block takes more than two tiles
    long long t0, left, per;  // this block's range, in tiles of cost
    int b, hk, qt, off;       // where it begins: a unit, and how far into its cost
};
// mbar_wait() of cpa_device.cuh, with a limit that a redo puts off: the rows that are not
// finite are done again key by key while the other warps wait, for as long as their caches
// are, and tell the time with every key tile.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, Ctrl* c) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if (n & 63u) continue;
        if (c->abort_flag) return false;
        const uint64_t since = max(t0, (uint64_t)c->redo_ns);
        if ((int64_t)(globaltimer_ns() - since) > (int64_t)kWaitLimitNs) {
            atomicOr(&c->bad, CPA_DEV_TIMEOUT);
            c->abort_flag = 1u;
            __threadfence_block();
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctrl* c) {
    // (the first look by itself: most waits find the phase complete)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, c));
}

constexpr uint32_t kOffWalk = 384;  // the softmax warps' walkers (before them: sums by warp)
static_assert(sizeof(Ctrl) <= kOffWalk, "control block");

// Cost of one KV head of a request, by a whole warp (r the same in every lane).
__device__ __forceinline__ long long head_cost(const WindowParams& p, const Request& r,
                                               int unit_cost) {
    const int TS = 2 * p.TSB, lane = threadIdx.x & 31;
    const int nq = (r.m + TS - 1) / TS;
    long long sum = 0;
    for (int qt = lane; qt < nq; qt += 32) {
        Unit x;
        unit_tiles(p, r, qt, x);
        sum += x.n_tiles + unit_cost;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The tiles of one KV head for a request per lane: short ones by their lane, long ones
// by the warp.
__device__ __forceinline__ long long lane_tiles(const WindowParams& p, const Request& r) {
    const int TS = 2 * p.TSB, lane = threadIdx.x & 31;
    const int nq = (r.m + TS - 1) / TS;
    long long sum = 0;
    for (int qt = 0; qt < nq && nq <= 8; ++qt) {
        Unit x;
        unit_tiles(p, r, qt, x);
        sum += x.n_tiles;
    }
    __syncwarp();
    for (uint32_t many = __ballot_sync(0xffffffffu, nq > 8); many != 0u; many &= many - 1u) {
        const int src = __ffs((int)many) - 1;
        Request q;
        q.t0 = 0;
        q.m = __shfl_sync(0xffffffffu, r.m, src);
        q.L = __shfl_sync(0xffffffffu, r.L, src);
        const long long c = head_cost(p, q, 0);
        if (lane == src) sum = c;
    }
    return sum;
}

// Every thread: the problem's cost, this block's range, and the unit where it
// begins.  Each thread sums a run of requests; one scan over the block follows.
__device__ void schedule(const WindowParams& p, Ctrl* c, long long* sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_thread = (p.B + kThreads - 1) / kThreads, b0 = (int)threadIdx.x * per_thread;
    uint32_t bad = 0;
    long long mine = 0, units = 0;
    for (int i = 0; i < per_thread; ++i) {
        Request r = {0, 0, 0};
        if (b0 + i < p.B) r = request_of(p, b0 + i, bad);
        mine += lane_tiles(p, r) * p.H_kv;
        units += (long long)((r.m + 2 * p.TSB - 1) / (2 * p.TSB)) * p.H_kv;
    }
    if (bad) atomicOr(&c->bad, bad);
    long long incl = mine, incl_units = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        const long long z = __shfl_up_sync(0xffffffffu, incl_units, o);
        if (lane >= o) {
            incl += y;
            incl_units += z;
        }
    }
    if (lane == 31) {
        sums[warp] = incl;
        sums[kWarps + warp] = incl_units;
    }
    __syncthreads();
    long long total = 0, before = incl - mine, total_units = 0, units_before = incl_units - units;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            before += sums[w];
            units_before += sums[kWarps + w];
        }
        total += sums[w];
        total_units += sums[kWarps + w];
    }
    const int unit_cost = total <= 2 * p.n_cta ? 0 : kUnitCost;
    total += unit_cost * total_units;
    before += unit_cost * units_before;
    mine += unit_cost * units;
    long long per = (total + p.n_cta - 1) / p.n_cta;
    if (unit_cost) per = max(per, (long long)(kMinTiles + kUnitCost));
    const long long t0 = per * blockIdx.x;
    if (threadIdx.x == 0) {
        c->per = per;
        c->unit_cost = unit_cost;
        c->t0 = t0;
        c->left = t0 < total ? min(per, total - t0) : 0;
    }
    // the warp whose requests hold position t0 looks through them
    const uint32_t here = __ballot_sync(0xffffffffu, before <= t0 && t0 < before + mine);
    if (here) {
        const int src = __ffs((int)here) - 1;
        long long run = __shfl_sync(0xffffffffu, before, src);
        for (int b = __shfl_sync(0xffffffffu, b0, src);; ++b) {
            const Request r = request_of(p, b, bad);
            const long long per_head = head_cost(p, r, unit_cost);
            if (t0 >= run + per_head * p.H_kv) {
                run += per_head * p.H_kv;
                continue;
            }
            // the head, then the query tile
            long long off = t0 - run;
            const int hk = (int)(off / per_head);
            off -= hk * per_head;
            const int TS = 2 * p.TSB, nq = (r.m + TS - 1) / TS;
            long long at = 0;
            for (int q0 = 0; q0 < nq && at <= off; q0 += 32) {
                int cost = 0;
                if (q0 + lane < nq) {
                    Unit x;
                    unit_tiles(p, r, q0 + lane, x);
                    cost = x.n_tiles + unit_cost;
                }
                long long in = cost;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += y;
                }
                const long long ex = at + in - cost;
                if (ex <= off && off < ex + cost) {
                    c->b = b;
                    c->hk = hk;
                    c->qt = q0 + lane;
                    c->off = (int)(off - ex);
                }
                at += __shfl_sync(0xffffffffu, in, 31);
            }
            break;
        }
    }
    __syncthreads();
}

// Walks the pieces (unit, tiles [j0, j1)) of this block's range; j0 == j1 past the
// last.  A unit's own cost counts as lying before its first tile.
struct Walker {
    Unit x;
    Request r;       // x's request
    int unit_cost;
    long long left;  // cost of the range after this piece
    int j0, j1;
    __device__ __forceinline__ void cut(int off) {
        const int take = (int)min((long long)x.n_tiles + unit_cost - off, left);
        left -= take;
        j0 = max(0, off - unit_cost);
        j1 = max(0, off + take - unit_cost);  // (0: the range ends before the first tile)
    }
    __device__ __forceinline__ bool more() const { return j0 < j1; }
    __device__ __forceinline__ void init(const WindowParams& p, const Ctrl* c) {
        left = c->left;
        unit_cost = c->unit_cost;
        uint32_t bad = 0;
        r = request_of(p, c->b, bad);
        x = unit_of(p, r, c->b, c->hk, c->qt);
        cut(c->off);
    }
    __device__ __forceinline__ void next(const WindowParams& p) {
        if (left == 0) {
            j0 = j1;
            return;
        }
        int b = x.b, hk = x.hk, qt = x.qt + 1;
        if (qt * 2 * p.TSB >= r.m) {
            qt = 0;
            if (++hk == p.H_kv) {
                hk = 0;
                uint32_t bad = 0;
                do r = request_of(p, ++b, bad);
                while (r.m == 0);  // (cost is left, so a request with tokens is)
            }
        }
        x = unit_of(p, r, b, hk, qt);
        cut(0);
    }
    // query tiles that hold tokens
    __device__ __forceinline__ int tiles_q(const WindowParams& p) const {
        return x.ntok > p.TSB ? 2 : 1;
    }
};

static_assert(kOffWalk + 8 * sizeof(Walker) <= kOffQ, "control block");

// The next piece of a walker in shared memory: one lane walks.
__device__ __forceinline__ void advance(Walker& w, const WindowParams& p) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) w.next(p);
    __syncwarp();
}

// 128 TMEM columns of this warp's lanes, loaded and waited for.
#define W8(i) "=r"(r[i + 0]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
              "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
__device__ __forceinline__ void tmem_ld_x128(uint32_t taddr, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, "
        "[%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : W8(0), W8(8), W8(16), W8(24), W8(32), W8(40), W8(48), W8(56), W8(64), W8(72), W8(80),
          W8(88), W8(96), W8(104), W8(112), W8(120)
        : "r"(taddr)
        : "memory");
}
#undef W8

__device__ __forceinline__ uint32_t bits_below(int n) {
    return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void store32(uint32_t* ptr, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(ptr), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r));
    return r;
}
// The products and commits of cpa_device.cuh, issued by the lane whose `lead` is set.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// One row over tiles [j0, j1) of its unit, by a whole warp, key by key: what the
// row does not see is not touched.  Lane l ends up with dimensions 4 l .. 4 l + 3
// of o (normalised); returns the log-sum-exp in log2 units.
__device__ __forceinline__ float slow_row(const WindowParams& p, Ctrl* c, const Unit& x, int j0,
                                       int j1, size_t qrow, int pos, float (&o)[4]) {
    const int lane = threadIdx.x & 31;
    const uint2 qr = __ldg(reinterpret_cast<const uint2*>(p.q + qrow * 128) + lane);
    const float q0 = __uint_as_float(qr.x << 16), q1 = __uint_as_float(qr.x & 0xFFFF0000u);
    const float q2 = __uint_as_float(qr.y << 16), q3 = __uint_as_float(qr.y & 0xFFFF0000u);
    const int32_t* trow = p.table + (size_t)x.b * p.stride;
    float m = ninf_f(), l = 0.f;
    o[0] = o[1] = o[2] = o[3] = 0.f;
    // four keys at a time, so that their loads and sums overlap
    for (int j = j0; j < j1; ++j) {
        const int key0 = key0_of(x, j), stop = min(key0 + 128, pos + 1);
        if (lane == 0) c->redo_ns = globaltimer_ns();
        for (int k4 = key0; k4 < stop; k4 += 4) {
            float s[4], v[4][4];
            bool on[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int key = k4 + u;
                on[u] = key < stop && (p.window == 0 || key > pos - p.window || key < p.sinks);
                const int pg = on[u] ? __ldg(trow + (key >> p.lp)) : -1;
                on[u] = on[u] && pg >= 0 && pg < p.num_pages;
                uint2 kr = make_uint2(0u, 0u), vr = kr;
                if (on[u]) {
                    const size_t off =
                        ((((size_t)pg << p.lp) + (key & ((1 << p.lp) - 1))) * p.H_kv + x.hk) * 128 +
                        lane * 4;
                    kr = __ldg(reinterpret_cast<const uint2*>(p.k_pages + off));
                    vr = __ldg(reinterpret_cast<const uint2*>(p.v_pages + off));
                }
                s[u] = q0 * __uint_as_float(kr.x << 16) + q1 * __uint_as_float(kr.x & 0xFFFF0000u) +
                       q2 * __uint_as_float(kr.y << 16) + q3 * __uint_as_float(kr.y & 0xFFFF0000u);
                v[u][0] = __uint_as_float(vr.x << 16);
                v[u][1] = __uint_as_float(vr.x & 0xFFFF0000u);
                v[u][2] = __uint_as_float(vr.y << 16);
                v[u][3] = __uint_as_float(vr.y & 0xFFFF0000u);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], d);
            float mn = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s[u] = on[u] ? s[u] * p.scale_log2 : ninf_f();
                mn = fmaxf(mn, s[u]);
            }
            const float r = mn == ninf_f() ? 0.f : mn, f = ex2(m - r);
            l *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (!on[u]) continue;
                const float e = ex2(s[u] - r);
                l += e;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] += e * v[u][i];
            }
            m = mn;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    return l == 0.f ? ninf_f() : m + lg2(l);
}

__global__ void __launch_bounds__(kThreads, 1) window_kernel(const __grid_constant__ WindowParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* const bad_word = &ctrl->bad;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&ctrl->k_full[i], 1);
            mbar_init(&ctrl->k_empty[i], 2);  // the two issuing warps
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&ctrl->v_full[i], 1);
            mbar_init(&ctrl->v_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctrl->q_full[i], 1);
            mbar_init(&ctrl->q_empty[i], 1);
            mbar_init(&ctrl->s_full[i], 1);
            mbar_init(&ctrl->p_full[i][0], 4);  // one arrival per softmax warp
            mbar_init(&ctrl->p_full[i][1], 4);
            mbar_init(&ctrl->o_full[i], 1);
            mbar_init(&ctrl->turn[i], 1);
        }
        mbar_init(&ctrl->mma_done, 2);
        ctrl->redo_ns = 0;
        ctrl->abort_flag = 0;
        ctrl->bad = 0;
        fence_barrier_init();
        prefetch_tmap(&p.qmap);
        prefetch_tmap(&p.kmap);
        prefetch_tmap(&p.vmap);
    }
    if (warp == 11) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
    }
    // V rows that a tile does not load keep what was there: begin with zeros
    for (uint32_t i = threadIdx.x; i < kVStages * kTileBytes / 16; i += kThreads)
        *reinterpret_cast<uint4*>(smem + kOffV + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    schedule(p, ctrl, reinterpret_cast<long long*>(smem + kOffWalk));
    const uint32_t tmem = ctrl->tmem_base;
    int4 desc = make_int4(-1, 0, 0, 0);

    if (ctrl->left > 0) {
        if (warp == 8 || warp == 9) {
            // ============================== loads: warp 8 K, warp 9 Q and V
            const bool is_k = warp == 8;
            const CUtensorMap* map = is_k ? &p.kmap : &p.vmap;
            uint64_t* const full = is_k ? ctrl->k_full : ctrl->v_full;
            uint64_t* const empty = is_k ? ctrl->k_empty : ctrl->v_empty;
            const int n_stages = is_k ? kKStages : kVStages;
            uint8_t* const ring = smem + (is_k ? kOffK : kOffV);
            // Q is read once: its lines leave L2 first (349 -> 347 us).  K and V asked to stay
            // gave 4 us more here, which the kernels after it lost again.
            const uint64_t pol = l2_policy_evict_normal(), pol_q = l2_policy_evict_first();
            const int NB = 128 / p.boxr;
            const uint32_t q_bytes = (uint32_t)(p.G * p.TSB) * 2u * 128u;  // of one query tile
            uint32_t q_loads[2] = {0u, 0u};
            long long g = 0;
            int st = 0;
            uint32_t par = 1;  // parity of the ring's previous round
            bool ok = true;
            Walker w;
            w.init(p, ctrl);
            for (; w.more() && ok; w.next(p)) {
                const Unit& x = w.x;
                const int end = x.p0 + x.ntok;
                const int32_t* trow = p.table + (size_t)x.b * p.stride;
                // lane bi: the page of box bi of a tile, or -1 where no row sees any of it
                auto page_of = [&](int j) -> int {
                    const int pos = key0_of(x, j) + lane * p.boxr;
                    if (lane >= NB || j >= w.j1 || pos >= end ||
                        (pos + p.boxr <= x.lo && pos >= x.sink))
                        return -1;
                    const int pg = __ldg(trow + (pos >> p.lp));
                    if (pg < 0 || pg >= p.num_pages) {
                        atomicOr(bad_word, CPA_DEV_BAD_PAGE);
                        return -1;
                    }
                    return pg;
                };
                int page = page_of(w.j0);
                if (is_k) {
                    // the unit that this block leaves unfinished, for the join
                    if (w.j0 == 0 && w.j1 < x.n_tiles) {
                        // (it ends with this piece, which ends with the range)
                        const long long last = ctrl->t0 + ctrl->left + x.n_tiles - w.j1 - 1;
                        desc = make_int4(x.t0, x.ntok, x.hk,
                                         (int)(last / ctrl->per - blockIdx.x) + 1);
                    }
                } else {
                    const int nq = w.tiles_q(p);
                    for (int mt = 0; mt < nq && ok; ++mt) {
                        if (q_loads[mt] > 0)
                            ok = wait_warp(&ctrl->q_empty[mt], (q_loads[mt] - 1) & 1u, ctrl);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&ctrl->q_full[mt], q_bytes);
                            for (int h = 0; h < 2; ++h)
                                tma_load_3d(smem + kOffQ + mt * kTileBytes + h * kHalf, &p.qmap, h * 64,
                                            x.hk * p.G, x.t0 + mt * p.TSB, &ctrl->q_full[mt], pol_q);
                        }
                        __syncwarp();
                        ++q_loads[mt];
                    }
                    if (!ok) break;
                }
                for (int j = w.j0; j < w.j1; ++j, ++g) {
                    const int next_page = page_of(j + 1);
                    if (g >= n_stages) {
                        ok = wait_warp(&empty[st], par, ctrl);
                        if (!ok) break;
                    }
                    const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
                    if (lane == 0)
                        mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(mask) * 2u * p.boxr * 128u);
                    __syncwarp();
                    uint8_t* dst = ring + (uint32_t)st * kTileBytes;
                    const int key0 = key0_of(x, j);
                    for (int t0 = 0; t0 < 2 * NB; t0 += 32) {
                        const int t = t0 + lane, bi = (t < 2 * NB ? t : 0) >> 1, h = t & 1;
                        const int pg = __shfl_sync(0xffffffffu, page, bi & 31);
                        if (t < 2 * NB && pg >= 0)
                            tma_load_3d(dst + h * kHalf + bi * p.boxr * 128, map, h * 64, x.hk,
                                        (int)(((uint32_t)pg << p.lp) +
                                              (uint32_t)((key0 + bi * p.boxr) & ((1 << p.lp) - 1))),
                                        &full[st], pol);
                    }
                    page = next_page;
                    if (++st == n_stages) {
                        st = 0;
                        par ^= 1u;
                    }
                    if (!is_k && j == w.j0) {
                        // the next unit's Q into L2: its load is then short
                        Walker y = w;
                        y.next(p);
                        if (y.more() && lane < 2 * y.tiles_q(p))
                            prefetch_3d(&p.qmap, (lane & 1) * 64, y.x.hk * p.G,
                                        y.x.t0 + (lane >> 1) * p.TSB);
                    }
                }
            }
            for (int mt = 0; mt < 2; ++mt)
                if (q_loads[mt] > 0)
                    wait_on(&ctrl->q_full[mt], (q_loads[mt] - 1) & 1u, ctrl);
            // no copy may be in flight when the block leaves
            for (int s = 0; s < n_stages; ++s)
                if (s < g) {
                    const long long last = s + (g - 1 - s) / n_stages * n_stages;
                    wait_on(&full[s], (uint32_t)((last / n_stages) & 1), ctrl);
                }
            __syncwarp();
        } else if (warp >= 10) {
            // ============================== products of query tile mt
            // All lanes run the loop, so that addresses and descriptors stay uniform
            // across the warp; one elected lane's predicate issues.
            const int mt = warp - 10;
            const uint32_t lead = elect_one();
            const uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
            const uint32_t idesc_o = idesc_bf16_f32(128, 128, true);
            const uint64_t q_desc = sdesc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t k_desc = sdesc_sw128(sbase + kOffK, 16, 1024);
            const uint64_t v_desc = sdesc_sw128(sbase + kOffV, kHalf, 1024);
            const uint64_t a_desc = q_desc + mt * (kTileBytes >> 4);
            const uint32_t s_col = tmem + mt * 128u, o_col = tmem + 256u + mt * 128u;
            int ks = 0, vs = 0;  // stage of the tile whose scores / values are next
            uint32_t kpar = 0, vpar = 0, qpar = 0, ppar = 0, tpar = mt == 0 ? 1u : 0u;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t par) {
                ok = ok && wait_warp(bar, par, ctrl);
                return ok;
            };
            // half of PV: 64 keys
            auto issue_pv = [&](int half, bool first) {
                const uint64_t b = v_desc + (uint32_t)vs * (kTileBytes >> 4);
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {
                    const int kk = half * 4 + k4;
                    mma_ts(lead, o_col, s_col + kk * 8u, b + ((kk * 16 * 128) >> 4), idesc_o,
                           first && kk == 0 ? 0u : 1u);
                }
            };
            // what the tile before the current one was
            int nq_prev = 0;
            bool first_prev = false, last_prev = false;
            // A round: PV of the tile before, S of this one (after the last tile there is
            // one more round).  The weights are waited for last, as what comes last; the
            // turn is handed on when all is issued.
            auto round = [&](int nq, bool first, bool last) {
                const bool pv = mt < nq_prev, sc = mt < nq;
                if (pv && !wait(&ctrl->v_full[vs], vpar)) return;
                if (sc && !wait(&ctrl->k_full[ks], kpar)) return;
                if (sc && first) {
                    if (!wait(&ctrl->q_full[mt], qpar)) return;
                    qpar ^= 1u;
                }
                if (!wait(&ctrl->turn[mt], tpar)) return;
                tpar ^= 1u;
                if (pv) {
                    if (!wait(&ctrl->p_full[mt][0], ppar)) return;
                    tc_fence_after_sync();
                    issue_pv(0, first_prev);
                    if (!wait(&ctrl->p_full[mt][1], ppar)) return;
                    ppar ^= 1u;
                    tc_fence_after_sync();
                    issue_pv(1, false);
                    if (last_prev) commit(lead, &ctrl->o_full[mt]);
                    commit(lead, &ctrl->v_empty[vs]);
                } else if (nq_prev && lead) {
                    mbar_arrive(&ctrl->v_empty[vs]);
                }
                if (sc) {
                    tc_fence_after_sync();
                    const uint64_t b = k_desc + (uint32_t)ks * (kTileBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        mma_ss(lead, s_col, a_desc + o, b + o, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    commit(lead, &ctrl->s_full[mt]);
                    if (last) commit(lead, &ctrl->q_empty[mt]);
                    commit(lead, &ctrl->k_empty[ks]);
                } else if (nq && lead) {
                    mbar_arrive(&ctrl->k_empty[ks]);
                }
                if (lead) mbar_arrive(&ctrl->turn[mt ^ 1]);
                __syncwarp();
                if (nq_prev && ++vs == kVStages) {
                    vs = 0;
                    vpar ^= 1u;
                }
                if (nq && ++ks == kKStages) {
                    ks = 0;
                    kpar ^= 1u;
                }
                nq_prev = nq;
                first_prev = first;
                last_prev = last;
            };
            Walker w;
            w.init(p, ctrl);
            for (; w.more() && ok; w.next(p))
                for (int j = w.j0; j < w.j1 && ok; ++j)
                    round(w.tiles_q(p), j == w.j0, j == w.j1 - 1);
            if (ok) round(0, false, false);
            commit(lead, &ctrl->mma_done);
            wait_warp(&ctrl->mma_done, 0, ctrl);
        } else if (warp < 8) {
            // ============================== softmax and output
            const int mt = warp >> 2;
            const int r = (warp & 3) * 32 + lane, R = mt * 128 + r;
            const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_addr = tmem + lane_addr + mt * 128u;
            const uint32_t o_addr = tmem + lane_addr + 256u + mt * 128u;
            const int it = r / p.G, gq = r - it * p.G;
            uint32_t spar = 0, opar = 0;
            long long g = 0;  // key tiles of this block so far (V's ring)
            bool ok = true;
            // the walk of this warp, in shared memory: registers are for the scores
            Walker& w = reinterpret_cast<Walker*>(smem + kOffWalk)[warp];
            if (lane == 0) w.init(p, ctrl);
            __syncwarp();
            while (w.more() && ok) {
                const Unit& xs = w.x;
                if (mt >= w.tiles_q(p)) {
                    g += w.j1 - w.j0;
                    advance(w, p);
                    continue;
                }
                const int tok = mt * p.TSB + it;
                const bool active = it < p.TSB && tok < xs.ntok;
                const int pos = xs.p0 + tok;
                const int jend = w.j1, n_sink = xs.n_sink, skip = xs.w0 - xs.n_sink;
                // positions of this query tile's first and last token
                const int p_min = xs.p0 + mt * p.TSB;
                // keys up to here are hidden from its last token, unless they are sinks
                const int hidden = p.window > 0
                                       ? xs.p0 + min(xs.ntok, (mt + 1) * p.TSB) - 1 - p.window
                                       : -1;
                // tile whose loaded box goes on past the sequence's end
                const int tail = ((xs.p0 + xs.ntok + p.boxr - 1) & ~(p.boxr - 1)) > xs.L ? xs.n_tiles - 1 : -1;
                float m_used = ninf_f(), l = 0.f;
                for (int j = w.j0; j < jend; ++j, ++g) {
                    const int key0 = (j < n_sink ? j : j + skip) << 7;
                    const bool whole =
                        key0 + 127 <= p_min && (key0 > hidden || key0 + 128 <= p.sinks);
                    ok = wait_warp(&ctrl->s_full[mt], spar, ctrl);
                    if (!ok) break;
                    spar ^= 1u;
                    tc_fence_after_sync();
                    uint32_t s[128];
                    tmem_ld_x128(s_addr, s);
                    if (!whole) {
                        // columns [a, z) by position, and those below sk as sinks
                        const int a = p.window > 0 ? pos + 1 - p.window - key0 : 0;
                        const int z = pos + 1 - key0, sk = min(p.sinks - key0, z);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            const uint32_t bits =
                                (bits_below(z - 32 * q4) & ~bits_below(a - 32 * q4)) |
                                bits_below(sk - 32 * q4);
                            // (most groups of an edge tile are whole for the whole warp)
                            if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(bits >> c & 1u)) s[32 * q4 + c] = 0xff800000u;
                        }
                    }
                    float m4[4] = {ninf_f(), ninf_f(), ninf_f(), ninf_f()};
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        m4[c & 3] = fmax3(m4[c & 3],
                                          fmax3(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1]),
                                                __uint_as_float(s[4 * c + 2])),
                                          __uint_as_float(s[4 * c + 3]));
                    const float tmax =
                        fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
                    // O holds every earlier tile of this unit: PV(j - 1) was issued before
                    // S(j), whose completion s_full told
                    const bool need = active && m_used != ninf_f() && tmax > m_used + kRescale;
                    if (__any_sync(0xffffffffu, need)) {
                        const float f = need ? ex2(m_used - tmax) : 1.f;
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 8) {
                            uint32_t v[8];
                            tmem_ld_x8(o_addr + c0, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                            asm volatile(
                                "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], "
                                "{%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(o_addr + c0),
                                "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                                "r"(v[6]), "r"(v[7])
                                : "memory");
                        }
                        if (need) {
                            l *= f;
                            m_used = tmax;
                        }
                    }
                    if (m_used == ninf_f()) m_used = tmax;
                    const float mref = m_used == ninf_f() ? 0.f : m_used;
                    // slots past the sequence's end in the last loaded box: their V rows are
                    // cleared (by both query tiles, each before its own products)
                    if (j == tail) {
                        const int st = (int)(g % kVStages);
                        ok = wait_warp(&ctrl->v_full[st], (uint32_t)((g / kVStages) & 1), ctrl);
                        if (!ok) break;
                        const int first = xs.L - key0;
                        const int stop = min(128, (first + p.boxr - 1) & ~(p.boxr - 1));
                        uint8_t* vb = smem + kOffV + (uint32_t)st * kTileBytes;
                        for (int i = r; i < 16 * (stop - first); i += 128)
                            *reinterpret_cast<uint4*>(vb + (i & 1) * kHalf + first * 128 + (i >> 1) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    // P = 2^(s * scale - m) in bf16 over the first 64 columns of the scores
                    // (a weight's rounding of 2^-9 is of the size of the output's own; the
                    // sum is of the unrounded weights in 32 bits)
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
                    const float2 nm2 = make_float2(-mref, -mref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 t = __ffma2_rn(
                                make_float2(__uint_as_float(s[32 * q4 + 2 * c]),
                                            __uint_as_float(s[32 * q4 + 2 * c + 1])),
                                sc2, nm2);
                            const float ea = ex2(t.x), eb = ex2(t.y);
                            sum[c & 1] = __fadd2_rn(sum[c & 1], make_float2(ea, eb));
                            pk[c] = pack_bf16x2(ea, eb);
                        }
                        tmem_st_x16_nowait(s_addr + 16u * q4, pk);
                        if (q4 & 1) {  // 64 keys: their products may begin
                            tmem_wait_st();
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ctrl->p_full[mt][q4 >> 1]);
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                }
                if (!ok) break;

                // ---- output: the row, or its part of a unit cut by the block's range.  The
                // walk goes on first, while the last products run.
                const Unit x = w.x;
                const int j0 = w.j0, j1 = w.j1;
                advance(w, p);
                ok = wait_warp(&ctrl->o_full[mt], opar, ctrl);
                if (!ok) break;
                opar ^= 1u;
                tc_fence_after_sync();
                const bool split = j0 > 0 || j1 < x.n_tiles;
                const size_t slot = 2 * (size_t)blockIdx.x + (j0 > 0 ? 0 : 1);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float lse2 = l == 0.f ? ninf_f() : m_used + lg2(l);
                const int row = (x.t0 + (active ? tok : 0)) * p.H_q + x.hk * p.G + (active ? gq : 0);
                // rows of the lane pair, -1 where there is none
                const int row_x = __shfl_xor_sync(0xffffffffu, active ? row : -1, 1);
                const int row_e = lane & 1 ? row_x : (active ? row : -1);
                const int row_o = lane & 1 ? (active ? row : -1) : row_x;
                float check = lse2 == ninf_f() ? 0.f : lse2;
                float4* po = p.part_o + slot * 32 * kRows + R;
                // (Two lanes exchange halves, so that they write 64 bytes of a row together:
                // 355 -> 350 us against 32 bytes of a row by each; 128 or 256 bytes together
                // would give 1 us more before the cost of the exchange.  Through shared memory
                // the whole lines cost as much, and the 32 KB that the third K stage needs.)
#pragma unroll 1
                for (int c0 = 0; c0 < 128; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld_x32(o_addr + c0, v);
                    float f[32];
                    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        f[i] = __uint_as_float(v[i]) * inv;
                        z[i & 3] = fmaf(f[i], 0.f, z[i & 3]);  // NaN once any is not finite
                    }
                    check += (z[0] + z[1]) + (z[2] + z[3]);
                    if (split) {
                        if (active) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                po[(size_t)(c0 / 4 + i) * kRows] =
                                    make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                        }
                    } else {
                        uint32_t w[2][8], x[8];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                w[i][e] = pack_bf16x2(f[16 * i + 2 * e], f[16 * i + 2 * e + 1]);
                        const bool odd = lane & 1;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = __shfl_xor_sync(0xffffffffu, odd ? w[0][e] : w[1][e], 1);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            w[0][e] = odd ? x[e] : w[0][e];
                            w[1][e] = odd ? w[1][e] : x[e];
                        }
                        uint32_t* out = reinterpret_cast<uint32_t*>(p.o) + c0 / 2 + (odd ? 8 : 0);
                        if (row_e >= 0) store32(out + (size_t)row_e * 64, w[0]);
                        if (row_o >= 0) store32(out + (size_t)row_o * 64, w[1]);
                    }
                }
                if (active) {
                    if (split) p.part_lse[slot * kRows + R] = lse2;
                    else p.lse[row] = lse2 == ninf_f() ? lse2 : lse2 * kLn2;
                }
                tc_fence_before_sync();  // O may be written again after this warp's next P
                __syncwarp();
                // (a sum that is not a number comes from a seen score: the row's result is
                // that, in every column)
                uint32_t again =
                    __ballot_sync(0xffffffffu, active && isfinite(l) && !isfinite(check));
                for (; again != 0u; again &= again - 1u) {
                    const int src = __ffs((int)again) - 1;
                    const size_t row_a = (size_t)__shfl_sync(0xffffffffu, row, src);
                    const int pos_a = __shfl_sync(0xffffffffu, pos, src);
                    const int R_a = __shfl_sync(0xffffffffu, R, src);
                    float f[4];
                    const float z = slow_row(p, ctrl, x, j0, j1, row_a, pos_a, f);
                    if (split) {
                        p.part_o[(slot * 32 + lane) * kRows + R_a] = make_float4(f[0], f[1], f[2], f[3]);
                        if (lane == 0) p.part_lse[slot * kRows + R_a] = z;
                    } else {
                        reinterpret_cast<uint2*>(p.o + row_a * 128)[lane] =
                            make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
                        if (lane == 0) p.lse[row_a] = z == ninf_f() ? z : z * kLn2;
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 11) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (warp == 8 && lane == 0) {
        p.desc[blockIdx.x] = desc;
        p.bad[blockIdx.x] = ctrl->bad;
    }
}

// Joins the unit that starts in block c's range and goes on past its end: its
// parts are block c's second slot and the first slots of the blocks after it, in
// that order.  A block does 32 rows (grid.y), a thread 4 columns of a row at a
// time.  The last block, whose range nothing follows, gathers the status word.
__global__ void __launch_bounds__(256) window_join_kernel(const __grid_constant__ WindowParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y > 0) return;
        __shared__ uint32_t all;
        if (threadIdx.x == 0) all = 0;
        __syncthreads();
        uint32_t bad = 0;
        for (int i = threadIdx.x; i < p.n_cta; i += 256) bad |= __ldcg(p.bad + i);
        if (bad) atomicOr(&all, bad);
        __syncthreads();
        if (threadIdx.x == 0) *p.status = all;
        return;
    }
    const int4 d = __ldcg(p.desc + blockIdx.x);
    if (d.x < 0) return;
    const int np = d.w;
    const int R = blockIdx.y * 32 + (threadIdx.x & 31), r = R & 127;
    const int it = r / p.G, gq = r - it * p.G;
    const int tok = (R >> 7) * p.TSB + it;
    if (it >= p.TSB || tok >= d.y) return;
    const size_t row = (size_t)(d.x + tok) * p.H_q + d.z * p.G + gq;
    auto slot = [&](int i) -> size_t { return 2 * ((size_t)blockIdx.x + i) + (i == 0 ? 1 : 0); };
    float m = ninf_f(), sum = 0.f;
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int g0 = threadIdx.x >> 5;  // column groups g0, g0 + 8, g0 + 16, g0 + 24
    for (int i0 = 0; i0 < np; i0 += 4) {  // four parts' loads in flight at a time
        float4 y[4][4];
        float z[4], mx = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const size_t at = slot(min(i0 + i, np - 1));
            z[i] = __ldcg(p.part_lse + at * kRows + R);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[i][k] = __ldcg(p.part_o + (at * 32 + g0 + 8 * k) * kRows + R);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i0 + i < np) mx = fmaxf(mx, z[i]);
        const float ref = mx == ninf_f() ? 0.f : mx, f = ex2(m - ref);
        sum *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            acc[k].x *= f;
            acc[k].y *= f;
            acc[k].z *= f;
            acc[k].w *= f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i0 + i >= np) break;
            const float w = ex2(z[i] - ref);
            sum += w;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k].x += w * y[i][k].x;
                acc[k].y += w * y[i][k].y;
                acc[k].z += w * y[i][k].z;
                acc[k].w += w * y[i][k].w;
            }
        }
        m = mx;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<uint2*>(p.o + row * 128)[g0 + 8 * k] =
            make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                       pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (g0 == 0)
        p.lse[row] = sum == 0.f ? ninf_f() : ((m == ninf_f() ? 0.f : m) + lg2(sum)) * kLn2;
}

struct WindowWs {
    size_t bad, desc, part_lse, part_o, total;
};
WindowWs window_ws(int n_cta) {
    WindowWs w;
    w.bad = kStatusBytes;
    w.desc = align_up(w.bad + (size_t)n_cta * 4, 256);
    w.part_lse = align_up(w.desc + (size_t)n_cta * 16, 256);
    w.part_o = align_up(w.part_lse + (size_t)2 * n_cta * kRows * 4, 256);
    w.total = align_up(w.part_o + (size_t)2 * n_cta * kRows * 128 * 4, 256);
    return w;
}

cudaError_t raise_smem_once() {
    static PerDevice<int> state;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return (cudaError_t)state.run(dev, (int)cudaErrorInvalidDevice, [](int&) {
        return (int)cudaFuncSetAttribute(window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmem);
    });
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_window_prefill_workspace_size(int B, int T, int H_q, int H_kv, int head_dim,
                                         int page_size, int max_new) {
    if (B < 1 || T < 0 || max_new < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv ||
        H_q / H_kv > 128 || head_dim != 128 || !page_size_ok(page_size))
        return 0;
    const int n_sm = sm_count();
    return n_sm <= 0 ? 0 : window_ws(n_sm).total;
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
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned32(o))
        return CPA_ERR_INVALID_ARG;
    if (head_dim != 128 || !page_size_ok(page_size) || H_q / H_kv > 128)
        return CPA_ERR_UNSUPPORTED;
    if (pt_stride < 1 || pt_stride < ((long long)max_seq_len + page_size - 1) / page_size)
        return CPA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    if ((long long)T * H_q > (1ll << 31) / 128) return CPA_ERR_UNSUPPORTED;
    if (max_seq_len > kMaxLength) return CPA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < kStatusBytes) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return cudaMemsetAsync(workspace, 0, 4, s) == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    const WindowWs w = window_ws(n_sm);
    if (workspace_bytes < w.total) return CPA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    WindowParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = static_cast<const __nv_bfloat16*>(k_pages);
    p.v_pages = static_cast<const __nv_bfloat16*>(v_pages);
    p.table = page_table;
    p.q_start = q_start;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.bad = reinterpret_cast<uint32_t*>(ws + w.bad);
    p.desc = reinterpret_cast<int4*>(ws + w.desc);
    p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    p.part_o = reinterpret_cast<float4*>(ws + w.part_o);
    p.stride = pt_stride;
    p.B = B;
    p.T = T;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.G = H_q / H_kv;
    p.TSB = 128 / p.G;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.boxr = page_size < 128 ? page_size : 128;
    p.num_pages = num_pages;
    p.max_new = max_new;
    p.max_len = max_seq_len;
    p.window = window;
    p.sinks = sinks;
    p.n_cta = n_sm;
    p.scale_log2 = sm_scale * kLog2e;
    const uint64_t slots = (uint64_t)num_pages * page_size;
    if (!make_map(&p.qmap, q, H_q, (uint64_t)T, p.G, p.TSB) ||
        !make_map(&p.kmap, k_pages, H_kv, slots, 1, p.boxr) ||
        !make_map(&p.vmap, v_pages, H_kv, slots, 1, p.boxr))
        return CPA_ERR_CUDA;
    if (raise_smem_once() != cudaSuccess) return CPA_ERR_CUDA;
    window_kernel<<<n_sm, kThreads, kSmem, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CPA_ERR_LAUNCH;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_sm, kRows / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_join_kernel, p) == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

}  // extern "C"
