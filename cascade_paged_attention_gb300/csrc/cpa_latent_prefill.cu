// cpa_latent_prefill.cu -- causal prefill of ragged prompt chunks over expanded
// latents, on the tensor cores (tcgen05): a head's key is its own 128 elements and 64
// that all heads share, its value 128.
//
// The plan is that of cpa_window.cu: a unit is two tiles of 128 query tokens of one request
// and head against the key tiles (128 keys) up to its last token; both query tiles meet each
// K/V tile while it is in shared memory and take turns on the tensor cores, in the order
//     PV0(i-1) S0(i) PV1(i-1) S1(i)   for key tile i;
// P overwrites the scores that it came from, so S0, S1, O0 and O1 fill the 512 columns of
// TMEM; an issuing warp for each query tile; the order goes on from a unit into the next.
//
// What differs: keys of 192 columns make S 1.5 times as long as PV, so that the softmax of one
// query tile (about 1150 cycles) hides behind the other's products (1280 at the nominal rate);
// and Q takes 96 KB of shared memory, which leaves 128 KB.  K and V therefore share one ring
// of eight slots of 16 KB, filled in the order of need: a key tile is three slots of K (128
// keys of 64 columns each, the third the shared part) and two of V (64 keys of 128 columns).
// Each is free as soon as its own products are done.
//
// Who does what.  A call with few units a block is split as in cpa_window.cu: the key tiles of
// all units lie end to end in the order request, head, query tokens, every block takes a range
// of equal cost, and a second kernel joins the units that a range's end cuts.  With heads that
// share no keys that order has every head's K and V in use at a time, more than L2 holds
// (2 x 8192 tokens, 32 heads: 3.8 GB read from DRAM in place of 0.6).  A call with many units
// therefore hands them out whole, a few heads at a time, the longest of these heads first and
// long requests before short ones, so that what is left at the end is short; unless a few long units,
// or a last wave of like ones, would keep some blocks at work for long after the others.  Either
// way the warp that loads K and V finds the units, and the others read them from a ring in shared
// memory.
//
// Values that are not numbers: as in cpa_window.cu.
//
// What bounds it: the tensor cores.  2 x 8192 tokens of 32 heads take 870 to 910 us in a captured
// graph, 1.51 to 1.58 PFLOP/s of products that the mask leaves, 0.80 to 0.84 of the measured rate, and
// 900 to 915 as a program calls it; a round of both query tiles takes 2920 cycles where its products
// need 2560 at the nominal rate (scores read Q and K from shared memory, which the loads write and the
// weights do not leave alone), a unit's end 7600.  Six chunks of 200 to 640 tokens behind contexts: 300
// us, 0.66 (317 and 0.62 as a program calls it), because a request's last unit may hold one query tile:
// it loads 80 KB a key tile for half the products (3800 cycles; with the key tiles shared out to both
// pipelines no fewer).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_host.h"
#include "cpa_mma.cuh"

namespace cpa {
namespace {

constexpr int kNope = 128, kRope = 64, kQk = kNope + kRope, kV = 128;
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 256;  // query tokens of a unit
constexpr int kTile = 128;  // keys of a tile, query tokens of a query tile
constexpr int kSlots = 8;
constexpr uint32_t kSlotBytes = 128u * 128u;
constexpr uint32_t kQBytes = 3 * kSlotBytes;
constexpr uint32_t kOffQ = 1024;
constexpr uint32_t kOffRing = kOffQ + 2 * kQBytes;
constexpr uint32_t kSmem = kOffRing + kSlots * kSlotBytes + 1024;  // (aligned up inside)
// What a unit costs besides its tiles, in tiles; nothing in a call of few tiles, which lasts as
// long as its longest chain of them (448 tiles 24.0 -> 20.5 us, 1300 tiles 31.7 -> 31.0; up to
// twelve tiles a block: 38.2 -> 41.3 for 1400 tiles in 250 units).
constexpr int kUnitCost = 3;
constexpr int kFewTiles = 6;  // of a block
constexpr int kMinTiles = 2;  // fewest tiles of a block where units have a cost
// Units a block from which they may be handed out whole (12 chunks with 5 units a block 533 -> 497
// us, 2 x 2000 tokens with 3 units a block 104 -> 96 us, six chunks with 3 units a block 328 us both):
// the most that q's rows can hold, which the host knows.
constexpr int kWholeUnits = 2;
// They are where that keeps the blocks about as busy as equal ranges do.  Of the units of s tiles and
// more some block has the average number, rounded up, and the call is at least as long as these: a
// fifth more than a range is let pass, since whole units find K and V in L2.  (Whole against ranges,
// and the bound over a range: one chunk of 2560 tokens behind 30000 1200 and 998 us, 1.3; ten of 256 behind 8000
// 360 and 298, 1.4; 32 tokens behind 131072 beside a prompt of 2400 1397 and 459, 4.2; three of 100
// behind 4000 in a buffer of 8192 rows 71 and 67, 1.6.  One chunk of 4096 behind 30000 1676 and 1696,
// 1.1; ten of 512 behind 2000 205 and 213, 1.1; 2 x 2000 tokens 98 and 102, 0.8; six chunks 297 and 324,
// 0.8; 64 tokens behind 20000 beside two prompts of 4000 301 and 326, 1.0.)
constexpr int kEvenPart = 5;  // a fifth
// Whole units are handed out in the order of their requests' lengths, in classes of an eighth of the
// longest.  (Six chunks in the order of the batch 326 us, blocks at work for 327 to 655 thousand
// cycles; so 295, 446 to 559 thousand; with 4 or 16 classes 293 and 297.  12 chunks 491 -> 455 us,
// 16 chunks 906 -> 829.)
constexpr int kClasses = 8;  // (and the lengths of units that the rule above looks at)
constexpr int kMostHeads = 8;       // that are handed out side by side,
constexpr int kSharedKeys = 65536;  // as long as their keys are no more than these (32 MB)
constexpr float kRescale = 8.0f;  // O is rescaled when a row's maximum grew by more than 2^8
static_assert(kSmem <= 232448, "shared memory of one block");

struct ExpandedParams {
    CUtensorMap qmap, kmap, rmap, vmap;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_nope;
    const __nv_bfloat16* k_rope;
    const __nv_bfloat16* v;
    const int32_t* q_start;
    const int32_t* k_start;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    uint32_t* bad;    // [n_cta] what each block found wrong
    int4* desc;       // [n_cta] (first token, tokens, head, parts) of the unit that starts in
                      // the block's range and goes on past it; first token -1: none
    float* part_lse;  // [2 n_cta][kRows], log2 units
    float4* part_o;   // [2 n_cta][32 groups of 4 columns][kRows]
    size_t k_token, k_head, r_token, v_token, v_head;  // strides in elements
    uint32_t* counter;  // units handed out beyond the blocks' first ones
    int B, T, T_k, H, n_cta;
    int may_whole;      // units may be handed out whole
    float scale_log2;
};

// One request: its new tokens and its keys; m = 0 where nothing is to be done.
struct Request {
    int t0, m, k0, L;
};
__device__ __forceinline__ Request request_of(const int32_t* q_start, const int32_t* k_start, int T, int T_k,
                                              int b, uint32_t& bad) {
    const int s0 = __ldg(q_start + b), s1 = __ldg(q_start + b + 1);
    const int k0 = __ldg(k_start + b), k1 = __ldg(k_start + b + 1);
    Request r = {s0, 0, k0, 0};
    if (s0 < 0 || s1 < s0 || s1 > T || k0 < 0 || k1 < k0 || k1 > T_k || s1 - s0 > k1 - k0) {
        bad |= CPA_DEV_BAD_LENGTH;
    } else {
        r.m = s1 - s0;
        r.L = k1 - k0;
    }
    return r;
}
__device__ __forceinline__ Request request_of(const ExpandedParams& p, int b, uint32_t& bad) {
    return request_of(p.q_start, p.k_start, p.T, p.T_k, b, bad);
}
__device__ __forceinline__ int units_of(const Request& r) { return (r.m + kRows - 1) / kRows; }
// Tiles of a request's query tokens qt * kRows and on.
__device__ __forceinline__ int tiles_of(const Request& r, int qt) {
    return (r.L - r.m + min(r.m, (qt + 1) * kRows) + kTile - 1) / kTile;
}

// Units of a request of at least t tiles.
__device__ __forceinline__ int units_at_least(const Request& r, int t) {
    const int need = t * kTile - (kTile - 1) - (r.L - r.m);  // query tokens up to the unit's end
    return r.m < max(need, 1) ? 0 : units_of(r) + 1 - max(1, (need + kRows - 1) / kRows);
}

// The class of a request's length, the highest that of the longest.
__device__ __forceinline__ int class_of(const Request& r, int most) {
    return (tiles_of(r, units_of(r) - 1) * kClasses - 1) / most;
}

// A unit, or the part [j0, j1) of its tiles that a block does; j0 == j1: no more.
struct Piece {
    int t0, ntok;  // rows of q
    int p0;        // position of the first
    int k0, L;     // rows of k and v
    int h, nt, j0, j1;
    __device__ __forceinline__ int tiles_q() const { return ntok > kTile ? 2 : 1; }
};
constexpr int kPieces = 4;   // of the ring: the one that is loaded and the next, two behind
constexpr int kReaders = 11; // warps that read it

struct Ctrl {
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kSlots], empty[kSlots];
    uint64_t s_full[2], p_full[2][2], o_full[2];  // p_full: weights of keys 0..63, 64..127
    uint64_t turn[2];   // the issuing warps' turns
    uint64_t mma_done;
    volatile uint64_t alive_ns;  // the last sign of work that others may wait for (see wait_on)
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
    uint32_t bad;
    int most_tiles;           // of a unit
    int at_least[kClasses];   // units of at least so many eighths of it
    int whole;                // units are handed out whole
    int unit_cost;            // kUnitCost, or 0 where no block takes more than kFewTiles
    long long t0, left, per;  // this block's range, in tiles of cost
    int b, h, qt, off;        // where it begins: a unit, and how far into its cost
    Piece piece[kPieces];
};
// mbar_wait() of cpa_device.cuh, with a limit that signs of work put off: rows that are not
// finite are done again key by key while the other warps wait, and a warp without a part in a
// unit waits until it ends, for as long as the sequence is.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, Ctrl* c) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if (n & 63u) continue;
        if (c->abort_flag) return false;
        const uint64_t since = max(t0, (uint64_t)c->alive_ns);
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

static_assert(sizeof(Ctrl) + 2 * kWarps * 8 <= kOffQ && sizeof(Ctrl) % 8 == 0, "control block");

// Cost of one head of a request, by a whole warp (r the same in every lane).
__device__ __forceinline__ long long head_cost(const Request& r, int unit_cost) {
    const int lane = threadIdx.x & 31, nq = units_of(r);
    long long sum = 0;
    for (int qt = lane; qt < nq; qt += 32) sum += tiles_of(r, qt) + unit_cost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The tiles of one head for a request per lane: short ones by their lane, long ones by the
// warp.
__device__ __forceinline__ long long lane_tiles(const Request& r) {
    const int lane = threadIdx.x & 31, nq = units_of(r);
    long long sum = 0;
    for (int qt = 0; qt < nq && nq <= 8; ++qt) sum += tiles_of(r, qt);
    __syncwarp();
    for (uint32_t many = __ballot_sync(0xffffffffu, nq > 8); many != 0u; many &= many - 1u) {
        const int src = __ffs((int)many) - 1;
        Request q = {0, 0, 0, 0};
        q.m = __shfl_sync(0xffffffffu, r.m, src);
        q.L = __shfl_sync(0xffffffffu, r.L, src);
        const long long c = head_cost(q, 0);
        if (lane == src) sum = c;
    }
    return sum;
}

// Whether whole units keep the blocks about as busy as ranges of cost `per` (see kEvenPart); every
// thread.  (Not inlined: a few prompt tokens, which have no use for it, took 0.7 of 20.4 us more with it
// in the way.)
__device__ __noinline__ int whole_units(const ExpandedParams& p, Ctrl* c, long long per, int unit_cost) {
    const int lane = threadIdx.x & 31;
    const int per_thread = (p.B + kThreads - 1) / kThreads, b0 = (int)threadIdx.x * per_thread;
    // (the average rounded up is at most one unit more than it: short units need no count)
    if (c->most_tiles + unit_cost <= per / kEvenPart) return 1;
    uint32_t bad = 0;  // (known by now)
    auto eighths = [&](int k) { return (c->most_tiles * (k + 1) + kClasses - 1) / kClasses; };
    int n[kClasses] = {};
    for (int i = 0; i < per_thread && b0 + i < p.B; ++i) {
        const Request r = request_of(p, b0 + i, bad);
#pragma unroll
        for (int k = 0; k < kClasses; ++k) n[k] += units_at_least(r, eighths(k));
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kClasses; ++k) {
        const int sum = __reduce_add_sync(0xffffffffu, n[k] * p.H);
        if (lane == 0 && sum != 0) atomicAdd(&c->at_least[k], sum);
    }
    __syncthreads();
    long long longest = 0;
#pragma unroll
    for (int k = 0; k < kClasses; ++k)
        longest = max(longest, (long long)((c->at_least[k] + p.n_cta - 1) / p.n_cta) * (eighths(k) + unit_cost));
    return longest - per <= per / kEvenPart;
}

// Every thread: the problem's cost, this block's range, and the unit where it begins.  Each
// thread sums a run of requests; one scan over the block follows.
__device__ void schedule(const ExpandedParams& p, Ctrl* c, long long* sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_thread = (p.B + kThreads - 1) / kThreads, b0 = (int)threadIdx.x * per_thread;
    uint32_t bad = 0;
    long long mine = 0, units = 0;
    int most = 0;
    for (int i = 0; i < per_thread; ++i) {
        Request r = {0, 0, 0, 0};
        if (b0 + i < p.B) r = request_of(p, b0 + i, bad);
        mine += lane_tiles(r) * p.H;
        units += (long long)units_of(r) * p.H;
        if (r.m > 0) most = max(most, tiles_of(r, units_of(r) - 1));
    }
    if (bad) atomicOr(&c->bad, bad);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0 && most > 0) atomicMax(&c->most_tiles, most);
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
    const int unit_cost = total <= kFewTiles * p.n_cta ? 0 : kUnitCost;
    total += unit_cost * total_units;
    before += unit_cost * units_before;
    mine += unit_cost * units;
    long long per = (total + p.n_cta - 1) / p.n_cta;
    const int whole = p.may_whole ? whole_units(p, c, per, unit_cost) : 0;
    if (unit_cost) per = max(per, (long long)(kMinTiles + kUnitCost));
    const long long t0 = per * blockIdx.x;
    if (threadIdx.x == 0) {
        c->per = per;
        c->unit_cost = unit_cost;
        c->t0 = t0;
        c->left = t0 < total ? min(per, total - t0) : 0;
        c->whole = whole;
    }
    // the warp whose requests hold position t0 looks through them
    const uint32_t here = __ballot_sync(0xffffffffu, before <= t0 && t0 < before + mine);
    if (here) {
        const int src = __ffs((int)here) - 1;
        long long run = __shfl_sync(0xffffffffu, before, src);
        for (int b = __shfl_sync(0xffffffffu, b0, src);; ++b) {
            const Request r = request_of(p, b, bad);
            const long long per_head = head_cost(r, unit_cost);
            if (t0 >= run + per_head * p.H) {
                run += per_head * p.H;
                continue;
            }
            // the head, then the query tokens
            long long off = t0 - run;
            const int h = (int)(off / per_head);
            off -= h * per_head;
            const int nq = units_of(r);
            long long at = 0;
            for (int q0 = 0; q0 < nq && at <= off; q0 += 32) {
                const int cost = q0 + lane < nq ? tiles_of(r, q0 + lane) + unit_cost : 0;
                long long in = cost;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += y;
                }
                const long long ex = at + in - cost;
                if (ex <= off && off < ex + cost) {
                    c->b = b;
                    c->h = h;
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

// Finds this block's pieces, by a whole warp.
struct Finder {
    Request r;
    int b, h, qt, unit_cost;
    long long left;  // cost of the range after this piece
    int base, cls;   // whole units: the first of request b, and its class
    bool first, whole;
    __device__ __forceinline__ Piece piece(int j0, int j1) const {
        const int m0 = qt * kRows;
        return {r.t0 + m0, min(kRows, r.m - m0), r.L - r.m + m0, r.k0, r.L, h, tiles_of(r, qt), j0, j1};
    }
    // [off, ..) of the unit's cost, of which its own lies before its first tile
    __device__ __forceinline__ Piece cut(int off) {
        const int take = (int)min((long long)tiles_of(r, qt) + unit_cost - off, left);
        left -= take;
        // (0, 0: the range ends before the first tile)
        return piece(max(0, off - unit_cost), max(0, off + take - unit_cost));
    }
    __device__ __forceinline__ void init(const ExpandedParams& p, const Ctrl* c) {
        first = true;
        left = c->left;
        unit_cost = c->unit_cost;
        uint32_t bad = 0;
        base = 0;
        cls = kClasses - 1;
        whole = c->whole;
        // (a block without a range has no place where it begins)
        const bool range = !whole && left > 0;
        b = range ? c->b : -1;
        h = range ? c->h : 0;
        qt = range ? c->qt : 0;
        r = {0, 0, 0, 0};
        if (range) r = request_of(p, b, bad);
    }
    // (the warps that wait for the next piece may wait for as long as there are requests to pass over)
    static __device__ __forceinline__ void passed(Ctrl* c, int b) {
        if ((threadIdx.x & 31) == 0 && (b & 0xffff) < 32) c->alive_ns = globaltimer_ns();
    }
    // The next request of this class, then of those below; false: none.
    __device__ __forceinline__ bool advance(const ExpandedParams& p, Ctrl* c) {
        const int lane = threadIdx.x & 31;
        uint32_t bad = 0;
        for (; cls >= 0; --cls, b = -1) {
            for (int b0 = b + 1; b0 < p.B; b0 += 32) {
                passed(c, b0);
                Request q = {0, 0, 0, 0};
                if (b0 + lane < p.B) q = request_of(p, b0 + lane, bad);
                const uint32_t here =
                    __ballot_sync(0xffffffffu, q.m > 0 && class_of(q, c->most_tiles) == cls);
                if (here == 0u) continue;
                const int src = __ffs((int)here) - 1;
                b = b0 + src;
                r.t0 = __shfl_sync(0xffffffffu, q.t0, src);
                r.m = __shfl_sync(0xffffffffu, q.m, src);
                r.k0 = __shfl_sync(0xffffffffu, q.k0, src);
                r.L = __shfl_sync(0xffffffffu, q.L, src);
                return true;
            }
        }
        r.m = 0;
        return false;
    }
    __device__ __forceinline__ Piece next(const ExpandedParams& p, Ctrl* c) {
        uint32_t bad = 0;
        const Piece none = {};
        const bool begin = first;
        first = false;
        if (whole) {
            int u = blockIdx.x;
            if (!begin) {
                if ((threadIdx.x & 31) == 0) u = p.n_cta + (int)atomicAdd(p.counter, 1u);
                u = __shfl_sync(0xffffffffu, u, 0);
            }
            while (u - base >= units_of(r) * p.H) {
                base += units_of(r) * p.H;
                if (!advance(p, c)) return none;
            }
            // as many heads at a time as kSharedKeys allows, the last query tokens first
            const int nq = units_of(r);
            const int most = min(p.H, max(1, min(kMostHeads, kSharedKeys / max(r.L, 1))));
            const int x = u - base, h0 = x / (nq * most) * most;
            const int heads = min(most, p.H - h0), y = x - h0 * nq;
            qt = nq - 1 - y / heads;
            h = h0 + y % heads;
            return piece(0, tiles_of(r, qt));
        }
        if (begin) return left > 0 ? cut(c->off) : none;
        if (left == 0) return none;
        if ((++qt) * kRows >= r.m) {
            qt = 0;
            if (++h == p.H) {
                h = 0;
                do {  // (cost is left, so a request with tokens is)
                    r = request_of(p, ++b, bad);
                    if ((b & 0xffff) == 0) passed(c, b);
                } while (r.m == 0);
            }
        }
        return cut(0);
    }
};

// The pieces as the other warps read them.
struct Reader {
    uint32_t n;
    Piece x;
    // the next piece; false: no more, or a wait gave up
    __device__ __forceinline__ bool next(Ctrl* c) {
        if (!wait_warp(&c->piece_full[n % kPieces], (n / kPieces) & 1u, c)) return false;
        x = c->piece[n % kPieces];
        return x.j0 < x.j1;
    }
    // it is not looked at again
    __device__ __forceinline__ void done(Ctrl* c) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&c->piece_empty[n % kPieces]);
        ++n;
    }
};

// One row against keys [k0, k1) (rows of k and v) of head h, by a whole warp: what the row does
// not see is not touched.  Lane l ends up with columns 4 l .. 4 l + 3 of o (normalised); returns
// the log-sum-exp in log2 units.
__device__ __forceinline__ float slow_row(const ExpandedParams& p, Ctrl* c, size_t qrow, int h,
                                       int k0, int k1, float (&o)[4]) {
    const int lane = threadIdx.x & 31;
    const uint2 qn = __ldg(reinterpret_cast<const uint2*>(p.q + qrow * kQk) + lane);
    const uint32_t qr = __ldg(reinterpret_cast<const uint32_t*>(p.q + qrow * kQk + kNope) + lane);
    auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    float m = ninf_f(), l = 0.f;
    o[0] = o[1] = o[2] = o[3] = 0.f;
    // four keys at a time, so that their loads and sums overlap
    for (int k4 = k0; k4 < k1; k4 += 4) {
        if (lane == 0 && ((k4 - k0) & 127) == 0) c->alive_ns = globaltimer_ns();
        float s[4];
        uint2 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const size_t key = min(k4 + u, k1 - 1);
            const uint2 kn = __ldg(reinterpret_cast<const uint2*>(p.k_nope + key * p.k_token + h * p.k_head) + lane);
            const uint32_t kr = __ldg(reinterpret_cast<const uint32_t*>(p.k_rope + key * p.r_token) + lane);
            v[u] = __ldg(reinterpret_cast<const uint2*>(p.v + key * p.v_token + h * p.v_head) + lane);
            s[u] = lo(qn.x) * lo(kn.x) + hi(qn.x) * hi(kn.x) + lo(qn.y) * lo(kn.y) +
                   hi(qn.y) * hi(kn.y) + lo(qr) * lo(kr) + hi(qr) * hi(kr);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], d);
        float mn = m;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = k4 + u < k1 ? s[u] * p.scale_log2 : ninf_f();
            mn = fmaxf(mn, s[u]);
        }
        const float r = mn == ninf_f() ? 0.f : mn, f = ex2(m - r);
        l *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (k4 + u >= k1) continue;
            const float e = ex2(s[u] - r);
            l += e;
            o[0] += e * lo(v[u].x);
            o[1] += e * hi(v[u].x);
            o[2] += e * lo(v[u].y);
            o[3] += e * hi(v[u].y);
        }
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    return l == 0.f ? ninf_f() : m + lg2(l);
}

__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const __grid_constant__ ExpandedParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&ctrl->piece_full[i], 1);
            mbar_init(&ctrl->piece_empty[i], kReaders);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ctrl->full[i], 1);
            mbar_init(&ctrl->empty[i], 2);  // the two issuing warps
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
        ctrl->alive_ns = 0;
        ctrl->abort_flag = 0;
        ctrl->bad = 0;
        ctrl->most_tiles = 0;
        for (int i = 0; i < kClasses; ++i) ctrl->at_least[i] = 0;
        fence_barrier_init();
        prefetch_tmap(&p.qmap);
        prefetch_tmap(&p.kmap);
        prefetch_tmap(&p.rmap);
        prefetch_tmap(&p.vmap);
    }
    if (warp == 11) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    wait_for_earlier();
    schedule(p, ctrl, reinterpret_cast<long long*>(smem + sizeof(Ctrl)));
    const uint32_t tmem = ctrl->tmem_base;
    int4 desc = make_int4(-1, 0, 0, 0);

    {
        if (warp == 8) {
            // ============================== loads of K and V
            const uint64_t pol = l2_policy_evict_normal();
            uint32_t g = 0;  // slots so far
            uint32_t n = 0;  // pieces shown
            bool ok = true;
            Finder find;
            find.init(p, ctrl);
            auto show = [&]() -> Piece {
                const Piece x = find.next(p, ctrl);
                if (n >= kPieces)
                    ok = wait_warp(&ctrl->piece_empty[n % kPieces], (n / kPieces - 1) & 1u, ctrl);
                if (lane == 0 && ok) {
                    ctrl->piece[n % kPieces] = x;
                    mbar_arrive(&ctrl->piece_full[n % kPieces]);
                }
                __syncwarp();
                ++n;
                return x;
            };
            Piece x = show();
            while (x.j0 < x.j1 && ok) {
                // (one piece ahead, so that its Q can be asked for)
                const Piece next = show();
                if (!ok) break;
                if (x.j0 == 0 && x.j1 < x.nt) {
                    // the unit that this block leaves unfinished, for the join (it ends with
                    // this piece, which ends with the range)
                    const long long last = ctrl->t0 + ctrl->left + x.nt - x.j1 - 1;
                    desc = make_int4(x.t0, x.ntok, x.h, (int)(last / ctrl->per - blockIdx.x) + 1);
                }
                for (int j = x.j0; j < x.j1 && ok; ++j) {
                    if (lane == 0 && (j & 1023) == 0) ctrl->alive_ns = globaltimer_ns();
                    for (int i = 0; i < 5; ++i, ++g) {
                        const uint32_t st = g % kSlots;
                        if (g >= kSlots) {
                            ok = wait_warp(&ctrl->empty[st], (g / kSlots - 1) & 1u, ctrl);
                            if (!ok) break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&ctrl->full[st], kSlotBytes);
                            uint8_t* dst = smem + kOffRing + st * kSlotBytes;
                            const int key = x.k0 + j * kTile;
                            if (i < 2)
                                tma_load_3d(dst, &p.kmap, i * 64, x.h, key, &ctrl->full[st], pol);
                            else if (i == 2)
                                tma_load_2d(dst, &p.rmap, 0, key, &ctrl->full[st], pol);
                            else
                                for (int c = 0; c < 2; ++c)
                                    tma_load_3d(dst + c * (kSlotBytes / 2), &p.vmap, c * 64, x.h,
                                                key + (i - 3) * 64, &ctrl->full[st], pol);
                        }
                        __syncwarp();
                    }
                }
                x = next;
            }
            // no copy may be in flight when the block leaves
            for (uint32_t s = 0; s < kSlots; ++s)
                if (s < g && !wait_on(&ctrl->full[s], ((g - 1 - s) / kSlots) & 1u, ctrl))
                    mbar_drain(&ctrl->full[s], ((g - 1 - s) / kSlots) & 1u);
            __syncwarp();
        } else if (warp == 9) {
            // ============================== loads of Q
            const uint64_t pol_q = l2_policy_evict_first();
            uint32_t q_loads[2] = {0u, 0u};
            bool ok = true;
            Reader w = {};
            bool more = w.next(ctrl);
            while (more && ok) {
                const Piece x = w.x;
                const int nq = x.tiles_q();
                w.done(ctrl);
                more = w.next(ctrl);
                for (int mt = 0; mt < nq && ok; ++mt) {
                    if (q_loads[mt] > 0)
                        ok = wait_warp(&ctrl->q_empty[mt], (q_loads[mt] - 1) & 1u, ctrl);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ctrl->q_full[mt], kQBytes);
                        for (int c = 0; c < 3; ++c)
                            tma_load_3d(smem + kOffQ + mt * kQBytes + c * kSlotBytes, &p.qmap, c * 64, x.h,
                                        x.t0 + mt * kTile, &ctrl->q_full[mt], pol_q);
                    }
                    __syncwarp();
                    ++q_loads[mt];
                }
                // the next unit's Q into L2: its load is then short
                if (more && lane < 3 * w.x.tiles_q())
                    prefetch_3d(&p.qmap, lane % 3 * 64, w.x.h, w.x.t0 + lane / 3 * kTile);
            }
            for (int mt = 0; mt < 2; ++mt)
                if (q_loads[mt] > 0 && !wait_on(&ctrl->q_full[mt], (q_loads[mt] - 1) & 1u, ctrl))
                    mbar_drain(&ctrl->q_full[mt], (q_loads[mt] - 1) & 1u);
            __syncwarp();
        } else if (warp >= 10) {
            // ============================== products of query tile mt
            // All lanes run the loop, so that addresses and descriptors stay uniform
            // across the warp; one elected lane's predicate issues.
            const int mt = warp - 10;
            const uint32_t lead = elect_one();
            const uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
            const uint32_t idesc_o = idesc_bf16_f32(128, 128, true);
            const uint64_t q_desc = sdesc_sw128(sbase + kOffQ + mt * kQBytes, 16, 1024);
            const uint64_t k_desc = sdesc_sw128(sbase + kOffRing, 16, 1024);
            const uint64_t v_desc = sdesc_sw128(sbase + kOffRing, kSlotBytes / 2, 1024);
            constexpr uint32_t kStep = kSlotBytes >> 4;
            const uint32_t s_col = tmem + mt * 128u, o_col = tmem + 256u + mt * 128u;
            uint32_t kg = 0, vg = 3;  // ring positions of the tile whose scores / values are next
            uint32_t qpar = 0, ppar = 0, tpar = mt == 0 ? 1u : 0u;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t par) {
                ok = ok && wait_warp(bar, par, ctrl);
                return ok;
            };
            auto wait_slot = [&](uint32_t at) {
                return wait(&ctrl->full[at % kSlots], (at / kSlots) & 1u);
            };
            // half of PV: 64 keys
            auto issue_pv = [&](int half, bool first) {
                const uint64_t b = v_desc + (vg + half) % kSlots * kStep;
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4)
                    mma_ts(lead, o_col, s_col + (half * 4 + k4) * 8u, b + ((k4 * 16 * 128) >> 4), idesc_o,
                           first && k4 == 0 ? 0u : 1u);
                commit(lead, &ctrl->empty[(vg + half) % kSlots]);
            };
            // what the tile before the current one was
            int nq_prev = 0;
            bool first_prev = false, last_prev = false;
            // A round: PV of the tile before, S of this one (after the last tile there is
            // one more round).  The weights are waited for last, as what comes last; the
            // turn is handed on when all is issued.
            auto round = [&](int nq, bool first, bool last) {
                const bool pv = mt < nq_prev, sc = mt < nq;
                if (pv && !wait_slot(vg)) return;
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
                    if (!wait_slot(vg + 1)) return;
                    if (!wait(&ctrl->p_full[mt][1], ppar)) return;
                    ppar ^= 1u;
                    tc_fence_after_sync();
                    issue_pv(1, false);
                    if (last_prev) commit(lead, &ctrl->o_full[mt]);
                } else if (nq_prev && lead) {
                    mbar_arrive(&ctrl->empty[vg % kSlots]);
                    mbar_arrive(&ctrl->empty[(vg + 1) % kSlots]);
                }
                if (sc) {
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        if (!wait_slot(kg + c)) return;
                        const uint64_t b = k_desc + (kg + c) % kSlots * kStep;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(lead, s_col, q_desc + c * kStep + kk * 2, b + kk * 2, idesc_s,
                                   c + kk > 0 ? 1u : 0u);
                        commit(lead, &ctrl->empty[(kg + c) % kSlots]);
                        // The turn is handed on before the last third: the other warp is up when it
                        // is done (917 -> 890 us for 2 x 8192 tokens; before the second third 910).
                        // A warp without a part in the tile gives its slots back at once, and so
                        // may only be up when all of them have come.
                        if (c == (nq > 1 ? 1 : 2) && lead) mbar_arrive(&ctrl->turn[mt ^ 1]);
                    }
                    commit(lead, &ctrl->s_full[mt]);
                    if (last) commit(lead, &ctrl->q_empty[mt]);
                } else if (lead) {
                    for (int c = 0; c < 3 && nq; ++c) mbar_arrive(&ctrl->empty[(kg + c) % kSlots]);
                    mbar_arrive(&ctrl->turn[mt ^ 1]);
                }
                __syncwarp();
                if (nq_prev) vg += 5;
                if (nq) kg += 5;
                nq_prev = nq;
                first_prev = first;
                last_prev = last;
            };
            Reader w = {};
            while (ok && w.next(ctrl)) {
                const int nq = w.x.tiles_q(), n_tiles = w.x.j1 - w.x.j0;
                w.done(ctrl);
                for (int j = 0; j < n_tiles && ok; ++j) round(nq, j == 0, j == n_tiles - 1);
            }
            if (ok && kg > 0) round(0, false, false);
            commit(lead, &ctrl->mma_done);
            if (!wait_warp(&ctrl->mma_done, 0, ctrl)) mbar_drain(&ctrl->mma_done, 0);
        } else {
            // ============================== softmax and output
            const int mt = warp >> 2;
            const int r = (warp & 3) * 32 + lane, R = mt * 128 + r;
            const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_addr = tmem + lane_addr + mt * 128u;
            const uint32_t o_addr = tmem + lane_addr + 256u + mt * 128u;
            uint32_t spar = 0, opar = 0;
            uint32_t g = 0;  // key tiles of this block so far (the ring's position)
            bool ok = true;
            Reader w = {};
            while (ok && w.next(ctrl)) {
                const Piece x = w.x;
                w.done(ctrl);
                const int j0 = x.j0, j1 = x.j1, h = x.h, k0 = x.k0, L = x.L;
                if (mt >= x.tiles_q()) {
                    g += j1 - j0;
                    continue;
                }
                const bool active = R < x.ntok, split = j0 > 0 || j1 < x.nt;
                const int pos = x.p0 + R;
                const int p_min = x.p0 + mt * 128;  // position of this query tile's first token
                const int row = (x.t0 + (active ? R : 0)) * p.H + h;
                float m_used = ninf_f(), l = 0.f;
                for (int j = j0; j < j1; ++j, ++g) {
                    const int key0 = j << 7;
                    ok = wait_warp(&ctrl->s_full[mt], spar, ctrl);
                    if (!ok) break;
                    spar ^= 1u;
                    tc_fence_after_sync();
                    uint32_t s[128];
                    tmem_ld_x128(s_addr, s);
                    if (key0 + 127 > p_min) {
                        const int z = pos + 1 - key0;  // columns below z
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            const uint32_t bits = bits_below(z - 32 * q4);
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
                    // keys past the sequence's end (the next request's, or none): their V rows are
                    // cleared (by both query tiles, each before its own products)
                    if (key0 + 128 > L) {
                        const uint32_t at = 5 * g + 3;
                        ok = wait_warp(&ctrl->full[at % kSlots], (at / kSlots) & 1u, ctrl) &&
                             wait_warp(&ctrl->full[(at + 1) % kSlots], ((at + 1) / kSlots) & 1u, ctrl);
                        if (!ok) break;
                        const int first = L - key0;
                        for (int i = 16 * first + r; i < 16 * 128; i += 128) {  // 16 bytes of key i / 16
                            const int k = i >> 4, c = i & 15;
                            *reinterpret_cast<uint4*>(smem + kOffRing + (at + (k >> 6)) % kSlots * kSlotBytes +
                                                      (c >> 3) * (kSlotBytes / 2) + (k & 63) * 128 +
                                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
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

                // ---- output: the row, or its part of a unit cut by the block's range
                ok = wait_warp(&ctrl->o_full[mt], opar, ctrl);
                if (!ok) break;
                opar ^= 1u;
                tc_fence_after_sync();
                const size_t slot = 2 * (size_t)blockIdx.x + (j0 > 0 ? 0 : 1);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float lse2 = l == 0.f ? ninf_f() : m_used + lg2(l);
                // rows of the lane pair, -1 where there is none
                const int row_x = __shfl_xor_sync(0xffffffffu, active ? row : -1, 1);
                const int row_e = lane & 1 ? row_x : (active ? row : -1);
                const int row_o = lane & 1 ? (active ? row : -1) : row_x;
                float check = lse2 == ninf_f() ? 0.f : lse2;
                float4* po = p.part_o + slot * 32 * kRows + R;
                // (Two lanes exchange halves, so that they write 64 bytes of a row together, as in
                // cpa_window.cu.)
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
                    const float z = slow_row(p, ctrl, row_a, h, k0 + j0 * 128,
                                             k0 + min(j1 * 128, pos_a + 1), f);
                    if (split) {
                        p.part_o[(slot * 32 + lane) * kRows + R_a] = make_float4(f[0], f[1], f[2], f[3]);
                        if (lane == 0) p.part_lse[slot * kRows + R_a] = z;
                    } else {
                        reinterpret_cast<uint2*>(p.o + row_a * kV)[lane] =
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
__global__ void __launch_bounds__(256) expanded_join_kernel(const __grid_constant__ ExpandedParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_for_earlier();
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
    const int R = blockIdx.y * 32 + (threadIdx.x & 31);
    if (R >= d.y) return;
    const size_t row = (size_t)(d.x + R) * p.H + d.z;
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

// All that a call without new tokens does: its starts are looked at.
__global__ void __launch_bounds__(256) starts_kernel(const int32_t* q_start, const int32_t* k_start, int B,
                                                     int T_k, uint32_t* status) {
    uint32_t bad = 0;
    for (int b = threadIdx.x; b < B; b += 256) request_of(q_start, k_start, 0, T_k, b, bad);
    const bool any = __syncthreads_or((int)bad);
    if (threadIdx.x == 0) *status = any ? CPA_DEV_BAD_LENGTH : 0u;
}

struct ExpandedWs {
    size_t counter, bad, desc, part_lse, part_o, total;
};
ExpandedWs expanded_ws(int n_cta) {
    ExpandedWs w;
    w.counter = 128;  // (beside the status word)
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
        return (int)cudaFuncSetAttribute(expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmem);
    });
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_latent_prefill_workspace_size(int B, int T, int T_k, int H, int nope_dim, int rope_dim,
                                         int v_dim) {
    if (B < 1 || T < 0 || T_k < 0 || H < 1 || nope_dim != kNope || rope_dim != kRope || v_dim != kV)
        return 0;
    const int n_sm = sm_count();
    return n_sm <= 0 ? 0 : expanded_ws(n_sm).total;
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
    if (T == 0) {
        starts_kernel<<<1, 256, 0, s>>>(q_start, k_start, B, T_k, static_cast<uint32_t*>(workspace));
        return cudaGetLastError() == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
    }
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    const ExpandedWs w = expanded_ws(n_sm);
    if (workspace_bytes < w.total) return CPA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ExpandedParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_nope = static_cast<const __nv_bfloat16*>(k_nope);
    p.k_rope = static_cast<const __nv_bfloat16*>(k_rope);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_start = q_start;
    p.k_start = k_start;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.counter = reinterpret_cast<uint32_t*>(ws + w.counter);
    p.bad = reinterpret_cast<uint32_t*>(ws + w.bad);
    p.desc = reinterpret_cast<int4*>(ws + w.desc);
    p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    p.part_o = reinterpret_cast<float4*>(ws + w.part_o);
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
    p.n_cta = n_sm;
    // (no keys: every request is empty, or its starts are refused on the device; the maps are
    // not used then)
    const void* const kn = T_k > 0 ? k_nope : q;
    const void* const kr = T_k > 0 ? k_rope : q;
    const void* const vv = T_k > 0 ? v : q;
    const uint64_t keys = T_k > 0 ? (uint64_t)T_k : 1;
    if (!make_heads_map(&p.qmap, q, kQk, H, (uint64_t)T, kQk, (int64_t)H * kQk, 1, 128) ||
        !make_heads_map(&p.kmap, kn, kNope, H, keys, k_head_stride, k_token_stride, 1, 128) ||
        !make_heads_map(&p.vmap, vv, kV, H, keys, v_head_stride, v_token_stride, 1, 64) ||
        !make_rows_map(&p.rmap, kr, kRope, keys, rope_token_stride, 128))
        return CPA_ERR_CUDA;
    if (raise_smem_once() != cudaSuccess) return CPA_ERR_CUDA;
    p.may_whole = (long long)T * H >= (long long)kWholeUnits * n_sm * kRows;
    if (p.may_whole && cudaMemsetAsync(p.counter, 0, 4, s) != cudaSuccess) return CPA_ERR_CUDA;
    if (launch_overlapped(expanded_kernel, dim3((unsigned)n_sm), kThreads, kSmem, s, p) != cudaSuccess)
        return CPA_ERR_LAUNCH;
    return launch_overlapped(expanded_join_kernel,
                             dim3((unsigned)n_sm, (unsigned)((T < kRows ? T : kRows) + 31) / 32), 256, 0, s,
                             p) == cudaSuccess
               ? CPA_OK
               : CPA_ERR_LAUNCH;
}

}  // extern "C"
