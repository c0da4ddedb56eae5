// cpa_latent.cu -- decode over a paged cache of latents, in the absorbed form: every
// head's keys and values come from one vector of 512 + 64 elements a token, all of
// it the key, the first 512 the value.
//
// Unit: up to 64 rows of one request (a row is a (token, head) pair; whole tokens, or
// a part of one token's heads) against its key tiles of 64 tokens.  A tile is loaded
// once and read twice, as K (nine chunks of 64 columns) and as V (eight of them):
//     S[64 rows x 64 keys]    = Q K^T              M = 64, N = 64, 36 products
//     O^T[512 x rows]        += V^T P^T            M = 128 (four blocks), N = rows
// O^T and not O: its four blocks of 128 columns lie in the 128 lanes of TMEM, a column
// per row, so 64 rows need 256 of the 512 columns (as O[64 x 512] they would need all),
// and V^T comes straight from the tile, whose rows are keys.  P is the only operand that
// goes through shared memory.
//
// The order of the products: while one tile's scores go through the softmax, the next
// tile's are made.  What is ready goes first, values before scores where both are (they
// give the ring its places back).
//
// Warps (7): 0-3 softmax and output, 4 loads the tiles and 6 Q, 5 issues the products.  Every
// warp finds the block's range by itself, before the barriers are ready.  Scores lie 16 rows
// to a warp; a thread holds 16 scores of two rows, a row's maximum is exchanged between
// four lanes.  A rescale of O (a row's maximum grew by more than 2^8) is of columns, and
// so for all four warps: they agree on it with one barrier a tile.
//
// Values that are not numbers.  A masked key has weight 0, but 0 times a NaN in V is a
// NaN in a matrix product.  Slots past a sequence's end are cleared in shared memory.  Of
// keys that some rows of the request see and others do not (the last S - 1 at most)
// elements that are not finite are cleared too, and the rows that see them get NaN in those
// columns when the output is written: such an element is part of the key, whose score is
// infinite or NaN with it, so that the row is NaN throughout or the weight 0, and 0 times it NaN.
//
// Split.  As in cpa_decode the key tiles of all units lie end to end, every block takes a
// range of equal cost, and a unit cut by a range's end is joined by a second kernel in the
// order of its parts.
//
// What bounds it.  Up to 32 rows: HBM (64 x 2000 tokens, 16 heads: 39.7 us, 3.7 TB/s with the
// launches in it; 64 x 16000: 195 us, 6.05 TB/s, 0.89 of the copy rate).  64 rows: the ring.  It
// holds two tiles, and a tile stays in it for its load (2100 cycles), its scores (1220), the
// softmax (1000) and its values (810), some of them behind another tile's: 3230 cycles a tile,
// where shared memory needs 2490 for what the products of one SM read and the loads write, HBM 3100
// when no other block shares the tile and the products alone 2030 (64 x 16000 tokens, 64 heads: 202 us;
// 32 ragged requests of 128 heads: 114 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cmath>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_device.cuh"
#include "cpa_host.h"
#include "cpa_mma.cuh"

namespace cpa {
namespace {

constexpr int kC = 512, kR = 64, kSlot = kC + kR;
constexpr int kThreads = 224;
constexpr int kRows = 64;   // rows of a unit
constexpr int kKeys = 64;   // tokens of a tile
constexpr int kMaxTokens = 64;  // S: the mask of a request's last tokens is one word
// Eight tokens are one box of a load, 9 KB that lie together in a page: in shared memory
// nine chunks of 64 columns, eight rows of 128 bytes each.  Four of them, half a tile, are a
// slot of the ring.
constexpr uint32_t kBox = 9u * 1024u;
constexpr uint32_t kSlotBytes = 4 * kBox;
constexpr int kMaxSlots = 5;
// Halves that are asked into L2 ahead of their load.  (None, one, two: 64 x 2000 tokens 39.6, 39.8,
// 40.1 us; 64 x 16000 199, 195, 192, with 64 heads 217, 202, 201; 32 ragged requests of 128 heads
// 117.8, 113.7, 113.8; five tokens a request 53.9, 53.0, 53.3.)
constexpr int kAhead = 1;
constexpr uint32_t kOffQ = 1024;
constexpr uint32_t kMaxSmem = 232448;
constexpr uint32_t kColS = 256;  // TMEM: O^T in columns 0 .. 255, the scores of two tiles
// What a unit costs besides its tiles, in tiles.  (1, 2, 3: 64 x 2000 tokens 39.1, 39.8, 40.5 us, 32
// ragged requests of 128 heads 115.1, 113.7, 114.1, five tokens a request 54.1, 53.0, 54.3.)
constexpr int kUnitCost = 2;
constexpr float kRescale = 8.0f;  // O is rescaled when a row's maximum grew by more than 2^8

// Shared memory by rows of a unit: Q, P, then the ring.  Five slots up to 32 rows, four for 64.
CPA_HD uint32_t q_chunk(int rows) { return (uint32_t)((rows + 7) & ~7) * 128u; }
CPA_HD uint32_t off_p(int rows) { return kOffQ + 9u * q_chunk(rows); }
CPA_HD uint32_t off_k(int rows) { return off_p(rows) + (uint32_t)((rows + 15) & ~15) * 128u; }
CPA_HD int slots_of(int rows) {
    const int n = (int)((kMaxSmem - 1024u - off_k(rows)) / kSlotBytes);  // (aligned up inside)
    return n < kMaxSlots ? n : kMaxSlots;
}

struct LatentParams {
    CUtensorMap cmap, rmap, kmap;
    const __nv_bfloat16* pages;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* o;
    float* lse;
    uint32_t* status;
    uint32_t* bad;    // [n_cta] what each block found wrong
    int4* desc;       // (request, pair, parts, group) of units that start in a group's range and
                      // go on past it: [n_grp] by group (request -1: none), or, where there are no
                      // more units than groups, by unit (parts 1: none)
    float* part_lse;  // [2 n_cta][kRows], log2 units
    float* part_o;    // [2 n_cta][kRows][kC]
    int stride, B, S, H, lp, num_pages, max_len;
    int heads, n_ht;    // heads of a unit, and units of a token
    int toks, n_rt;     // tokens of a unit, and units of a request
    int cl, n_pairs;    // blocks of a group (they share key ranges), groups of units of a request
    int n_cta, n_grp;
    int by_unit;
    int n_slots;
    float scale_log2;
};

// The length of a request; 0 where it is out of range.
__device__ __forceinline__ int length_of(const LatentParams& p, int b, uint32_t& bad) {
    const int L = __ldg(p.lens + b);
    if (L >= 0 && L <= p.max_len) return L;
    bad |= CPA_DEV_BAD_LENGTH;
    return 0;
}
// (a request without keys has one tile, all of it masked, so that its rows are written)
__device__ __forceinline__ int tiles_of(int L) { return L > 0 ? (L + kKeys - 1) / kKeys : 1; }

struct Ctrl {
    uint64_t q_full, q_empty;
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots];
    uint64_t s_full[2], p_full, pv_done, o_full, o_empty, mma_done;  // (the last of the barriers)
    unsigned long long odd;  // keys L - S + 1 + i of the unit with values that are not finite
    uint32_t tmem_base;
    volatile uint32_t abort_flag;
    uint32_t bad;
    float row[kRows];         // factors of the rows for a rescale, or for the output
};
constexpr int kBarriers = 2 + 2 * kMaxSlots + 7;
static_assert(sizeof(Ctrl) <= kOffQ && offsetof(Ctrl, odd) == 8 * kBarriers, "control block");

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctrl* c) {
    // (the first look by itself: most waits find the phase complete)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, &c->abort_flag, &c->bad);
}

// Walks the pieces (unit, tiles [j0, j1)) of a group's range of cost, in tiles; j0 == j1 past
// the last.  A unit costs its tiles and unit_cost (kUnitCost, or 0 where no group takes more than
// two tiles), which counts as lying before its first tile.
struct Walker {
    int b, pair, L, nt, j0, j1, unit_cost;
    long long left;     // cost of the range after this piece
    long long end, per; // of the range; of every range
    __device__ __forceinline__ void cut(int off) {
        const int take = (int)min((long long)nt + unit_cost - off, left);
        left -= take;
        j0 = max(0, off - unit_cost);
        j1 = max(0, off + take - unit_cost);  // (0: the range ends before the first tile)
    }
    __device__ __forceinline__ bool more() const { return j0 < j1; }
    __device__ __forceinline__ void at(const LatentParams& p, int off) {
        uint32_t bad = 0;
        L = length_of(p, b, bad);
        nt = tiles_of(L);
        cut(off);
    }
    // By a whole warp: the problem's cost, the range of group grp, and the unit where it begins.
    __device__ void init(const LatentParams& p, int grp, uint32_t& bad) {
        const int lane = threadIdx.x & 31;
        long long total = 0;
        int tiles = 0;  // of this lane's request in the last 32
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            tiles = b0 + lane < p.B ? tiles_of(length_of(p, b0 + lane, bad)) : 0;
            total += tiles;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= p.n_pairs;
        unit_cost = total <= 2 * p.n_grp ? 0 : kUnitCost;
        total += (long long)unit_cost * p.B * p.n_pairs;
        // (a 64-bit division is a long sequence)
        per = total < 0x7fffffffll - p.n_grp ? (int)(total + p.n_grp - 1) / p.n_grp
                                             : (total + p.n_grp - 1) / p.n_grp;
        const long long t0 = per * grp;
        left = t0 < total ? min(per, total - t0) : 0;
        end = t0 + left;
        b = pair = j0 = j1 = 0;
        if (left == 0) return;
        long long before = 0;  // cost of the requests before these 32
        for (int b0 = 0;; b0 += 32) {
            if (p.B > 32) {
                uint32_t none = 0;
                tiles = b0 + lane < p.B ? tiles_of(length_of(p, b0 + lane, none)) : 0;
            }
            const int cost = tiles + unit_cost;
            const long long mine = b0 + lane < p.B ? (long long)cost * p.n_pairs : 0;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const long long from = before + incl - mine;
            const uint32_t here = __ballot_sync(0xffffffffu, from <= t0 && t0 < from + mine);
            if (here) {
                const int src = __ffs((int)here) - 1;
                b = b0 + src;
                const long long in = __shfl_sync(0xffffffffu, t0 - from, src);
                const int of = __shfl_sync(0xffffffffu, cost, src);
                pair = in < 0x7fffffffll ? (int)in / of : (int)(in / of);
                L = length_of(p, b, bad);
                nt = of - unit_cost;
                cut((int)(in - (long long)pair * of));
                return;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __device__ __forceinline__ void next(const LatentParams& p) {
        if (left == 0) {
            j0 = j1;
            return;
        }
        if (++pair == p.n_pairs) {
            pair = 0;
            ++b;
        }
        at(p, 0);
    }
};

// The rows of a unit: heads h0 .. h0 + nh - 1 of tokens s0 .. s0 + ns - 1, n of them.  (Whole
// tokens or one of them: row x of the unit is row `first` + x of the request.)
struct Rows {
    int s0, ns, h0, nh, n, first;
    __device__ __forceinline__ Rows(const LatentParams& p, int rt) {
        s0 = rt / p.n_ht * p.toks;
        h0 = rt % p.n_ht * p.heads;
        ns = min(p.toks, p.S - s0);
        nh = min(p.heads, p.H - h0);
        n = ns * nh;
        first = s0 * p.H + h0;
    }
};

__global__ void __launch_bounds__(kThreads, 1) latent_kernel(const __grid_constant__ LatentParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = blockIdx.x / p.cl, rank = blockIdx.x % p.cl;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x < kBarriers) {
        uint64_t* const bar = &ctrl->q_full + threadIdx.x;
        // (one arrival per softmax warp, where they arrive)
        mbar_init(bar, bar == &ctrl->p_full || bar == &ctrl->o_empty ? 4 : 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        ctrl->odd = 0;
        ctrl->abort_flag = 0;
        ctrl->bad = 0;
    }
    if (warp == 5) {
        tmem_alloc(&ctrl->tmem_base, 512);
        tmem_relinquish();
    }
    wait_for_earlier();
    uint32_t bad = 0;
    Walker w;
    w.init(p, grp, bad);
    // the slot of the pool that box `at` of the walk's request begins with, or -1
    auto box_of = [&](int at) -> int {
        const int pos = at * 8;
        if (at >= 8 * w.j1 || pos >= w.L) return -1;
        const int pg = __ldg(p.table + (size_t)w.b * p.stride + (pos >> p.lp));
        if (pg < 0 || pg >= p.num_pages) {
            bad |= CPA_DEV_BAD_PAGE;
            return -1;
        }
        return (int)(((uint32_t)pg << p.lp) + (uint32_t)(pos & ((1 << p.lp) - 1)));
    };
    // 32 boxes (eight halves) are looked up at a time, a lane each, and the next 32
    int at = 8 * w.j0, boxes = -1, boxes_next = -1;
    if (warp == 4) {
        boxes = box_of(at + lane);
        boxes_next = box_of(at + 32 + lane);
        prefetch_tmap(&p.kmap);
    }
    if (warp == 6 && lane < 2) prefetch_tmap(lane ? &p.cmap : &p.rmap);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctrl->tmem_base;
    int4 desc = make_int4(-1, 0, 0, 0);
    const int rows = p.heads * p.toks, rows_n = (rows + 15) & ~15;  // N of the products of O^T
    const uint32_t o_p = off_p(rows), o_k = off_k(rows);
    const int n_slots = p.n_slots;

    if (w.more()) {
        if (warp == 4) {
            // ============================== loads
            const uint64_t pol = p.n_pairs * p.cl > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
            uint32_t h = 0;  // halves of tiles so far
            int slot = 0;
            uint32_t par = 1;  // parity of the ring's previous round
            bool ok = true;
            for (; w.more() && ok; w.next(p)) {
                if (w.j0 == 0) {
                    // for the join: a unit that this group leaves unfinished ends with this piece,
                    // which ends with the range
                    int parts = 1;
                    if (w.j1 < w.nt) {
                        const long long last = w.end + w.nt - w.j1 - 1;
                        parts = (int)(last / w.per - grp) + 1;
                        desc = make_int4(w.b, w.pair, parts, grp);
                    }
                    if (p.by_unit && lane == 0 && rank == 0)
                        p.desc[w.b * p.n_pairs + w.pair] = make_int4(w.b, w.pair, parts, grp);
                }
                if (h > 0) {
                    at = 8 * w.j0;
                    boxes = box_of(at + lane);
                    boxes_next = box_of(at + 32 + lane);
                }
                for (int half = 2 * w.j0; half < 2 * w.j1; ++half, ++h) {
                    const int i4 = (4 * half - at) & 31;
                    if (half > 2 * w.j0 && i4 == 0) {
                        at += 32;
                        boxes = boxes_next;
                        boxes_next = box_of(at + 32 + lane);
                    }
                    const int box = __shfl_sync(0xffffffffu, boxes, i4 + (lane & 3));
                    // what the ring has no place for yet comes into L2 meanwhile
                    const int far = i4 + kAhead * 4 + (lane & 3);
                    const int b0 = __shfl_sync(0xffffffffu, boxes, far & 31);
                    const int b1 = __shfl_sync(0xffffffffu, boxes_next, far & 31);
                    const int ahead = far < 32 ? b0 : b1;
                    if (h >= (uint32_t)n_slots && lane < 4 && ahead >= 0) prefetch_3d(&p.kmap, 0, ahead, 0);
                    __syncwarp();
                    if (h >= (uint32_t)n_slots) {
                        ok = wait_warp(&ctrl->k_empty[slot], par, ctrl);
                        if (!ok) break;
                    }
                    const uint32_t mask = __ballot_sync(0xffffffffu, lane < 4 && box >= 0);
                    if (lane == 0)
                        mbar_arrive_expect_tx(&ctrl->k_full[slot], (uint32_t)__popc(mask) * kBox);
                    __syncwarp();
                    if (lane < 4 && box >= 0)
                        tma_load_3d(smem + o_k + slot * kSlotBytes + lane * kBox, &p.kmap, 0, box, 0,
                                    &ctrl->k_full[slot], pol);
                    __syncwarp();
                    if (++slot == n_slots) {
                        slot = 0;
                        par ^= 1u;
                    }
                }
            }
            // (a wait gave up: the units that begin in the rest of the range have entries all the
            // same, with nothing to join)
            if (p.by_unit && rank == 0)
                for (; w.more(); w.next(p))
                    if (lane == 0 && w.j0 == 0) p.desc[w.b * p.n_pairs + w.pair] = make_int4(w.b, w.pair, 1, grp);
            // no copy may be in flight when the block leaves
            for (uint32_t i = 0; i < (uint32_t)n_slots; ++i)
                if (i < h && !mbar_wait(&ctrl->k_full[i], ((h - 1 - i) / n_slots) & 1u, &ctrl->abort_flag,
                                        &ctrl->bad))
                    mbar_drain(&ctrl->k_full[i], ((h - 1 - i) / n_slots) & 1u);
            __syncwarp();
        } else if (warp == 6) {
            // ============================== loads of Q
            const uint64_t pol_q = l2_policy_evict_first();
            const uint32_t chunk = q_chunk(rows), q_bytes = (uint32_t)rows * 9u * 128u;
            uint32_t q_loads = 0;
            for (; w.more(); w.next(p)) {
                const Rows r(p, w.pair * p.cl + rank);
                // (this wait lasts as long as the unit: others find out if the pipeline is broken)
                if (q_loads > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(&ctrl->q_empty, (q_loads - 1) & 1u, &ctrl->abort_flag,
                                                       &ctrl->bad, 100 * kWaitLimitNs)))
                    break;
                if (lane == 0) mbar_arrive_expect_tx(&ctrl->q_full, q_bytes);
                __syncwarp();
                if (lane < 9)
                    tma_load_3d(smem + kOffQ + lane * chunk, lane < 8 ? &p.cmap : &p.rmap,
                                lane < 8 ? lane * 64 : 0, r.h0, w.b * p.S + r.s0, &ctrl->q_full, pol_q);
                __syncwarp();
                ++q_loads;
            }
            // (no copy may be in flight when the block leaves)
            if (!mbar_wait(&ctrl->q_full, (q_loads - 1) & 1u, &ctrl->abort_flag, &ctrl->bad))
                mbar_drain(&ctrl->q_full, (q_loads - 1) & 1u);
            __syncwarp();
        } else if (warp == 5) {
            // ============================== products
            // All lanes run the loop, so that addresses and descriptors stay uniform across
            // the warp; one elected lane's predicate issues.
            const uint32_t lead = elect_one();
            const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys, false);
            const uint32_t idesc_h = idesc_bf16_f32(kRows, kKeys / 2, false);
            const uint32_t idesc_o = idesc_bf16_f32(128, rows_n, false) | (1u << 15);  // A: keys are rows
            const uint32_t chunk = q_chunk(rows) >> 4;
            const uint64_t q_desc = sdesc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t k_desc = sdesc_sw128(sbase + o_k, 16, kBox);
            const uint64_t v_desc = sdesc_sw128(sbase + o_k, 1024, kBox);  // chunk after chunk, keys as rows
            const uint64_t p_desc = sdesc_sw128(sbase + o_p, 16, 1024);
            // Two walks over the same tiles: scores g, and the values of tile d behind it.  What is
            // ready goes first; the values where both are, whose places the next loads wait for.
            uint32_t g = 0, d = 0, d_pieces = 0;
            int ks = 0, vs = 0;  // slots of their first halves
            uint32_t kpar = 0, qpar = 0;
            Walker& wk = w;
            Walker wv = w;
            int jk = wk.j0, jv = wv.j0;
            uint64_t since = 0;
            uint32_t n_idle = 0;
            while (wv.more()) {
                bool did = false;
                if (d < g &&
                    __all_sync(0xffffffffu, mbar_test(&ctrl->p_full, d & 1u) &&
                                                (jv > wv.j0 || d_pieces == 0 ||
                                                 mbar_test(&ctrl->o_empty, (d_pieces - 1) & 1u)))) {
                    tc_fence_after_sync();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t a = v_desc + ((vs * kSlotBytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                            for (int blk = 0; blk < 4; ++blk)
                                mma_ss(lead, tmem + blk * kRows, a + ((kk * 2 * kBox + blk * 2048) >> 4),
                                       p_desc + (half * 2 + kk) * 2, idesc_o,
                                       jv == wv.j0 && half + kk == 0 ? 0u : 1u);
                        commit(lead, &ctrl->k_empty[vs]);
                        if (++vs == n_slots) vs = 0;
                    }
                    commit(lead, &ctrl->pv_done);
                    ++d;
                    if (++jv == wv.j1) {
                        commit(lead, &ctrl->o_full);
                        ++d_pieces;
                        wv.next(p);
                        jv = wv.j0;
                    }
                    did = true;
                }
                if (!did && wk.more() && g - d < 2) {
                    const int ks2 = ks + 1 == n_slots ? 0 : ks + 1;
                    const uint32_t kpar2 = ks2 == 0 ? kpar ^ 1u : kpar;
                    if (__all_sync(0xffffffffu, mbar_test(&ctrl->k_full[ks2], kpar2) &&
                                                    mbar_test(&ctrl->k_full[ks], kpar) &&
                                                    (jk > wk.j0 || mbar_test(&ctrl->q_full, qpar)))) {
                        tc_fence_after_sync();
                        const uint32_t s_col = tmem + kColS + (g & 1u) * kKeys;
                        const uint64_t b = k_desc + ((ks * kSlotBytes) >> 4);
                        if (ks2 > 0) {
                            for (int ch = 0; ch < 9; ++ch)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_ss(lead, s_col, q_desc + ch * chunk + kk * 2, b + ch * 64 + kk * 2,
                                           idesc_s, ch + kk > 0 ? 1u : 0u);
                        } else {  // the tile's halves are the ring's last slot and its first
                            for (int ch = 0; ch < 9; ++ch)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    mma_ss(lead, s_col, q_desc + ch * chunk + kk * 2, b + ch * 64 + kk * 2,
                                           idesc_h, ch + kk > 0 ? 1u : 0u);
                                    mma_ss(lead, s_col + 32, q_desc + ch * chunk + kk * 2,
                                           k_desc + ch * 64 + kk * 2, idesc_h, ch + kk > 0 ? 1u : 0u);
                                }
                        }
                        commit(lead, &ctrl->s_full[g & 1u]);
                        ++g;
                        ks = ks2 + 1 == n_slots ? 0 : ks2 + 1;
                        if (ks < 2) kpar ^= 1u;
                        if (++jk == wk.j1) {
                            commit(lead, &ctrl->q_empty);
                            qpar ^= 1u;
                            wk.next(p);
                            jk = wk.j0;
                        }
                        did = true;
                    }
                }
                if (did) {
                    n_idle = 0;
                    continue;
                }
                // nothing is ready: wait, with the limit of every wait
                if (n_idle++ == 0) since = globaltimer_ns();
                if ((n_idle & 63u) == 0) {
                    const bool late = globaltimer_ns() - since > kWaitLimitNs;
                    if (late) {
                        atomicOr(&ctrl->bad, CPA_DEV_TIMEOUT);
                        ctrl->abort_flag = 1u;
                        __threadfence_block();
                    }
                    if (__any_sync(0xffffffffu, late || ctrl->abort_flag)) break;
                }
            }
            commit(lead, &ctrl->mma_done);
            if (!wait_warp(&ctrl->mma_done, 0, ctrl)) mbar_drain(&ctrl->mma_done, 0);
        } else {
            // ============================== softmax and output
            // Scores: rows 16 warp + lane / 4 (a) and 8 more (b), columns 8 i + 2 (lane % 4) and
            // the next.  Outputs: columns 128 blk + 32 warp + lane, a row per TMEM column.
            const uint32_t lanes = (uint32_t)(warp * 32) << 16;
            const int ra = warp * 16 + (lane >> 2), rb = ra + 8;
            uint32_t g = 0, pieces = 0;
            int vs = 0;  // slot of the tile's first half
            bool ok = true;
            for (; w.more(); w.next(p)) {
                const Rows r(p, w.pair * p.cl + rank);
                // the last key that a row sees; -1 for one that sees none, or is none
                const bool act_a = ra < r.n, act_b = rb < r.n;
                const int p_first = w.L - p.S + r.s0;
                const int pos_a = act_a ? max(p_first + ra / p.heads, -1) : -1;
                const int pos_b = act_b ? max(p_first + rb / p.heads, -1) : -1;
                float ma = ninf_f(), mb = ninf_f(), la = 0.f, lb = 0.f;  // (l: this lane's columns)
                // (the unit before has been read, and the first tile's barrier comes before what is
                // marked here)
                if (threadIdx.x == 0) ctrl->odd = 0;
                for (int j = w.j0; j < w.j1; ++j, ++g) {
                    const int key0 = j * kKeys;
                    ok = ok && wait_warp(&ctrl->s_full[g & 1u], (g >> 1) & 1u, ctrl);
                    uint32_t s[32];
                    float ta = ninf_f(), tb = ninf_f();
                    bool need_a = false, need_b = false;
                    if (ok) {
                        tc_fence_after_sync();
                        tmem_ld_16x256_x8(tmem + lanes + kColS + (g & 1u) * kKeys, s);
                        if (key0 + kKeys - 1 > p_first) {
                            const int c = key0 + 2 * (lane & 3);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    if (c + 8 * i + e > pos_a) s[4 * i + e] = 0xff800000u;
                                    if (c + 8 * i + e > pos_b) s[4 * i + 2 + e] = 0xff800000u;
                                }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            ta = fmax3(ta, __uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1]));
                            tb = fmax3(tb, __uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3]));
                        }
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, o));
                            tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, o));
                        }
                        ta *= p.scale_log2;
                        tb *= p.scale_log2;
                        need_a = act_a && ma != ninf_f() && ta > ma + kRescale;
                        need_b = act_b && mb != ninf_f() && tb > mb + kRescale;
                    }
                    if (!bar_and(1, 128, ok && !need_a && !need_b)) {
                        // O holds the tiles before this one when PV of the last is done
                        ok = ok && wait_warp(&ctrl->pv_done, (g - 1) & 1u, ctrl);
                        const float fa = need_a ? ex2(ma - ta) : 1.f, fb = need_b ? ex2(mb - tb) : 1.f;
                        if ((lane & 3) == 0) {
                            ctrl->row[ra] = fa;
                            ctrl->row[rb] = fb;
                        }
                        la *= fa;
                        lb *= fb;
                        if (need_a) ma = ta;
                        if (need_b) mb = tb;
                        ok = bar_and(1, 128, ok);
                        if (!ok) break;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c0 = 0; c0 < 4 * kRows; c0 += 8) {
                            if ((c0 & (kRows - 1)) >= rows_n) continue;
                            uint32_t v[8];
                            tmem_ld_x8(tmem + lanes + c0, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) *
                                                       ctrl->row[(c0 & (kRows - 1)) + i]);
                            tmem_st_x8_nowait(tmem + lanes + c0, v);
                        }
                        tmem_wait_st();
                        tc_fence_before_sync();
                        bar_and(1, 128, true);  // (the factors may be written again)
                    }
                    if (ma == ninf_f()) ma = ta;
                    if (mb == ninf_f()) mb = tb;
                    const float xa = ma == ninf_f() ? 0.f : ma, xb = mb == ninf_f() ? 0.f : mb;
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e0 = ex2(fmaf(__uint_as_float(s[4 * i]), p.scale_log2, -xa));
                        const float e1 = ex2(fmaf(__uint_as_float(s[4 * i + 1]), p.scale_log2, -xa));
                        const float e2 = ex2(fmaf(__uint_as_float(s[4 * i + 2]), p.scale_log2, -xb));
                        const float e3 = ex2(fmaf(__uint_as_float(s[4 * i + 3]), p.scale_log2, -xb));
                        la += e0 + e1;
                        lb += e2 + e3;
                        // (a weight's rounding of 2^-9 is of the size of the output's own; the
                        // sum is of the unrounded weights in 32 bits)
                        pk[2 * i] = pack_bf16x2(e0, e1);
                        pk[2 * i + 1] = pack_bf16x2(e2, e3);
                    }
                    // the weights' buffer is free, and so is what the products of this tile's
                    // scores read, when PV of the tile before is done
                    if (g > 0) ok = ok && wait_warp(&ctrl->pv_done, (g - 1) & 1u, ctrl);
                    // box bi of the tile, in its half's slot
                    const int vs2 = vs + 1 == n_slots ? 0 : vs + 1;
                    auto box_at = [&](int bi) -> uint8_t* {
                        return smem + o_k + (bi < 4 ? vs : vs2) * kSlotBytes + (bi & 3) * kBox;
                    };
                    if (key0 + kKeys > w.L) {
                        // slots past the sequence's end: a piece of 16 bytes of a row each
                        const int first = max(w.L - key0, 0);
                        for (int i = threadIdx.x + 64 * first; i < 64 * kKeys; i += 128) {
                            const int k = i >> 6, c = i & 63;
                            *reinterpret_cast<uint4*>(box_at(k >> 3) + (c >> 3) * 1024 + (k & 7) * 128 +
                                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (p.S > 1 && key0 + kKeys - 1 > p_first) {
                        // keys that not every row sees: a warp each
                        for (int k = max(key0, p_first + 1) + warp; k < min(key0 + kKeys, w.L); k += 4) {
                            bool odd = false;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint4* at = reinterpret_cast<uint4*>(
                                    box_at((k - key0) >> 3) + ((lane >> 3) + 4 * i) * 1024 +
                                    ((k - key0) & 7) * 128 + (lane & 7) * 16);
                                uint32_t x[4] = {at->x, at->y, at->z, at->w};
                                bool here = false;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((x[e] & 0x7F80u) == 0x7F80u) x[e] &= 0xFFFF0000u, here = true;
                                    if ((x[e] & 0x7F800000u) == 0x7F800000u) x[e] &= 0xFFFFu, here = true;
                                }
                                if (here) *at = make_uint4(x[0], x[1], x[2], x[3]);
                                odd |= here;
                            }
                            if (__any_sync(0xffffffffu, odd) && lane == 0)
                                atomicOr(&ctrl->odd, 1ull << (k - (w.L - p.S + 1)));
                        }
                    }
                    if (warp * 16 < rows_n) {
                        uint8_t* const dst = smem + o_p + (lane & 3) * 4;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            *reinterpret_cast<uint32_t*>(dst + ra * 128 + ((i ^ (ra & 7)) << 4)) = pk[2 * i];
                            *reinterpret_cast<uint32_t*>(dst + rb * 128 + ((i ^ (rb & 7)) << 4)) = pk[2 * i + 1];
                        }
                    }
                    vs = vs2 + 1 == n_slots ? 0 : vs2 + 1;
                    fence_proxy_async_smem();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctrl->p_full);
                }

                // ---- output: the rows, or their part of a unit cut by the range
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    la += __shfl_xor_sync(0xffffffffu, la, o);
                    lb += __shfl_xor_sync(0xffffffffu, lb, o);
                }
                const bool split = w.j0 > 0 || w.j1 < w.nt;
                const size_t slot = 2 * (size_t)blockIdx.x + (w.j0 > 0 ? 0 : 1);
                const size_t row0 = (size_t)w.b * p.S * p.H + r.first;  // of the output
                float* const part_l = p.part_lse + slot * kRows;
                if ((lane & 3) == 0) {
                    ctrl->row[ra] = la == 0.f ? 0.f : 1.f / la;
                    ctrl->row[rb] = lb == 0.f ? 0.f : 1.f / lb;
                    const float za = la == 0.f ? ninf_f() : ma + lg2(la);
                    const float zb = lb == 0.f ? ninf_f() : mb + lg2(lb);
                    if (act_a && ok) (split ? part_l : p.lse + row0)[ra] = split || la == 0.f ? za : za * kLn2;
                    if (act_b && ok) (split ? part_l : p.lse + row0)[rb] = split || lb == 0.f ? zb : zb * kLn2;
                }
                ok = ok && wait_warp(&ctrl->o_full, pieces & 1u, ctrl);
                ++pieces;
                ok = bar_and(1, 128, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const unsigned long long odd = ctrl->odd;
                const int col0 = warp * 32 + lane;
#pragma unroll 1
                for (int x0 = 0; x0 < r.n; x0 += 8) {
                    uint32_t v[4][8];
                    tmem_ld_4x8(tmem + lanes + x0, kRows, v);
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = ctrl->row[x0 + i];
                    if (split) {
                        float* out = p.part_o + (slot * kRows + x0) * kC + col0;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (x0 + i < r.n)
#pragma unroll
                                for (int blk = 0; blk < 4; ++blk)
                                    out[i * kC + blk * 128] = __uint_as_float(v[blk][i]) * f[i];
                    } else {
                        // two lanes exchange: an even one writes two columns of row x, an odd one
                        // of row x + 1
                        const bool up = lane & 1;
                        uint32_t* out = reinterpret_cast<uint32_t*>(p.o + (row0 + x0 + (up ? 1 : 0)) * kC) +
                                        (col0 >> 1);
#pragma unroll
                        for (int i = 0; i < 8; i += 2)
#pragma unroll
                            for (int blk = 0; blk < 4; ++blk) {
                                const float y0 = __uint_as_float(v[blk][i]) * f[i];
                                const float y1 = __uint_as_float(v[blk][i + 1]) * f[i + 1];
                                const float z = __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 1);
                                if (x0 + i + (up ? 1 : 0) < r.n)
                                    out[i * (kC / 2) + blk * 64] =
                                        up ? pack_bf16x2(z, y1) : pack_bf16x2(y0, z);
                            }
                    }
                }
                if (odd) {
                    // values that are not finite, to the rows that see them: a warp's own columns
                    // (the rows' values above are this warp's, but not all of them this lane's)
                    __threadfence_block();
                    __syncwarp();
                    for (unsigned long long m = odd; m; m &= m - 1) {
                        const int i = __ffsll((long long)m) - 1, k = w.L - p.S + 1 + i;
                        if (k < w.j0 * kKeys || k >= w.j1 * kKeys) continue;
                        const int pg = __ldg(p.table + (size_t)w.b * p.stride + (k >> p.lp));
                        if (pg < 0 || pg >= p.num_pages) continue;
                        const size_t at = (((size_t)pg << p.lp) + (k & ((1 << p.lp) - 1))) * kSlot;
                        for (int blk = 0; blk < 4; ++blk) {
                            const int col = blk * 128 + warp * 32 + lane;
                            if (isfinite(__bfloat162float(p.pages[at + col]))) continue;
                            const float nan = __int_as_float(0x7fffffff);
                            // token i + 1 of the request is at position k
                            for (int x = max(0, (i + 1 - r.s0) * p.heads); x < r.n; ++x) {
                                if (split)
                                    p.part_o[(slot * kRows + x) * kC + col] = nan;
                                else
                                    p.o[(row0 + x) * kC + col] = __float2bfloat16(nan);
                            }
                        }
                    }
                }
                tc_fence_before_sync();  // O may be written again
                bar_and(1, 128, true);   // (and so may the factors and the mask)
                if (lane == 0) mbar_arrive(&ctrl->o_empty);
            }
        }
    }

    if (bad) atomicOr(&ctrl->bad, bad);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (warp == 4 && lane == 0) {
        if (rank == 0 && !p.by_unit) p.desc[grp] = desc;
        p.bad[blockIdx.x] = ctrl->bad;
    }
}

// Joins the units that ranges cut: a unit's parts are the second slots of the group where it
// starts and the first slots of the groups after it, in that order.  Block (x, y) of the grid:
// entry x of desc, some of its rows, a warp for F * 128 columns of a row; the last x gathers the
// status word.  What a join takes is the latency of its loads, 16 / F parts at a time, and the
// launch of its blocks.
constexpr int kJoinWarps = 8;
constexpr int join_rows(int F) { return kJoinWarps * F / 4; }
template <int F>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const __grid_constant__ LatentParams p) {
    constexpr int kAtATime = 16 / F;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_for_earlier();
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y > 0) return;
        __shared__ uint32_t all;
        if (threadIdx.x == 0) all = 0;
        __syncthreads();
        uint32_t bad = 0;
        for (int i = threadIdx.x; i < p.n_cta; i += kJoinWarps * 32) bad |= __ldcg(p.bad + i);
        if (bad) atomicOr(&all, bad);
        __syncthreads();
        if (threadIdx.x == 0) *p.status = all;
        return;
    }
    const int rank = blockIdx.x % p.cl;
    const int4 d = __ldcg(p.desc + blockIdx.x / p.cl);
    if (!join_in_range(d.x, d.y, d.z, d.w, p.B, p.n_pairs, p.n_grp)) return;
    const Rows r(p, d.y * p.cl + rank);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, np = d.z;
    const int x = blockIdx.y * join_rows(F) + warp * F / 4;
    const int at4 = (warp * F & 3) * 32 + lane;  // float4 of the row
    if (x >= r.n) return;
    auto row_of = [&](int i) -> size_t {
        return (2 * ((size_t)(d.w + i) * p.cl + rank) + (i == 0 ? 1 : 0)) * kRows + x;
    };
    float m = ninf_f(), sum = 0.f;
    float4 acc[F];
#pragma unroll
    for (int k = 0; k < F; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < np; i0 += kAtATime) {
        float4 y[kAtATime][F];
        float z[kAtATime], mx = m;
#pragma unroll
        for (int i = 0; i < kAtATime; ++i) {
            const size_t at = row_of(min(i0 + i, np - 1));
            z[i] = __ldcg(p.part_lse + at);
#pragma unroll
            for (int k = 0; k < F; ++k)
                if (i0 + i < np) y[i][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kC) + 32 * k + at4);
        }
#pragma unroll
        for (int i = 0; i < kAtATime; ++i)
            if (i0 + i < np) mx = fmaxf(mx, z[i]);
        const float ref = mx == ninf_f() ? 0.f : mx, f = ex2(m - ref);
        sum *= f;
#pragma unroll
        for (int k = 0; k < F; ++k) {
            acc[k].x *= f;
            acc[k].y *= f;
            acc[k].z *= f;
            acc[k].w *= f;
        }
#pragma unroll
        for (int i = 0; i < kAtATime; ++i) {
            if (i0 + i >= np) break;
            const float w = ex2(z[i] - ref);
            sum += w;
#pragma unroll
            for (int k = 0; k < F; ++k) {
                acc[k].x += w * y[i][k].x;
                acc[k].y += w * y[i][k].y;
                acc[k].z += w * y[i][k].z;
                acc[k].w += w * y[i][k].w;
            }
        }
        m = mx;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t row = (size_t)d.x * p.S * p.H + r.first + x;
#pragma unroll
    for (int k = 0; k < F; ++k)
        reinterpret_cast<uint2*>(p.o + row * kC)[32 * k + at4] =
            make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                       pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (at4 == 0)
        p.lse[row] = sum == 0.f ? ninf_f() : ((m == ninf_f() ? 0.f : m) + lg2(sum)) * kLn2;
}

struct LatentWs {
    size_t bad, desc, part_lse, part_o, total;
};
LatentWs latent_ws(int n_cta) {
    LatentWs w;
    w.bad = kStatusBytes;
    w.desc = align_up(w.bad + (size_t)n_cta * 4, 256);
    w.part_lse = align_up(w.desc + (size_t)n_cta * 16, 256);
    w.part_o = align_up(w.part_lse + (size_t)2 * n_cta * kRows * 4, 256);
    w.total = align_up(w.part_o + (size_t)2 * n_cta * kRows * kC * 4, 256);
    return w;
}

// The pool seen as (64 columns, slot, chunk of 64 columns): boxes of eight slots, whole.
bool make_boxes_map(CUtensorMap* map, const void* base, uint64_t slots) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, slots, kSlot / 64};
    cuuint64_t strides[2] = {kSlot * 2, 128};
    cuuint32_t box[3] = {64, 8, kSlot / 64};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t raise_smem_once() {
    static PerDevice<int> state;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return (cudaError_t)state.run(dev, (int)cudaErrorInvalidDevice, [](int&) {
        return (int)cudaFuncSetAttribute(latent_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kMaxSmem);
    });
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_latent_decode_workspace_size(int B, int S, int H, int latent_dim, int rope_dim,
                                        int page_size) {
    if (B < 1 || S < 1 || S > kMaxTokens || H < 1 || latent_dim != kC || rope_dim != kR ||
        !page_size_ok(page_size))
        return 0;
    const int n_sm = sm_count();
    return n_sm <= 0 ? 0 : latent_ws(n_sm).total;
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
    if (latent_dim != kC || rope_dim != kR || !page_size_ok(page_size) || S > kMaxTokens)
        return CPA_ERR_UNSUPPORTED;
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
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    const LatentWs w = latent_ws(n_sm);
    if (workspace_bytes < w.total) return CPA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    LatentParams p = {};
    p.pages = static_cast<const __nv_bfloat16*>(pages);
    p.table = page_table;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.bad = reinterpret_cast<uint32_t*>(ws + w.bad);
    p.desc = reinterpret_cast<int4*>(ws + w.desc);
    p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    p.part_o = reinterpret_cast<float*>(ws + w.part_o);
    p.stride = pt_stride;
    p.B = B;
    p.S = S;
    p.H = H;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_len = max_seq_len;
    p.n_ht = (H + kRows - 1) / kRows;
    p.heads = (H + p.n_ht - 1) / p.n_ht;
    p.toks = p.n_ht > 1 ? 1 : kRows / H;
    if (p.toks > S) p.toks = S;
    p.n_rt = (S + p.toks - 1) / p.toks * p.n_ht;
    p.cl = p.n_rt % 2 == 0 && n_sm % 2 == 0 ? 2 : 1;
    p.n_pairs = p.n_rt / p.cl;
    p.n_cta = n_sm;
    p.n_grp = n_sm / p.cl;
    const long long units = (long long)B * p.n_pairs;
    p.by_unit = units <= p.n_grp;
    p.scale_log2 = sm_scale * kLog2e;
    if (!make_heads_map(&p.cmap, q_c, kC, H, (uint64_t)B * S, qc_head_stride, qc_token_stride, p.heads,
                        p.toks) ||
        !make_heads_map(&p.rmap, q_r, kR, H, (uint64_t)B * S, qr_head_stride, qr_token_stride, p.heads,
                        p.toks) ||
        !make_boxes_map(&p.kmap, pages, (uint64_t)num_pages * page_size))
        return CPA_ERR_CUDA;
    if (raise_smem_once() != cudaSuccess) return CPA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int rows = p.heads * p.toks;
    p.n_slots = slots_of(rows);
    const uint32_t smem = off_k(rows) + (uint32_t)p.n_slots * kSlotBytes + 1024;
    if (launch_overlapped(latent_kernel, dim3((unsigned)p.n_cta), kThreads, smem, s, p) !=
        cudaSuccess)
        return CPA_ERR_LAUNCH;
    // A unit has about n_grp / units parts: where they are many they are read many at a time, by
    // more warps (one request of 777 tokens 14.5 -> 10.2 us; 64 units of three parts 39.7 -> 41.1).
    const bool many = units * 4 <= p.n_grp;
    const int per_block = many ? join_rows(1) : join_rows(4);
    const dim3 grid((unsigned)((p.by_unit ? (int)units : p.n_grp) * p.cl + 1),
                    (unsigned)((rows + per_block - 1) / per_block));
    const cudaError_t e = many ? launch_overlapped(latent_join_kernel<1>, grid, kJoinWarps * 32, 0, s, p)
                               : launch_overlapped(latent_join_kernel<4>, grid, kJoinWarps * 32, 0, s, p);
    return e == cudaSuccess ? CPA_OK : CPA_ERR_LAUNCH;
}

}  // extern "C"
