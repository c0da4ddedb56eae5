// cpa_cache.cu -- the page operations of the cache: fork, free, copy pages,
// compact.  Forking and freeing work on block tables and page counts alone;
// copying and compacting move K and V of one layer's pools and are bound by
// HBM (every byte moved is read once and written once).
#include <cuda_runtime.h>
#include <stdint.h>

#include "cpa.h"
#include "cpa_checks.h"
#include "cpa_launch.cuh"

namespace cpa {
namespace {

constexpr int kForkThreads = 256;
constexpr int kChunkPages = 1024;  // pages of a chunk of the free-page map
constexpr int kChunkWords = kChunkPages / 32;

// Exclusive prefix sum of one value per thread over a block of kForkThreads;
// `total` is the block's sum.  `ws` holds one value per warp.
__device__ __forceinline__ int scan_block(int v, int* ws, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kForkThreads / 32; ++w) {
        if (w < warp) base += ws[w];
        total += ws[w];
    }
    __syncthreads();
    return base + x - v;
}

// ---------------------------------------------------------------- fork
// A fork runs as two kernels: this one takes down which pages are free (a bit
// per page, and a count per chunk of 1024 pages, a block each with one load a lane
// in flight per word) before the second changes any count, so that every child
// finds its page without waiting for another.  The second is launched while the
// first runs and waits for it on the device.
__global__ void __launch_bounds__(kForkThreads)
    free_map_kernel(const int32_t* __restrict__ refcounts, int num_pages, uint32_t* map,
                    int32_t* chunk_free, uint32_t* status) {
    __shared__ int ws[kForkThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0u;
    constexpr int kPerWarp = kChunkWords / (kForkThreads / 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long base = (long long)blockIdx.x * kChunkPages;
    int count[kPerWarp], mine = 0;
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        const long long pg = base + (warp * kPerWarp + i) * 32 + lane;
        count[i] = pg < num_pages ? __ldg(refcounts + pg) : 1;
    }
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
        const uint32_t bits = __ballot_sync(0xffffffffu, count[i] == 0);
        if (lane == 0) {
            map[(size_t)blockIdx.x * kChunkWords + warp * kPerWarp + i] = bits;
            mine += __popc(bits);
        }
    }
    int total;
    scan_block(mine, ws, total);
    if (threadIdx.x == 0) chunk_free[blockIdx.x] = total;
}

struct ForkParams {
    int32_t* table;
    int32_t* lens;
    const int32_t* parents;
    const int32_t* children;
    int32_t* refcounts;
    int32_t* copy_src;
    int32_t* copy_dst;
    const uint32_t* map;         // written by the kernel before (not through the
    const int32_t* chunk_free;   // read-only cache)
    uint32_t* status;
    int stride, n_rows, n, P, num_pages, n_chunks;
};

// Tokens of the last, partly filled page of pair j's parent: 0 where there is
// none (or the pair names no valid parent).
__device__ __forceinline__ int tail_of(const ForkParams& p, int j) {
    const int r = __ldg(p.parents + j);
    if (r < 0 || r >= p.n_rows) return 0;
    const int L = p.lens[r];
    if (L < 0 || L > (long long)p.stride * p.P) return 0;
    return L % p.P;
}

// One block per child.  A child that takes a page takes the free page whose
// rank is the number of earlier pairs with a partly filled page, so the pages
// given out do not depend on the order in which blocks run.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkParams p) {
    __shared__ int ws[kForkThreads / 32];
    __shared__ int found;
    const int i = blockIdx.x, tid = threadIdx.x;
    // (what the first kernel does not write is read before it is done)
    const int r = __ldg(p.parents + i), c = __ldg(p.children + i);
    bool ok = r >= 0 && r < p.n_rows && c >= 0 && c < p.n_rows;
    // is this child named twice, or a parent of this call?
    bool twice = false;
    for (int j = tid; j < p.n; j += kForkThreads)
        twice |= (j != i && __ldg(p.children + j) == c) || __ldg(p.parents + j) == c;
    ok = !__syncthreads_or(twice || !ok);
    // nothing is changed before the map is complete
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!ok) {
        if (tid == 0) {
            flag(p.status, CPA_DEV_BAD_ROW);
            p.copy_src[i] = -1;
            p.copy_dst[i] = -1;
        }
        return;
    }
    const int L = p.lens[r];
    if (L < 0 || L > (long long)p.stride * p.P) {
        if (tid == 0) {
            flag(p.status, CPA_DEV_BAD_LENGTH);
            p.copy_src[i] = -1;
            p.copy_dst[i] = -1;
        }
        return;
    }
    const int whole = L / p.P;
    const bool tail = L % p.P != 0;
    int fresh = -1;
    if (tail) {
        int before = 0;
        for (int j = tid; j < i; j += kForkThreads) before += tail_of(p, j) != 0;
        int rank;
        scan_block(before, ws, rank);
        // the chunk that holds the free page of that rank, then the page
        if (tid == 0) found = -1;
        __syncthreads();
        int passed = 0, chunk = -1;
        for (int k0 = 0; k0 < p.n_chunks && chunk < 0; k0 += kForkThreads) {
            const int k = k0 + tid;
            const int v = k < p.n_chunks ? __ldcg(p.chunk_free + k) : 0;
            int sum;
            const int at = passed + scan_block(v, ws, sum);
            if (at <= rank && rank < at + v) found = k;
            __syncthreads();
            chunk = found;
            if (chunk < 0) passed += sum;
            // (the pages of the chunks before `chunk` within this step)
            if (chunk >= 0) {
                int prior;
                scan_block(k < chunk ? v : 0, ws, prior);
                passed += prior;
            }
        }
        __syncthreads();
        if (tid == 0) found = -1;
        __syncthreads();
        if (chunk >= 0) {
            const int want = rank - passed;
            const uint32_t bits =
                tid < kChunkWords ? __ldcg(p.map + (size_t)chunk * kChunkWords + tid) : 0u;
            int sum;
            const int at = scan_block(__popc(bits), ws, sum);
            if (at <= want && want < at + __popc(bits)) {
                uint32_t b = bits;
                for (int k = at; k < want; ++k) b &= b - 1u;
                found = chunk * kChunkPages + tid * 32 + __ffs((int)b) - 1;
            }
            __syncthreads();
        }
        fresh = found;
    }
    const int32_t* from = p.table + (size_t)r * p.stride;
    int32_t* to = p.table + (size_t)c * p.stride;
    bool bad = false;
    for (int k = tid; k < p.stride; k += kForkThreads) {
        int e = -1;
        if (k < whole) {
            e = from[k];
            if (e < -1 || e >= p.num_pages) {
                bad = true;
                e = -1;
            } else if (e >= 0) {  // (-1: a page that the parent gave back)
                atomicAdd(p.refcounts + e, 1);
            }
        } else if (k == whole && tail) {
            e = fresh;
        }
        to[k] = e;
    }
    if (bad) flag(p.status, CPA_DEV_BAD_PAGE);
    if (tid == 0) {
        p.lens[c] = L;
        int src = -1;
        if (fresh >= 0) {
            p.refcounts[fresh] = 1;
            src = from[whole];
            if (src < 0 || src >= p.num_pages) {
                flag(p.status, CPA_DEV_BAD_PAGE);
                src = -1;
            }
        } else if (tail) {
            flag(p.status, CPA_DEV_NO_PAGE);
        }
        p.copy_src[i] = src;
        p.copy_dst[i] = src >= 0 ? fresh : -1;
    }
}

// ---------------------------------------------------------------- free
// An entry is taken out of the table with an exchange, so that an entry named twice
// is given back once whatever the order.  Returns what was wrong.
__device__ __forceinline__ uint32_t give_back(int32_t* entry, int32_t* refcounts, int num_pages) {
    const int e = atomicExch(entry, -1);
    if (e == -1) return 0u;
    if (e < 0 || e >= num_pages) return CPA_DEV_BAD_PAGE;
    if (atomicSub(refcounts + e, 1) > 0) return 0u;
    atomicAdd(refcounts + e, 1);  // it stays as it was
    return CPA_DEV_BAD_COUNT;
}

__device__ __forceinline__ uint32_t range_bits(int r, int a, int b, int stride, int n_rows) {
    if (r < 0 || r >= n_rows) return CPA_DEV_BAD_ROW;
    return a < 0 || a > stride || b < 0 || b > stride ? CPA_DEV_BAD_LENGTH : 0u;
}

// One block per named range.
__global__ void __launch_bounds__(256)
    free_kernel(int32_t* table, int stride, int n_rows, const int32_t* __restrict__ rows,
                const int32_t* __restrict__ first, const int32_t* __restrict__ last,
                int32_t* refcounts, int num_pages, uint32_t* status) {
    const int i = blockIdx.x;
    const int r = __ldg(rows + i), a = __ldg(first + i), b = __ldg(last + i);
    wait_for_clear();
    uint32_t bad = range_bits(r, a, b, stride, n_rows);
    if (!bad) {
        int32_t* row = table + (size_t)r * stride;
        for (int k = a + threadIdx.x; k < b; k += blockDim.x)
            bad |= give_back(row + k, refcounts, num_pages);
    }
    if (bad) flag(status, bad);
}

// The same for a small call by one block, an entry a thread, which writes the status
// word as well.
constexpr int kFreeThreads = 1024;
__global__ void __launch_bounds__(kFreeThreads)
    free_small_kernel(int32_t* table, int stride, int n_rows, const int32_t* __restrict__ rows,
                      const int32_t* __restrict__ first, const int32_t* __restrict__ last, int n,
                      int32_t* refcounts, int num_pages, uint32_t* status) {
    __shared__ uint32_t all;
    if (threadIdx.x == 0) all = 0u;
    __syncthreads();
    const int i = threadIdx.x / stride, k = threadIdx.x - i * stride;
    if (i < n) {
        const int r = __ldg(rows + i), a = __ldg(first + i), b = __ldg(last + i);
        uint32_t bad = range_bits(r, a, b, stride, n_rows);
        if (!bad && k >= a && k < b)
            bad = give_back(table + (size_t)r * stride + k, refcounts, num_pages);
        if (bad) atomicOr(&all, bad);
    }
    __syncthreads();
    if (threadIdx.x == 0) *status = all;
}

// ---------------------------------------------------------------- copies
constexpr int kUnroll = 8;  // 16-byte loads that a lane has in flight

// A warp copies pieces of 4 KB: 8 loads of 16 bytes a lane, then the stores.
constexpr int kPieceBytes = 32 * 16 * kUnroll;

__global__ void __launch_bounds__(256)
    copy_pages_kernel(uint8_t* k_pages, uint8_t* v_pages, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int n, int num_pages, size_t page_bytes,
                      int pieces, uint32_t* status) {
    // the last block looks over all pairs and writes the status word; the others
    // pass over what is out of range
    if (blockIdx.x == gridDim.x - 1) {
        bool bad = false;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int s = __ldg(src + i), d = __ldg(dst + i);
            bad |= !(s == -1 && d == -1) && (s < 0 || s >= num_pages || d < 0 || d >= num_pages);
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *status = bad ? CPA_DEV_BAD_PAGE : 0u;
        return;
    }
    const int lane = threadIdx.x & 31;
    const long long n_items = (long long)n * 2 * pieces;
    const long long step = (long long)(gridDim.x - 1) * 8;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < n_items; it += step) {
        const int i = (int)(it / (2 * pieces)), rest = (int)(it - (long long)i * 2 * pieces);
        const int s = __ldg(src + i), d = __ldg(dst + i);
        if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) continue;
        uint8_t* pool = rest < pieces ? k_pages : v_pages;
        const size_t off = (size_t)(rest < pieces ? rest : rest - pieces) * kPieceBytes;
        const int n16 = (int)(((page_bytes - off < kPieceBytes) ? page_bytes - off : kPieceBytes) / 16);
        const uint4* from = reinterpret_cast<const uint4*>(pool + (size_t)s * page_bytes + off);
        uint4* to = reinterpret_cast<uint4*>(pool + (size_t)d * page_bytes + off);
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (u * 32 + lane < n16) x[u] = __ldcs(from + u * 32 + lane);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (u * 32 + lane < n16) __stcs(to + u * 32 + lane, x[u]);
    }
}

struct CompactParams {
    uint8_t* k_pages;
    uint8_t* v_pages;
    const int32_t* src_table;
    const int32_t* src_rows;
    const int32_t* src_pos;
    const int32_t* n_keep;
    const int32_t* dst_table;
    const int32_t* dst_start;
    uint32_t* status;
    int src_stride, n_src_rows, dst_stride, max_keep, B, lp, num_pages;
    int token16;  // 16-byte units of a token's K (or V)
    int status_block;  // the last block looks over the whole call and writes the status word
};

// The source row of request b and its count; false where they are out of range.
// What is wrong goes to `bad`.
__device__ __forceinline__ bool compact_row(const CompactParams& p, int b, int& row, int& keep,
                                            uint32_t& bad) {
    row = p.src_rows ? __ldg(p.src_rows + b) : b;
    keep = __ldg(p.n_keep + b);
    if (row < 0 || row >= p.n_src_rows) {
        bad |= CPA_DEV_BAD_ROW;
        return false;
    }
    if (keep < 0 || keep > p.max_keep) {
        bad |= CPA_DEV_BAD_LENGTH;
        return false;
    }
    return true;
}

// Token slot (index into a pool's tokens) of position pos of a table row; -1 where
// it is out of range.
__device__ __forceinline__ long long slot_of(const CompactParams& p, const int32_t* row,
                                             int stride, long long pos, uint32_t& bad) {
    if (pos < 0 || pos >= ((long long)stride << p.lp)) {
        bad |= CPA_DEV_BAD_LENGTH;
        return -1;
    }
    const int pg = __ldg(row + (pos >> p.lp));
    if (pg < 0 || pg >= p.num_pages) {
        bad |= CPA_DEV_BAD_PAGE;
        return -1;
    }
    return ((long long)pg << p.lp) + (pos & ((1 << p.lp) - 1));
}

// Source and destination slot of token i of request b; false where there is none.
__device__ __forceinline__ bool compact_item(const CompactParams& p, int b, int i, long long& s,
                                             long long& d, uint32_t& bad) {
    int row, keep;
    if (!compact_row(p, b, row, keep, bad) || i >= keep) return false;
    s = slot_of(p, p.src_table + (size_t)row * p.src_stride, p.src_stride,
                __ldg(p.src_pos + (size_t)b * p.max_keep + i), bad);
    d = slot_of(p, p.dst_table + (size_t)b * p.dst_stride, p.dst_stride,
                (long long)__ldg(p.dst_start + b) + i, bad);
    return s >= 0 && d >= 0;
}

// From one table to another: no slot is both read and written, so every token
// is on its own.  A warp moves one token's K and V at a time.
__global__ void __launch_bounds__(256, 4) compact_kernel(CompactParams p) {
    const int lane = threadIdx.x & 31;
    const long long n_items = (long long)p.B * p.max_keep;
    uint32_t bad = 0;
    if (p.status_block && blockIdx.x == gridDim.x - 1) {
        __shared__ uint32_t all;
        if (threadIdx.x == 0) all = 0u;
        __syncthreads();
        long long s, d;
        for (int it = threadIdx.x; it < n_items; it += 256)
            compact_item(p, it / p.max_keep, it % p.max_keep, s, d, bad);
        if (bad) atomicOr(&all, bad);
        __syncthreads();
        if (threadIdx.x == 0) *p.status = all;
        return;
    }
    if (!p.status_block) wait_for_clear();
    const long long step = (long long)(gridDim.x - p.status_block) * 8;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < n_items; it += step) {
        long long s, d;
        const int b = (int)(it / p.max_keep);
        if (!compact_item(p, b, (int)(it - (long long)b * p.max_keep), s, d, bad)) continue;
        const size_t from = (size_t)s * p.token16, to = (size_t)d * p.token16;
        const uint4* ks = reinterpret_cast<const uint4*>(p.k_pages) + from;
        const uint4* vs = reinterpret_cast<const uint4*>(p.v_pages) + from;
        uint4* kd = reinterpret_cast<uint4*>(p.k_pages) + to;
        uint4* vd = reinterpret_cast<uint4*>(p.v_pages) + to;
        for (int e0 = lane; e0 < p.token16; e0 += 32 * kUnroll / 2) {
            uint4 x[kUnroll / 2], y[kUnroll / 2];
#pragma unroll
            for (int u = 0; u < kUnroll / 2; ++u)
                if (e0 + u * 32 < p.token16) {
                    x[u] = __ldcs(ks + e0 + u * 32);
                    y[u] = __ldcs(vs + e0 + u * 32);
                }
#pragma unroll
            for (int u = 0; u < kUnroll / 2; ++u)
                if (e0 + u * 32 < p.token16) {
                    __stcs(kd + e0 + u * 32, x[u]);
                    __stcs(vd + e0 + u * 32, y[u]);
                }
        }
    }
    if (bad && !p.status_block && lane == 0) flag(p.status, bad);
}

// Within one row: positions only move down (dst_start + i <= src_pos[i], both
// ascending), so a slot that token i overwrites was read for a token at or
// before i.  A thread owns 16 bytes of every token and walks the tokens in
// order, 8 at a time, reads before writes: no two threads share a byte.
__global__ void __launch_bounds__(128) compact_in_place_kernel(CompactParams p) {
    const int b = blockIdx.x;
    const int e = blockIdx.y * blockDim.x + threadIdx.x;
    int row, keep;
    uint32_t bad = 0;
    wait_for_clear();
    if (e >= 2 * p.token16) return;
    if (!compact_row(p, b, row, keep, bad)) {
        flag(p.status, bad);
        return;
    }
    const bool v = e >= p.token16;
    uint4* pool = v ? reinterpret_cast<uint4*>(p.v_pages) + (e - p.token16)
                    : reinterpret_cast<uint4*>(p.k_pages) + e;
    const int32_t* trow = p.src_table + (size_t)row * p.src_stride;
    const int32_t* pos = p.src_pos + (size_t)b * p.max_keep;
    const long long start = __ldg(p.dst_start + b);
    long long prev = start - 1;
    for (int i0 = 0; i0 < keep; i0 += kUnroll) {
        uint4 x[kUnroll];
        long long to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            to[u] = -1;
            if (i0 + u >= keep) continue;
            const long long a = __ldg(pos + i0 + u);
            // ascending from dst_start - 1 on: then src_pos[i] >= dst_start + i
            if (a <= prev) {
                bad |= CPA_DEV_BAD_LENGTH;
                continue;
            }
            prev = a;
            const long long s = slot_of(p, trow, p.src_stride, a, bad);
            const long long d = slot_of(p, trow, p.src_stride, start + i0 + u, bad);
            if (s < 0 || d < 0) continue;
            x[u] = pool[s * p.token16];
            to[u] = d;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] >= 0) pool[to[u] * p.token16] = x[u];
    }
    if (bad) flag(p.status, bad);
}

struct ForkWs {
    size_t chunk_free, map, total;
    int n_chunks;
};
ForkWs fork_ws(int num_pages) {
    ForkWs w;
    w.n_chunks = (num_pages + kChunkPages - 1) / kChunkPages;
    w.chunk_free = kStatusBytes;
    w.map = align_up(w.chunk_free + (size_t)w.n_chunks * 4, 256);
    w.total = w.map + align_up((size_t)w.n_chunks * kChunkWords * 4, 512);
    return w;
}

bool rows_ok(int pt_stride, int n_rows) {
    return pt_stride >= 1 && n_rows >= 1;
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" {

size_t cpa_cache_fork_workspace_size(int num_pages) {
    return num_pages < 1 ? 0 : fork_ws(num_pages).total;
}

cpa_status cpa_cache_fork(int32_t* page_table, int pt_stride, int n_rows, int32_t* seq_lens,
                          const int32_t* parents, const int32_t* children, int n,
                          int32_t* refcounts, int page_size, int num_pages, int32_t* copy_src,
                          int32_t* copy_dst, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream) {
    if (!page_table || !seq_lens || !refcounts || n < 0 || num_pages < 1 ||
        !rows_ok(pt_stride, n_rows))
        return CPA_ERR_INVALID_ARG;
    if (n > 0 && (!parents || !children || !copy_src || !copy_dst)) return CPA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size)) return CPA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    const ForkWs w = fork_ws(num_pages);
    if (!workspace || workspace_bytes < w.total) return CPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return CPA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) return clear_status(workspace, s);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ForkParams p;
    p.table = page_table;
    p.lens = seq_lens;
    p.parents = parents;
    p.children = children;
    p.refcounts = refcounts;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.chunk_free = reinterpret_cast<int32_t*>(ws + w.chunk_free);
    p.map = reinterpret_cast<uint32_t*>(ws + w.map);
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.stride = pt_stride;
    p.n_rows = n_rows;
    p.n = n;
    p.P = page_size;
    p.num_pages = num_pages;
    p.n_chunks = w.n_chunks;
    free_map_kernel<<<w.n_chunks, kForkThreads, 0, s>>>(
        refcounts, num_pages, reinterpret_cast<uint32_t*>(ws + w.map),
        reinterpret_cast<int32_t*>(ws + w.chunk_free), p.status);
    const cpa_status st = launched();
    if (st != CPA_OK) return st;
    return launch_dependent(fork_kernel, dim3((unsigned)n), kForkThreads, s, p);
}

cpa_status cpa_cache_free(int32_t* page_table, int pt_stride, int n_rows, const int32_t* rows,
                          const int32_t* first, const int32_t* last, int n, int32_t* refcounts,
                          int num_pages, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream) {
    if (!page_table || !refcounts || n < 0 || num_pages < 1 || !rows_ok(pt_stride, n_rows))
        return CPA_ERR_INVALID_ARG;
    if (n > 0 && (!rows || !first || !last)) return CPA_ERR_INVALID_ARG;
    const cpa_status st = status_ws(workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) return clear_status(workspace, s);
    uint32_t* const status = static_cast<uint32_t*>(workspace);
    // One launch in place of two, which is what a small call waits for: 4 sequences of 49
    // pages 8.9 -> 7.2 us called from Python (on the device 2.1 -> 2.2; 1024 entries 2.1 -> 2.7).
    if ((long long)n * pt_stride <= kFreeThreads) {
        const int threads = (n * pt_stride + 31) / 32 * 32;
        free_small_kernel<<<1, threads, 0, s>>>(page_table, pt_stride, n_rows, rows, first, last,
                                                n, refcounts, num_pages, status);
        return launched();
    }
    return launch_cleared(free_kernel, dim3((unsigned)n), 256, s, status, page_table, pt_stride,
                          n_rows, rows, first, last, refcounts, num_pages, status);
}

cpa_status cpa_cache_copy_pages(void* k_pages, void* v_pages, const int32_t* copy_src,
                                const int32_t* copy_dst, int n, int num_pages,
                                size_t page_bytes, void* workspace, size_t workspace_bytes,
                                cpa_stream_t stream) {
    if (!k_pages || !v_pages || n < 0 || num_pages < 1 || page_bytes < 16 || page_bytes % 16)
        return CPA_ERR_INVALID_ARG;
    if (n > 0 && (!copy_src || !copy_dst)) return CPA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages)) return CPA_ERR_INVALID_ARG;
    if (page_bytes > ((size_t)1 << 30)) return CPA_ERR_UNSUPPORTED;
    const cpa_status st = status_ws(workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) return clear_status(workspace, s);
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    const int pieces = (int)((page_bytes + kPieceBytes - 1) / kPieceBytes);
    long long blocks = ((long long)n * 2 * pieces + 7) / 8;
    if (blocks > (long long)n_sm * 8) blocks = (long long)n_sm * 8;
    copy_pages_kernel<<<(unsigned)blocks + 1, 256, 0, s>>>(
        static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages), copy_src, copy_dst, n,
        num_pages, page_bytes, pieces, static_cast<uint32_t*>(workspace));
    return launched();
}

cpa_status cpa_cache_compact(void* k_pages, void* v_pages, const int32_t* src_table,
                             int src_stride, int n_src_rows, const int32_t* src_rows,
                             const int32_t* src_pos, int max_keep, const int32_t* n_keep,
                             const int32_t* dst_table, int dst_stride, const int32_t* dst_start,
                             int B, int page_size, int num_pages, size_t token_bytes,
                             void* workspace, size_t workspace_bytes, cpa_stream_t stream) {
    if (!k_pages || !v_pages || !src_table || !n_keep || !dst_start || B < 1 || max_keep < 0 ||
        num_pages < 1 || !rows_ok(src_stride, n_src_rows) || token_bytes < 16 || token_bytes % 16)
        return CPA_ERR_INVALID_ARG;
    if ((max_keep > 0 && !src_pos) || (dst_table && dst_stride < 1)) return CPA_ERR_INVALID_ARG;
    if (!src_rows && n_src_rows < B) return CPA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages)) return CPA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size) || token_bytes > ((size_t)1 << 20)) return CPA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > (1ll << 31)) return CPA_ERR_UNSUPPORTED;
    const cpa_status st = status_ws(workspace, workspace_bytes);
    if (st != CPA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (max_keep == 0) return clear_status(workspace, s);
    const int n_sm = sm_count();
    if (n_sm <= 0) return CPA_ERR_CUDA;
    CompactParams p;
    // A block more looks a small call over and writes the status word (64 requests of up
    // to 6 tokens: 3.6 -> 3.0 us against clear_kernel); a large one has each warp
    // report into a cleared word, because one block would be looking long after the
    // others are done.
    p.status_block = dst_table && (long long)B * max_keep <= 4096 ? 1 : 0;
    p.k_pages = static_cast<uint8_t*>(k_pages);
    p.v_pages = static_cast<uint8_t*>(v_pages);
    p.src_table = src_table;
    p.src_rows = src_rows;
    p.src_pos = src_pos;
    p.n_keep = n_keep;
    p.dst_table = dst_table;
    p.dst_start = dst_start;
    p.status = static_cast<uint32_t*>(workspace);
    p.src_stride = src_stride;
    p.n_src_rows = n_src_rows;
    p.dst_stride = dst_stride;
    p.max_keep = max_keep;
    p.B = B;
    p.lp = 31 - __builtin_clz((unsigned)page_size);
    p.num_pages = num_pages;
    p.token16 = (int)(token_bytes / 16);
    if (!dst_table) {
        const dim3 grid((unsigned)B, (unsigned)((2 * p.token16 + 127) / 128));
        return launch_cleared(compact_in_place_kernel, grid, 128, s, p.status, p);
    }
    // a warp per token, in more blocks than run at a time: those of short requests end
    // at once (78.3 us with 4 blocks an SM, 72.1 with 8, 71.3 with 64, for 400 MB read
    // and written)
    long long blocks = ((long long)B * max_keep + 7) / 8;
    if (blocks > (long long)n_sm * 64) blocks = (long long)n_sm * 64;
    const dim3 grid((unsigned)blocks + p.status_block);
    if (!p.status_block) return launch_cleared(compact_kernel, grid, 256, s, p.status, p);
    compact_kernel<<<grid, 256, 0, s>>>(p);
    return launched();
}

}  // extern "C"
