/*
 * cpa.h -- C ABI of the cascade paged-attention library (libcpa.so) for
 * GB300 (sm_103a).
 *
 * The method.  For one query q and a key set split into disjoint parts A and
 * B, attention over A and over B can be computed separately and merged
 * exactly by their log-sum-exp values ("Cascade attention" page,
 * zdszero.github.io/cascade_attention.html, section on the split property):
 *     LSE = log(e^LSE_A + e^LSE_B),  o = e^(LSE_A-LSE) o_A + e^(LSE_B-LSE) o_B.
 * In tree speculative-decoding verify, request b holds a prefix of L_b cached
 * tokens and topk branches of S draft tokens each; draft s of branch k
 * attends the whole prefix plus drafts 0..s of its own branch (same page,
 * "Topk > 1").  Cascade reads the shared prefix once per request (Pass A, all
 * topk*S draft queries of the request together), each branch's own drafts
 * once (Pass B) and merges the two.  Naive expand instead runs B*topk
 * independent requests over L_b + S keys each and so reads every prefix topk
 * times (same page, "Naive Expand").  The same split covers prefill after a
 * prefix-cache hit of H tokens: the M = N - H suffix queries attend the
 * cached prefix (an M x H rectangle) and each other causally (a triangle),
 * merged the same way ("Causal Attention ... KV hit area" page, sections 2-3).
 *
 * Conventions shared by every call.
 *   - Data types: q, k_pages, v_pages and bf16 outputs are bfloat16 (2 bytes);
 *     lse and fp32 outputs are float.  head_dim must be 128.
 *   - Paged KV pool (KV-cache tutorial, sections 5.2-5.3): k_pages and
 *     v_pages are [num_pages, page_size, H_kv, head_dim], row-major.  Logical
 *     position pos of a sequence with block table `tab` is page
 *     tab[pos / page_size], slot pos % page_size.  Slots past a sequence's
 *     end are never used: their contents may be anything, NaN included.
 *   - Grouped-query attention: query head h reads KV head h / (H_q / H_kv)
 *     (repeat_interleave grouping, tutorial section 6.3).  H_q / H_kv must be
 *     a power of two no larger than 128.
 *   - Verify token order: q and o are [B*topk*S, H_q, head_dim] and lse is
 *     [B*topk*S, H_q]; token t = (b*topk + k)*S + s is draft s of branch k of
 *     request b.
 *   - lse is the natural-log log-sum-exp of the scaled scores over the keys a
 *     row sees; a row that sees no key gets lse = -inf and o = 0.
 *   - Pointers passed as `const void*` / `void*` / `float*` / `int32_t*` are
 *     DEVICE pointers (16-byte aligned for q, k_pages, v_pages, o) unless a
 *     comment says host.  The caller owns every buffer, including the
 *     workspace; the library never allocates, frees or synchronises (except
 *     cpa_get_device_status and cpa_noalloc_device_status, which say so).
 *     Calls are asynchronous on `stream` (NULL = legacy default stream) and
 *     launch nothing when they return an error, except the calls that launch
 *     two kernels (cpa_cascade_verify_shared when its shared prefix ends inside
 *     a page, the cpa_decode calls, cpa_window_prefill, cpa_cache_fork,
 *     cpa_cache_free where n * pt_stride is above 1024, cpa_cache_compact in
 *     place or where B * max_keep is above 4096, cpa_latent_decode,
 *     cpa_latent_prefill with a memset before them in a call of many units, the
 *     appends and gathers where B is above 8192 or T / page_size above 16384):
 *     they check every argument
 *     before the first, so only CPA_ERR_LAUNCH or CPA_ERR_CUDA from the second
 *     launch can follow a launch already made.
 *   - Errors: arguments that can be checked on the host return a status
 *     before any launch.  Problems only the GPU can see (a page id outside
 *     [0, num_pages), a prefix length outside [0, max_prefix_len], a pipeline
 *     wait that exceeded its time limit) set bits in a status word at the
 *     start of the workspace, which cpa_get_device_status reads.  Each
 *     workspace-taking call clears that word and the merge counters it uses
 *     (an asynchronous memset or kernel on `stream`) or has its kernels write
 *     the word whole.  Nothing crosses the ABI as an exception, and no kernel
 *     traps, asserts or prints.
 *   - When the device status word has any bit set after a call, that call's
 *     outputs are undefined (they may be partial, stale or computed from a
 *     truncated mask) unless the call says what they are; only the status word
 *     is meaningful.
 *   - A workspace must not be used by two calls that can run at the same time.
 */
#ifndef CPA_H_
#define CPA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* A CUDA stream (cudaStream_t / CUstream). */
typedef struct CUstream_st* cpa_stream_t;

typedef enum cpa_status {
    CPA_OK = 0,
    CPA_ERR_INVALID_ARG = 1,  /* bad pointer, size, stride or shape */
    CPA_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels implement */
    CPA_ERR_WORKSPACE = 3,    /* workspace missing or too small */
    CPA_ERR_LAUNCH = 4,       /* a kernel launch failed */
    CPA_ERR_BAD_PAGE = 5,     /* device saw a page id outside [0, num_pages) */
    CPA_ERR_TIMEOUT = 6,      /* device pipeline wait exceeded its limit */
    CPA_ERR_CUDA = 7,         /* a CUDA runtime call failed */
    CPA_ERR_BAD_LENGTH = 8,   /* device saw a prefix length outside [0, max_prefix_len] */
    CPA_ERR_BAD_TREE = 9,     /* device saw a tree parent index outside [-1, i) */
    CPA_ERR_BAD_ROW = 10,     /* device saw a table row out of range, or named twice */
    CPA_ERR_NO_PAGE = 11,     /* the pool had fewer free pages than were asked for */
    CPA_ERR_BAD_COUNT = 12    /* a page was given back more often than it was taken */
} cpa_status;

/* Bits of the device status word (first 4 bytes of a workspace). */
#define CPA_DEV_BAD_PAGE 0x1u
#define CPA_DEV_TIMEOUT 0x2u
#define CPA_DEV_BAD_LENGTH 0x4u
#define CPA_DEV_BAD_TREE 0x8u
#define CPA_DEV_BAD_ROW 0x10u
#define CPA_DEV_NO_PAGE 0x20u
#define CPA_DEV_BAD_COUNT 0x40u

/* Largest draft tree cpa_tree_verify accepts (one 64-bit ancestor mask per node). */
#define CPA_MAX_TREE_NODES 64

/* Which part of the prefix-hit prefill to compute (cpa_prefill_hit). */
#define CPA_PREFILL_FULL 0 /* rectangle + triangle, merged; o is bf16 */
#define CPA_PREFILL_RECT 1 /* keys 0..H-1 only; o is fp32 */
#define CPA_PREFILL_TRI 2  /* keys H..H+i only; o is fp32 */

/* Human-readable name of a status code (static string). */
const char* cpa_status_string(cpa_status status);

/*
 * Bytes of workspace cpa_cascade_verify, cpa_cascade_pass_a and
 * cpa_naive_expand_verify need for these sizes on the current device.  The
 * workspace holds the device status word, one merge counter per work unit
 * and the fp32 partial results of work units that are split across CTAs.
 * Returns 0 for sizes the calls would reject.
 */
size_t cpa_cascade_verify_workspace_size(int B, int topk, int S, int H_q, int H_kv, int head_dim,
                                         int page_size);

/*
 * Cascade verify attention (the whole hot path): Pass A + Pass B + merge.
 *   q                  bf16 [B*topk*S, H_q, head_dim]
 *   k_pages, v_pages   bf16 [num_pages, page_size, H_kv, head_dim]
 *   prefix_page_table  int32 [B, prefix_pt_stride]: request b's prefix pages
 *                      ("metadata.page_table" of the cascade page); entries
 *                      past ceil(L_b / page_size) are not read.
 *   draft_page_table   int32 [B*topk, draft_pt_stride]: branch (b, k)'s draft
 *                      pages ("forward_metadata_spec_decode_expand.page_table");
 *                      draft j is at logical position j of its branch.
 *   prefix_lens        int32 [B] on the device: L_b >= 0 ("cache_seqlens").
 *   max_prefix_len     host-side upper bound of every L_b; prefix_pt_stride
 *                      must be >= ceil(max_prefix_len / page_size).
 *   sm_scale           softmax scale (> 0), normally 1/sqrt(head_dim).
 *   o                  bf16 [B*topk*S, H_q, head_dim] output.
 *   lse                fp32 [B*topk*S, H_q] output (natural log).
 * Supported: head_dim 128; page_size in {8,16,32,64,128,256}; 1 <= S <= 16
 * and S <= page_size (a branch's drafts share its first draft page);
 * topk <= 16 when S <= 8, topk <= 8 when S > 8 (the branches' draft blocks of
 * 8 or 16 rows fill one 128-key tile); topk*S*(H_q/H_kv) <= 256.
 */
cpa_status cpa_cascade_verify(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* prefix_page_table, int prefix_pt_stride,
                              const int32_t* draft_page_table, int draft_pt_stride,
                              const int32_t* prefix_lens, int B, int topk, int S, int H_q,
                              int H_kv, int head_dim, int page_size, int num_pages,
                              int max_prefix_len, float sm_scale, void* o, float* lse,
                              void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * Naive-expand verify: the comparison baseline.  Same arguments and result
 * as cpa_cascade_verify, but every branch (b, k) is run as its own request
 * over its L_b + S logical keys (prefix pages, then its own draft pages), so
 * each prefix is read topk times: B*topk*(L+S) KV tokens in total (cascade
 * page, "Naive Expand").  Supported: S*(H_q/H_kv) <= 256, S <= 16,
 * S <= page_size.  Workspace: cpa_cascade_verify_workspace_size.
 */
cpa_status cpa_naive_expand_verify(const void* q, const void* k_pages, const void* v_pages,
                                   const int32_t* prefix_page_table, int prefix_pt_stride,
                                   const int32_t* draft_page_table, int draft_pt_stride,
                                   const int32_t* prefix_lens, int B, int topk, int S, int H_q,
                                   int H_kv, int head_dim, int page_size, int num_pages,
                                   int max_prefix_len, float sm_scale, void* o, float* lse,
                                   void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * Pass A alone (cascade page, first segment): every draft query of request b
 * against the request's prefix keys 0..L_b-1, read once per request.
 *   o_a   fp32 [B*topk*S, H_q, head_dim];  lse_a fp32 [B*topk*S, H_q].
 * A request with L_b = 0 gives o_a = 0, lse_a = -inf.
 */
cpa_status cpa_cascade_pass_a(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* prefix_page_table, int prefix_pt_stride,
                              const int32_t* prefix_lens, int B, int topk, int S, int H_q,
                              int H_kv, int head_dim, int page_size, int num_pages,
                              int max_prefix_len, float sm_scale, float* o_a, float* lse_a,
                              void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * Pass B alone (cascade page, second segment): B*topk virtual requests; draft
 * s of branch (b, k) against that branch's drafts 0..s, one warp per
 * (branch, query head) with a warp-level online softmax.
 *   o_b   fp32 [B*topk*S, H_q, head_dim];  lse_b fp32 [B*topk*S, H_q].
 * The workspace only needs to hold the status word: at least
 * cpa_status_workspace_size() bytes.  Supported: head_dim 128.
 */
cpa_status cpa_cascade_pass_b(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* draft_page_table, int draft_pt_stride, int B,
                              int topk, int S, int H_q, int H_kv, int head_dim, int page_size,
                              int num_pages, float sm_scale, float* o_b, float* lse_b,
                              void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/* Bytes of workspace that hold only the device status word. */
size_t cpa_status_workspace_size(void);

/*
 * merge_state (cascade page): for each of n_tokens*H rows,
 *   lse = log(e^lse_a + e^lse_b),  o = e^(lse_a-lse) o_a + e^(lse_b-lse) o_b,
 * computed about max(lse_a, lse_b) so nothing overflows; a -inf side
 * contributes nothing and two -inf sides give o = 0, lse = -inf.
 *   o_a, o_b  fp32 [n_tokens, H, head_dim];  lse_a, lse_b fp32 [n_tokens, H]
 *   o_out     bf16 [n_tokens, H, head_dim];  lse_out fp32 [n_tokens, H]
 * Supported: head_dim a multiple of 4 and at most 512.
 */
cpa_status cpa_merge_state(const float* o_a, const float* lse_a, const float* o_b,
                           const float* lse_b, int n_tokens, int H, int head_dim, void* o_out,
                           float* lse_out, cpa_stream_t stream);

/*
 * Cascade verify over FP8 KV pages (KV-cache tutorial, section 4.5 "FP8 KV":
 * half the bytes of bf16, with a per-tensor or per-channel scale).  Same
 * arguments, layout, token order and results as cpa_cascade_verify, except:
 *   k_pages, v_pages   uint8 [num_pages, page_size, H_kv, head_dim] E4M3 codes
 *                      (1 sign, 4 exponent bits with bias 7, 3 mantissa bits;
 *                      exponent 0 holds zero and subnormals); element value =
 *                      decoded code x scale.
 *   k_scale, v_scale   fp32 on the device: one value each when
 *                      scale_per_channel is 0, else [H_kv, head_dim] each
 *                      (one scale per KV head and channel).
 * q stays bf16 and o bf16, lse fp32.  The two NaN codes (0x7F, 0xFF) must not
 * appear in slots a row sees: they are read as +-480 x scale, not as NaN
 * (every other code is exact).  Slots past a sequence's end may hold any byte.
 * Arithmetic: codes are widened exactly to f16 on chip; q x k_scale is
 * rounded to f16 once (so |q x k_scale| must stay below 65504), P is f16,
 * accumulation fp32.  Supported: as for cpa_cascade_verify, and
 * topk*S*(H_q/H_kv) <= 128 (one M tile).  Workspace:
 * cpa_cascade_verify_workspace_size.
 */
cpa_status cpa_cascade_verify_fp8(const void* q, const void* k_pages, const void* v_pages,
                                  const float* k_scale, const float* v_scale,
                                  int scale_per_channel, const int32_t* prefix_page_table,
                                  int prefix_pt_stride, const int32_t* draft_page_table,
                                  int draft_pt_stride, const int32_t* prefix_lens, int B, int topk,
                                  int S, int H_q, int H_kv, int head_dim, int page_size,
                                  int num_pages, int max_prefix_len, float sm_scale, void* o,
                                  float* lse, void* workspace, size_t workspace_bytes,
                                  cpa_stream_t stream);

/*
 * Pass A alone over FP8 KV pages: cpa_cascade_pass_a's result (fp32 o_a,
 * lse_a) with the pools and scales of cpa_cascade_verify_fp8.
 */
cpa_status cpa_cascade_pass_a_fp8(const void* q, const void* k_pages, const void* v_pages,
                                  const float* k_scale, const float* v_scale,
                                  int scale_per_channel, const int32_t* prefix_page_table,
                                  int prefix_pt_stride, const int32_t* prefix_lens, int B,
                                  int topk, int S, int H_q, int H_kv, int head_dim, int page_size,
                                  int num_pages, int max_prefix_len, float sm_scale, float* o_a,
                                  float* lse_a, void* workspace, size_t workspace_bytes,
                                  cpa_stream_t stream);

/*
 * Bytes of workspace cpa_prefill_hit needs for these sizes on the current
 * device (0 for sizes it would reject).
 */
size_t cpa_prefill_hit_workspace_size(int B, int N, int H_hit, int H_q, int H_kv, int head_dim,
                                      int page_size);

/*
 * Prefill after a prefix-cache hit ("Causal Attention ... KV hit area"
 * page): B requests of N tokens whose first H_hit tokens were cached; the
 * KV of all N tokens is already in the paged pool.  Suffix token i (absolute
 * position H_hit + i) attends keys 0..H_hit+i: the rectangle 0..H_hit-1 and
 * the causal triangle H_hit..H_hit+i, merged by the LSE identity.
 *   q           bf16 [B*M, H_q, head_dim], M = N - H_hit, token b*M + i
 *   page_table  int32 [B, pt_stride], pt_stride >= ceil(N / page_size)
 *   part        CPA_PREFILL_FULL (o bf16), CPA_PREFILL_RECT or
 *               CPA_PREFILL_TRI (o fp32: the piece alone, for checking)
 *   o, lse      [B*M, H_q, head_dim] and fp32 [B*M, H_q]
 * Supported: head_dim 128, page_size in {8,...,256}, 0 <= H_hit <= N.
 */
cpa_status cpa_prefill_hit(const void* q, const void* k_pages, const void* v_pages,
                           const int32_t* page_table, int pt_stride, int B, int N, int H_hit,
                           int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                           float sm_scale, int part, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, cpa_stream_t stream);

/*
 * Bytes of workspace cpa_cascade_verify_shared needs for these sizes on the
 * current device (0 for sizes it would reject), for either of its schedules.
 * Besides the status word and merge scratch it holds the first level's fp32
 * partial result, B*topk*S*H_q*(head_dim + 1) floats.
 */
size_t cpa_cascade_verify_shared_workspace_size(int B, int n_groups, int topk, int S, int H_q,
                                                int H_kv, int head_dim, int page_size);

/*
 * Multi-level cascade verify.  Requests whose block tables begin with the
 * same physical pages share that prefix (KV-cache tutorial, block-table
 * example of section 5.3; share_prefix of section 6.2), e.g. one system
 * prompt for a whole batch.  The B requests form n_groups groups of
 * B/n_groups consecutive requests; each group has one shared prefix of
 * shared_len tokens, each request then its own prefix, each branch its own
 * drafts.  Draft s of branch k of request b sees the group's shared prefix,
 * request b's own prefix and drafts 0..s of branch k.  The shared prefix is
 * read from memory once per group:
 *   - shared_len a multiple of page_size: one launch of the fused cascade
 *     kernel; each request's prefix walk covers the group's shared pages and
 *     then its own, and the requests of a group, scheduled together, take the
 *     shared pages from L2 after the first read.
 *   - otherwise three levels merged by the cascade page's log-sum-exp
 *     identity: the shared prefix for all the group's draft queries at once
 *     (the tensor-core kernel in its rectangle mode, the group's queries as one
 *     block of suffix queries), then the own prefix once per request and the
 *     drafts once per branch (the fused cascade kernel), which merges.
 * Both give the same result up to rounding.
 *   shared_page_table  int32 [n_groups, shared_pt_stride]: the group's shared
 *                      pages; shared_pt_stride >= ceil(shared_len/page_size).
 *                      May be NULL when shared_len is 0.
 *   shared_len         host: shared prefix length of every group (>= 0).
 *   prefix_page_table, prefix_lens
 *                      each request's own prefix (the tokens after the shared
 *                      part), own position j at page row[j / page_size], slot
 *                      j % page_size; max_prefix_len bounds prefix_lens.
 *   other arguments    as for cpa_cascade_verify.
 * Supported: as for cpa_cascade_verify, and B a multiple of n_groups.
 */
cpa_status cpa_cascade_verify_shared(const void* q, const void* k_pages, const void* v_pages,
                                     const int32_t* shared_page_table, int shared_pt_stride,
                                     int n_groups, int shared_len,
                                     const int32_t* prefix_page_table, int prefix_pt_stride,
                                     const int32_t* draft_page_table, int draft_pt_stride,
                                     const int32_t* prefix_lens, int B, int topk, int S, int H_q,
                                     int H_kv, int head_dim, int page_size, int num_pages,
                                     int max_prefix_len, float sm_scale, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes,
                                     cpa_stream_t stream);

/*
 * Bytes of workspace cpa_tree_verify needs for these sizes on the current
 * device (0 for sizes it would reject): the status word and the merge
 * scratch of the attention kernel.
 */
size_t cpa_tree_verify_workspace_size(int B, int N, int H_q, int H_kv, int head_dim,
                                      int page_size);

/*
 * Verify over general draft trees (KV-cache tutorial, section 8.2 tip box
 * on tree attention, and Q14): request b holds a prefix of L_b cached tokens
 * and a draft tree of N nodes, flattened so that every parent comes before
 * its children (BFS order does).  Node i attends the whole prefix and the
 * tree nodes of A(i), its ancestors and itself: the mask M[i, j] = 1 iff j is
 * in A(i), the tree generalisation of the causal mask.  The chain-per-branch
 * case of cpa_cascade_verify is the forest of topk chains.  One launch: the
 * tensor-core kernel reads the prefix once per request for all N nodes (the
 * cascade page's Pass A) and takes the N tree nodes as one more tile of the
 * same online softmax, masked per row by the node's ancestor mask (built on
 * chip from the parent array), so the two parts are merged there.
 *   q                  bf16 [B*N, H_q, head_dim]; token b*N + i is node i of
 *                      request b.
 *   tree_page_table    int32 [B, tree_pt_stride]: node j of request b's tree
 *                      is at logical position j (page j / page_size, slot
 *                      j % page_size); tree_pt_stride >= ceil(N / page_size).
 *   tree_parents       int32 [B, N] on the device: the BFS index of node i's
 *                      parent, or -1 for a root (a node whose parent is the
 *                      last prefix token; several roots make a forest).  Each
 *                      parent index must be below its node's; the device
 *                      sets CPA_DEV_BAD_TREE where it is not.
 *   other arguments    as for cpa_cascade_verify (topk = 1, S = N).
 *   o, lse             bf16 [B*N, H_q, head_dim], fp32 [B*N, H_q].
 * Supported: head_dim 128; 1 <= N <= CPA_MAX_TREE_NODES;
 * N*(H_q/H_kv) <= 256; page sizes as for cpa_cascade_verify.
 */
cpa_status cpa_tree_verify(const void* q, const void* k_pages, const void* v_pages,
                           const int32_t* prefix_page_table, int prefix_pt_stride,
                           const int32_t* tree_page_table, int tree_pt_stride,
                           const int32_t* prefix_lens, const int32_t* tree_parents, int B, int N,
                           int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                           int max_prefix_len, float sm_scale, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * The tree part of cpa_tree_verify alone: node i of request b against the
 * tree nodes of A(i) only.  One CTA per (request, KV head) stages that
 * head's N tree K/V rows in shared memory; a warp then serves one node and
 * up to 4 query heads of the group at a time.  q needs 8-byte alignment,
 * k_pages, v_pages and o_b 16-byte alignment.
 *   o_b   fp32 [B*N, H_q, head_dim];  lse_b fp32 [B*N, H_q].
 * Workspace: at least cpa_status_workspace_size() bytes (the status word).
 * Supported: head_dim 128; 1 <= N <= CPA_MAX_TREE_NODES.
 */
cpa_status cpa_tree_pass_b(const void* q, const void* k_pages, const void* v_pages,
                           const int32_t* tree_page_table, int tree_pt_stride,
                           const int32_t* tree_parents, int B, int N, int H_q, int H_kv,
                           int head_dim, int page_size, int num_pages, float sm_scale,
                           float* o_b, float* lse_b, void* workspace, size_t workspace_bytes,
                           cpa_stream_t stream);

/*
 * Decode: attention of one new token per request over the paged cache.  Row b
 * of q is the token at position seq_lens[b] - 1; its own K/V is already in the
 * cache, as are those of every earlier token that it sees.  It sees key j when
 *     j < seq_lens[b]  and  (window == 0, or j >= seq_lens[b] - window,
 *                            or j < sinks):
 * all keys, or the last `window` (itself among them) and the first `sinks`.
 * Keys that are not seen are not read, nor are their table entries: the pages
 * a window has left behind may have been given back (cpa_cache_free).
 *   q           bf16 [B, H_q, head_dim]
 *   page_table  int32 [B, pt_stride], pt_stride >= ceil(max_seq_len / page_size)
 *   seq_lens    int32 [B] on the device, 0 <= seq_lens[b] <= max_seq_len; a
 *               request of length 0 gets o = 0, lse = -inf
 *   o, lse      bf16 [B, H_q, head_dim], fp32 [B, H_q]; not over any input
 * A NaN or an infinity in V reaches the requests that see it and no others; an
 * infinity stays one unless another of unlike sign meets it.
 * The work is split over the visible length and joined, in a fixed order: the
 * result of a call depends on its inputs and the device's SM count alone.
 * Supported: head_dim 128; page_size in {8,16,32,64,128,256}; any H_q that is a
 * multiple of H_kv; B * H_q up to 2^24; max_seq_len up to 2^30; k_pages and v_pages
 * 32-byte aligned.
 */
size_t cpa_decode_workspace_size(int B, int H_q, int H_kv, int head_dim, int page_size);

cpa_status cpa_decode(const void* q, const void* k_pages, const void* v_pages,
                      const int32_t* page_table, int pt_stride, const int32_t* seq_lens, int B,
                      int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                      int max_seq_len, int window, int sinks, float sm_scale, void* o, float* lse,
                      void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * Decode over FP8 E4M3 pages: cpa_decode with the pools and scales of
 * cpa_cascade_verify_fp8.  Codes are widened exactly to f16 (a NaN code that a
 * row sees gives NaN); q x k_scale is held as two f16 terms, so it must stay
 * below 65504 in magnitude; a weight is f16, to 2^-11 of itself down to 2^-21 of
 * the row's largest and to 2^-32 of that below; sums are fp32.
 */
cpa_status cpa_decode_fp8(const void* q, const void* k_pages, const void* v_pages,
                          const float* k_scale, const float* v_scale, int scale_per_channel,
                          const int32_t* page_table, int pt_stride, const int32_t* seq_lens,
                          int B, int H_q, int H_kv, int head_dim, int page_size, int num_pages,
                          int max_seq_len, int window, int sinks, float sm_scale, void* o,
                          float* lse, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream);

/*
 * Prefill of prompt chunks of unequal length, causal, with an optional sliding
 * window and sinks.  Request b has the new tokens q_start[b] .. q_start[b+1]-1
 * of q, m_b of them; they are the last m_b tokens of its sequence of
 * seq_lens[b] tokens, whose K/V (the new tokens' among them) is in the cache.
 * New token i is at position p = seq_lens[b] - m_b + i and sees key j when
 *     j <= p  and  (window == 0, or j > p - window, or j < sinks).
 * Pages that no new token sees are not read, nor are their table entries.
 *   q           bf16 [T, H_q, head_dim]
 *   page_table  int32 [B, pt_stride], pt_stride >= ceil(max_seq_len / page_size)
 *   q_start     int32 [B + 1] on the device, ascending, 0 <= q_start[0] and
 *               q_start[B] <= T; rows of o and lse before q_start[0] or at and
 *               past q_start[B] are left as they were
 *   seq_lens    int32 [B] on the device, m_b <= seq_lens[b] <= max_seq_len
 *   max_new     host-side upper bound of every m_b
 *   o, lse      bf16 [T, H_q, head_dim], fp32 [T, H_q]; not over any input
 * A q_start that is not ascending or leaves [0, T], an m_b above max_new or
 * above seq_lens[b], or a length above max_seq_len sets CPA_DEV_BAD_LENGTH.
 * A NaN or an infinity in V reaches the rows that see it and no others; a call
 * with many rows beside such values is exact, and slow.
 * Supported: head_dim 128; page_size in {8,16,32,64,128,256}; H_q / H_kv <= 128;
 * T * H_q up to 2^24; max_seq_len up to 2^30; o 32-byte aligned.
 */
size_t cpa_window_prefill_workspace_size(int B, int T, int H_q, int H_kv, int head_dim,
                                         int page_size, int max_new);

cpa_status cpa_window_prefill(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* page_table, int pt_stride, const int32_t* q_start,
                              const int32_t* seq_lens, int B, int T, int H_q, int H_kv,
                              int head_dim, int page_size, int num_pages, int max_new,
                              int max_seq_len, int window, int sinks, float sm_scale, void* o,
                              float* lse, void* workspace, size_t workspace_bytes,
                              cpa_stream_t stream);

/*
 * The page operations of the cache.  A page of the pool is free when its count
 * is 0: refcounts is int32 [num_pages] on the device, the number of table
 * entries that hold the page, and the caller keeps it (a page taken by the
 * caller's own means has count 1).  Tables and counts serve every layer, so
 * forking and freeing touch them alone; copying and compacting move K and V of
 * one layer's pools.
 *
 * cpa_cache_fork: sequence children[i] becomes a copy of sequence parents[i]
 * (rows of one page_table [n_rows, pt_stride] and of seq_lens [n_rows]).  The
 * parent's whole pages are shared, their counts raised by one each; entries of
 * -1 among them (pages that a window has left and that were given back) are -1
 * in the child's row too.  A last, partly filled page is not shared: the child
 * gets the lowest free page that no earlier i got, with count 1, and
 * (copy_src[i], copy_dst[i]) names the two pages, for cpa_cache_copy_pages to
 * copy in every layer.  Where there is nothing to copy both are -1.  Entries
 * past the child's last page become -1.  The entries that row children[i] held
 * before are not given back: free them first.
 *   parents, children  int32 [n] on the device.  A parent may have many
 *                      children; a child may not be named twice, nor be a
 *                      parent in the same call (CPA_DEV_BAD_ROW: such children
 *                      are left as they were, their pairs -1, and the page that
 *                      such an i would have got stays free and goes to no other).
 *                      So it is with a parent whose length is outside
 *                      [0, pt_stride * page_size] (CPA_DEV_BAD_LENGTH).
 *   copy_src, copy_dst int32 [n] on the device, output.
 * With too few free pages (CPA_DEV_NO_PAGE) the children that got none have -1
 * as their last page and their pair; all else is as described, so freeing the
 * row undoes the fork.  An entry of the parent that is no page id and not -1, or
 * a last, partly filled page that is -1, sets CPA_DEV_BAD_PAGE.  n may be 0.
 */
size_t cpa_cache_fork_workspace_size(int num_pages);

cpa_status cpa_cache_fork(int32_t* page_table, int pt_stride, int n_rows, int32_t* seq_lens,
                          const int32_t* parents, const int32_t* children, int n,
                          int32_t* refcounts, int page_size, int num_pages, int32_t* copy_src,
                          int32_t* copy_dst, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream);

/*
 * cpa_cache_free: for each i, entries first[i] .. last[i]-1 of row rows[i] are
 * given back: the page's count is lowered by one and the entry becomes -1.
 * Entries that are -1 already are passed over, so that naming an entry twice
 * gives it back once.  0 .. pt_stride frees a whole sequence; a window of W
 * tokens with S sinks over L tokens has left the pages ceil(S / page_size) ..
 * max(L - W, 0) / page_size behind (seq_lens does not change).  A count that is
 * 0 already stays 0 and sets CPA_DEV_BAD_COUNT; a bound outside [0, pt_stride]
 * sets CPA_DEV_BAD_LENGTH, a row outside [0, n_rows) CPA_DEV_BAD_ROW, and
 * nothing of that i is given back (first[i] >= last[i]: an empty range).
 * Workspace: cpa_status_workspace_size().
 */
cpa_status cpa_cache_free(int32_t* page_table, int pt_stride, int n_rows, const int32_t* rows,
                          const int32_t* first, const int32_t* last, int n, int32_t* refcounts,
                          int num_pages, void* workspace, size_t workspace_bytes,
                          cpa_stream_t stream);

/*
 * cpa_cache_copy_pages: page copy_dst[i] of both pools becomes a copy of page
 * copy_src[i], for each of the n pairs; pairs of two -1 are passed over.  No
 * page may be the destination of two pairs, nor the source of one and the
 * destination of another: the contents of such pages are undefined.  page_bytes
 * (one page of one pool) is a multiple of 16.  Workspace:
 * cpa_status_workspace_size().
 */
cpa_status cpa_cache_copy_pages(void* k_pages, void* v_pages, const int32_t* copy_src,
                                const int32_t* copy_dst, int n, int num_pages,
                                size_t page_bytes, void* workspace, size_t workspace_bytes,
                                cpa_stream_t stream);

/*
 * cpa_cache_compact: the kept tokens of a sequence move together.  For request
 * b and i < n_keep[b], K and V of position src_pos[b][i] of row src_rows[b] of
 * src_table move to position dst_start[b] + i of row b of dst_table.  After a
 * verify step that is how accepted drafts join the prefix: src_table the
 * draft (or tree) table, src_pos the accepted path, dst_table the prefix table
 * and dst_start the prefix lengths.
 *   src_table   int32 [n_src_rows, src_stride]
 *   src_rows    int32 [B] on the device, or NULL: row b
 *   src_pos     int32 [B, max_keep];  n_keep int32 [B], 0 <= n_keep[b] <= max_keep
 *   dst_table   int32 [B, dst_stride], or NULL: the move is within the source
 *               row, whose positions have to be ascending with dst_start[b] + i
 *               <= src_pos[b][i] (a history pruned in place); no row may be named
 *               twice, and a page that another sequence holds too changes for both
 *   dst_start   int32 [B] on the device
 *   token_bytes K (or V) of one token: H_kv x head_dim x element size, a
 *               multiple of 16
 * With a dst_table no slot may be both read and written by the call, or written
 * twice.  A row outside [0, n_src_rows) sets CPA_DEV_BAD_ROW; a count or
 * position outside its table, or one that breaks the order in place,
 * CPA_DEV_BAD_LENGTH.  Workspace: cpa_status_workspace_size().
 */
cpa_status cpa_cache_compact(void* k_pages, void* v_pages, const int32_t* src_table,
                             int src_stride, int n_src_rows, const int32_t* src_rows,
                             const int32_t* src_pos, int max_keep, const int32_t* n_keep,
                             const int32_t* dst_table, int dst_stride, const int32_t* dst_start,
                             int B, int page_size, int num_pages, size_t token_bytes,
                             void* workspace, size_t workspace_bytes, cpa_stream_t stream);

/*
 * Rows of new tokens written to the pages, and rows read back.
 *
 * cpa_cache_append: K and V of the new tokens of each request go to their slots.
 * Request b has the rows new_start[b] .. new_start[b+1]-1 of k_new and v_new, m_b
 * of them; they are the last m_b tokens of its sequence of seq_lens[b] tokens
 * (the new ones among them, as cpa_window_prefill takes it): row new_start[b] + i
 * goes to position seq_lens[b] - m_b + i.  Every other slot is left as it was.
 *   k_new, v_new  T rows of token_bytes, 16-byte aligned, k_stride_bytes and
 *                 v_stride_bytes apart (multiples of 16: rows may lie inside
 *                 wider ones, as those of a fused projection do)
 *   page_table    int32 [B, pt_stride]
 *   new_start     int32 [B + 1] on the device, ascending, 0 <= new_start[0] and
 *                 new_start[B] <= T; rows outside belong to no request
 *   seq_lens      int32 [B] on the device, m_b <= seq_lens[b] <= pt_stride * page_size
 *                 (and 2^30)
 *   token_bytes   K (or V) of one token: H_kv x head_dim x element size, a
 *                 multiple of 16 up to 2^20
 * No slot may be written twice by a call: a page that two sequences share takes new
 * tokens of one of them at most (cpa_cache_fork shares whole pages only).
 * A new_start that is not ascending or leaves [0, T] or a length out of range sets
 * CPA_DEV_BAD_LENGTH, a page id outside [0, num_pages) CPA_DEV_BAD_PAGE; such a
 * request's, or such a page's, tokens are not written, all others are (a request is
 * judged by its own start, end and length; a call whose starts do not ascend is slow).
 * T up to 2^30, T * token_bytes below 2^45.  Workspace: cpa_status_workspace_size().
 */
cpa_status cpa_cache_append(const void* k_new, const void* v_new, size_t k_stride_bytes,
                            size_t v_stride_bytes, void* k_pages, void* v_pages,
                            const int32_t* page_table, int pt_stride, const int32_t* new_start,
                            const int32_t* seq_lens, int B, int T, int page_size, int num_pages,
                            size_t token_bytes, void* workspace, size_t workspace_bytes,
                            cpa_stream_t stream);

/*
 * cpa_cache_append_fp8: bf16 rows of `channels` (H_kv x head_dim, a multiple of 16
 * up to 2^19) quantised into FP8 E4M3 pages, with the scales that
 * cpa_cascade_verify_fp8 and cpa_decode_fp8 read (fp32, one value or one per
 * channel): the code of x is x / scale in 32 bits, rounded to the nearest E4M3
 * value, ties to even, and cut at +-448 (infinities too); a NaN stays one.
 */
cpa_status cpa_cache_append_fp8(const void* k_new, const void* v_new, size_t k_stride_bytes,
                                size_t v_stride_bytes, void* k_pages, void* v_pages,
                                const float* k_scale, const float* v_scale, int scale_per_channel,
                                const int32_t* page_table, int pt_stride,
                                const int32_t* new_start, const int32_t* seq_lens, int B, int T,
                                int channels, int page_size, int num_pages, void* workspace,
                                size_t workspace_bytes, cpa_stream_t stream);

/*
 * cpa_cache_gather: rows of the cache as one contiguous array.  Request b's tokens
 * at positions first[b] .. first[b] + n_b - 1 go to rows out_start[b] ..
 * out_start[b+1]-1, n_b of them, of k_out and v_out (T rows of token_bytes each,
 * 16-byte aligned, not over any input).  first NULL: position 0.  Rows of no
 * request, and those whose request or page sets a bit of the status word (as for
 * cpa_cache_append, with first[b] + n_b in the place of the length), are left as
 * they were; one that starts that do not ascend give to two requests holds values of
 * theirs.  Workspace: cpa_status_workspace_size().
 */
cpa_status cpa_cache_gather(const void* k_pages, const void* v_pages, const int32_t* page_table,
                            int pt_stride, const int32_t* out_start, const int32_t* first, int B,
                            int T, int page_size, int num_pages, size_t token_bytes, void* k_out,
                            void* v_out, void* workspace, size_t workspace_bytes,
                            cpa_stream_t stream);

/* cpa_cache_gather_fp8: the same from FP8 E4M3 pages to bf16 rows: code x scale in 32
 * bits, rounded once (a NaN code gives NaN). */
cpa_status cpa_cache_gather_fp8(const void* k_pages, const void* v_pages, const float* k_scale,
                                const float* v_scale, int scale_per_channel,
                                const int32_t* page_table, int pt_stride,
                                const int32_t* out_start, const int32_t* first, int B, int T,
                                int channels, int page_size, int num_pages, void* k_out,
                                void* v_out, void* workspace, size_t workspace_bytes,
                                cpa_stream_t stream);

/*
 * Latent attention.  The keys and values of all heads come from one vector a token:
 * latent_dim elements c that every head's products expand, and rope_dim elements r
 * that carry the position and are part of every head's key as they are.  Head h has
 * the key [W_k,h c; r] and the value W_v,h c.  Two forms give the same attention:
 * absorbed (cpa_latent_decode: the queries go through W_k,h first and the outputs
 * through W_v,h afterwards, and attention is over the latents themselves) and
 * expanded (cpa_latent_prefill, over the products).  sm_scale is that of the expanded
 * head in both, (nope_dim + rope_dim)^-1/2 by custom.
 *
 * The cache of latents is one pool, bf16 [num_pages, page_size, latent_dim +
 * rope_dim], c first; the page operations take it as a pool of tokens of
 * 2 x (latent_dim + rope_dim) bytes.
 *
 * cpa_latent_append and cpa_latent_gather are cpa_cache_append and cpa_cache_gather
 * for that pool: the two parts come from, and go to, arrays of their own.
 */
cpa_status cpa_latent_append(const void* c_new, const void* r_new, size_t c_stride_bytes,
                             size_t r_stride_bytes, void* pages, const int32_t* page_table,
                             int pt_stride, const int32_t* new_start, const int32_t* seq_lens,
                             int B, int T, int latent_dim, int rope_dim, int page_size,
                             int num_pages, void* workspace, size_t workspace_bytes,
                             cpa_stream_t stream);

cpa_status cpa_latent_gather(const void* pages, const int32_t* page_table, int pt_stride,
                             const int32_t* out_start, const int32_t* first, int B, int T,
                             int latent_dim, int rope_dim, int page_size, int num_pages,
                             void* c_out, void* r_out, void* workspace, size_t workspace_bytes,
                             cpa_stream_t stream);

/*
 * cpa_latent_decode: S query tokens of each request against its paged latents.
 * Token s of request b is at position p = seq_lens[b] - S + s (S = 1: the newest
 * token; S > 1: a token and the drafts after it, whose latents are in the cache) and
 * sees the keys j <= p; with p < 0 it sees none.  Head h of it has the scores
 *     x_j = sm_scale (q_c . c_j + q_r . r_j)
 * and the output sum_j softmax(x)_j c_j, of latent_dim elements.
 *   q_c, q_r    bf16, element (t, h, i) at t * token_stride + h * head_stride + i
 *               for token t = b*S + s: latent_dim and rope_dim elements, strides in
 *               elements, multiples of 8 and positive (where there is more than one
 *               token, or head)
 *   page_table  int32 [B, pt_stride], pt_stride >= ceil(max_seq_len / page_size)
 *   seq_lens    int32 [B] on the device, 0 <= seq_lens[b] <= max_seq_len
 *   o, lse      bf16 [B*S, H, latent_dim] (32-byte aligned), fp32 [B*S, H]; not over
 *               any input
 * A NaN or an infinity in a latent reaches the rows that see it and no others.
 * The work is split over the visible length and joined, in a fixed order: the
 * result of a call depends on its inputs and the device's SM count alone.
 * Supported: latent_dim 512, rope_dim 64; page_size in {8,16,32,64,128,256};
 * S up to 64; B*S*H up to 2^22; max_seq_len up to 2^30.
 */
size_t cpa_latent_decode_workspace_size(int B, int S, int H, int latent_dim, int rope_dim,
                                        int page_size);

cpa_status cpa_latent_decode(const void* q_c, int64_t qc_token_stride, int64_t qc_head_stride,
                             const void* q_r, int64_t qr_token_stride, int64_t qr_head_stride,
                             const void* pages, const int32_t* page_table, int pt_stride,
                             const int32_t* seq_lens, int B, int S, int H, int latent_dim,
                             int rope_dim, int page_size, int num_pages, int max_seq_len,
                             float sm_scale, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, cpa_stream_t stream);

/*
 * cpa_latent_prefill: causal prefill of ragged prompt chunks over expanded latents,
 * which lie one after the other without pages.  Request b has the new tokens
 * q_start[b] .. q_start[b+1]-1 of q, m_b of them, and the keys and values
 * k_start[b] .. k_start[b+1]-1 of k_nope, k_rope and v, n_b >= m_b of them, the new
 * tokens' last; new token i sees the first n_b - m_b + i + 1 of them.
 *   q              bf16 [T, H, nope_dim + rope_dim], contiguous
 *   k_nope, v      bf16, element (j, h, i) at j * token_stride + h * head_stride + i,
 *                  strides in elements, multiples of 8 and positive: both may be slices
 *                  of one product [T_k, H, nope_dim + v_dim]
 *   k_rope         bf16 [T_k, rope_dim], rows rope_token_stride elements apart
 *   q_start, k_start  int32 [B + 1] on the device, ascending, within [0, T] and
 *                  [0, T_k]; rows of o and lse of no request are left as they were
 *   o, lse         bf16 [T, H, v_dim] (32-byte aligned), fp32 [T, H]; not over any input
 * A start that is not ascending or out of range, or an m_b above n_b, sets
 * CPA_DEV_BAD_LENGTH.  A NaN or an infinity in v reaches the rows that see it and no
 * others; a call with many rows beside such values is exact, and slow.
 * Supported: nope_dim 128, rope_dim 64, v_dim 128; T * H up to 2^24; T_k up to 2^30.
 */
size_t cpa_latent_prefill_workspace_size(int B, int T, int T_k, int H, int nope_dim, int rope_dim,
                                         int v_dim);

cpa_status cpa_latent_prefill(const void* q, const void* k_nope, int64_t k_token_stride,
                              int64_t k_head_stride, const void* k_rope, int64_t rope_token_stride,
                              const void* v, int64_t v_token_stride, int64_t v_head_stride,
                              const int32_t* q_start, const int32_t* k_start, int B, int T, int T_k,
                              int H, int nope_dim, int rope_dim, int v_dim, float sm_scale, void* o,
                              float* lse, void* workspace, size_t workspace_bytes,
                              cpa_stream_t stream);

/*
 * Read the device status word of `workspace` (written by the last call that
 * used it) into *status_out (host).  SYNCHRONISES `stream`.  Returns CPA_OK
 * when the word is 0, otherwise the status matching its most serious bit
 * (TIMEOUT, then BAD_ROW, BAD_PAGE, BAD_LENGTH, BAD_TREE, BAD_COUNT and
 * NO_PAGE).
 */
cpa_status cpa_get_device_status(const void* workspace, uint32_t* status_out,
                                  cpa_stream_t stream);

/*
 * Failure-detection check: launch one kernel that waits on a barrier nothing
 * will ever complete, with a wait limit of `limit_us` microseconds, so the
 * kernel gives up, sets CPA_DEV_TIMEOUT in the workspace status word and
 * returns.  Used by tests to exercise the bounded-wait path without hanging
 * the GPU.  Workspace: cpa_status_workspace_size() bytes.
 */
cpa_status cpa_debug_wait_timeout(void* workspace, size_t workspace_bytes, int limit_us,
                                  cpa_stream_t stream);

/*
 * Host-side view of the work partition the attention kernels use, for
 * tests: `total` tiles split over `n_ctas` CTAs, CTA c owning
 * [begin, end).  Returns the owner CTA of tile `tile` and fills begin/end
 * of CTA `cta` (host pointers).  Returns -1 on bad arguments, and -2 if the
 * two forms of the split arithmetic the kernels use (64-bit division, and
 * 32-bit division where total * n_ctas < 2^31) disagree, which they must not.
 */
int cpa_plan_partition(int64_t total, int n_ctas, int cta, int64_t tile, int64_t* begin,
                       int64_t* end);

/*
 * Static-scratch cascade verify: the same computation, arguments and
 * results as cpa_cascade_verify, but no workspace argument and no
 * allocation by anyone.  The source pages have no counterpart of this call;
 * it exists for callers that cannot call cudaMalloc.  Examples: an inference
 * engine that reserves nearly all HBM for its paged KV pool at start-up and
 * forbids later driver allocations (they would fail or fragment the pool);
 * a latency-critical decode loop that cannot pay for cudaMalloc's implicit
 * device-wide synchronisation; plugin code hosted by a framework that owns
 * every device buffer and hands the plugin no allocator.
 *
 * Scratch: a file-scope device array of CPA_STATIC_SCRATCH_BYTES, which every
 * GPU that loads this library holds until the process exits.  The scratch a
 * call needs is a fixed part that grows with the device's SM count (two fp32
 * partial-result slots of 256 rows x 128 columns per SM, about 262 KB per SM,
 * 40 MB on 152 SMs) plus 4 bytes per (request, KV head).  Sizes that need
 * more than the array are rejected with CPA_ERR_WORKSPACE before anything
 * is launched; so the usable shapes shrink as the SM count grows, and on a
 * part with more than about 180 SMs no shape fits.  Other invalid arguments
 * get the same status codes as cpa_cascade_verify.
 *
 * The first call on a device, with that device current, looks up the
 * array's device address (cudaGetSymbolAddress); make that first call
 * before any stream capture.  All calls on a device share the one array and
 * it keeps the last call's contents: each call clears the status word and
 * merge counters it needs (asynchronous memset on `stream`) before its
 * kernel runs.  Calls that overlap on the GPU (different streams, no
 * ordering between them) race on the array.
 *
 * Errors only the GPU can see (bad page id, bad prefix length, wait timeout)
 * go to the status word at the start of the array; read it with
 * cpa_noalloc_device_status.
 */
#define CPA_STATIC_SCRATCH_BYTES (48u * 1024u * 1024u)

cpa_status cpa_cascade_verify_noalloc(const void* q, const void* k_pages, const void* v_pages,
                                      const int32_t* prefix_page_table, int prefix_pt_stride,
                                      const int32_t* draft_page_table, int draft_pt_stride,
                                      const int32_t* prefix_lens, int B, int topk, int S, int H_q,
                                      int H_kv, int head_dim, int page_size, int num_pages,
                                      int max_prefix_len, float sm_scale, void* o, float* lse,
                                      cpa_stream_t stream);

/*
 * The device status word of the static scratch of the current device, as
 * written by the last cpa_cascade_verify_noalloc call on it, into
 * *status_out (host).  Same return values as cpa_get_device_status, and
 * like it SYNCHRONISES `stream`.  The source pages have no counterpart of
 * this call either.
 */
cpa_status cpa_noalloc_device_status(uint32_t* status_out, cpa_stream_t stream);

/* Library version, e.g. 100 for 0.1.0. */
int cpa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CPA_H_ */
