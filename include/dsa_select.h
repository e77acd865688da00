/*
 * dsa_select.h -- C ABI of the GB300 (sm_103a) DeepSeek-sparse-attention
 * indexer candidate-selection path.
 *
 * Given fp32 indexer logits [rows, W] and per-row [start, end) bounds, the
 * path
 *   1. scores every candidate block of B columns inside the row's live span
 *      [start, min(end, W)) by the block's maximum,
 *   2. takes the best Kb blocks (blocks past the span score -inf) and pins
 *      the block holding the newest token (column end - 1, which may lie past
 *      W),
 *   3. clamps each candidate's packed column start + b*B: inside the buffer
 *      it flags block b, past the buffer it sets the edge flag, which keeps
 *      column W - 1 only,
 *   4. writes -inf to every column of [0, min(end, W)) that is not kept and
 *      never writes a column at or past min(end, W),
 *   5. returns the best K column indices of the masked live span.
 * Sources: vLLM PR #57459, "[Perf][Attention] DSA candidate-block kernels walk
 * each row's live context", Summary; prhub report on vLLM PR #56628, "Stride
 * the DSA decode candidate mask over the live context", key source excerpts
 * (_mask_candidates_strided_kernel and _apply_candidate_mask_strided).
 *
 * Order: IEEE-754 totalOrder on the fp32 bit pattern (-NaN < -inf < ... <
 * -0 < +0 < ... < +inf < +NaN); among equal values the lower index wins.  All
 * results are exact (the path only compares and copies), so they match a
 * plain CPU definition bit for bit.
 *
 * Conventions for every call below:
 *   - Device pointers are CUDA device (or managed) addresses on the plan's
 *     device; the caller owns and allocates all of them.  The library owns
 *     only the host-side plan.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls only
 *     enqueue work: no host synchronisation, no allocation, no device
 *     attribute query, so they can be captured in a CUDA graph.  The launch
 *     grid depends on the plan (shapes) only; the work each CTA does follows
 *     the bounds in device memory, so a captured graph stays valid when the
 *     bounds change between replays.
 *   - A plan with rows == 0 makes every call a no-op returning DSA_OK; its
 *     pointers may then be NULL.
 *   - Every call returns a status code (below) and never aborts.  A launch
 *     failure is reported as DSA_ERR_CUDA; kernel faults surface, as usual
 *     for CUDA, at the next synchronising call.
 */
#ifndef DSA_SELECT_H
#define DSA_SELECT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t */

enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1, /* a NULL or misaligned pointer, a size out of range */
  DSA_ERR_UNSUPPORTED = 2, /* valid, but beyond what this build supports (e.g. shared memory) */
  DSA_ERR_CUDA = 3,        /* the CUDA runtime reported an error */
  DSA_ERR_TIMEOUT = 4      /* a bounded device-side wait gave up */
};

/* Static shape of one call site.  All sizes count fp32 elements. */
typedef struct dsa_select_cfg {
  int32_t rows;          /* R >= 0 rows of logits                                    */
  int32_t block_size;    /* B in [1, 4096]: columns per candidate block               */
  int64_t width;         /* W in [1, 2^31 - 1]: columns per row (buffer width)        */
  int64_t row_stride;    /* elements between rows; rows may not overlap               */
  int64_t col_stride;    /* elements between columns (>= 1; 2 = packed pairs)         */
  int32_t block_topk;    /* Kb in [1, 4096]: candidate blocks kept besides the pin    */
  int32_t row_topk;      /* K in [1, 4096]: column indices returned per row           */
  int32_t row_repeat;    /* rep >= 1: rows r read bound entry r / rep                 */
  int32_t repeat_causal; /* 1: end of row r = ends[r/rep] - (rep-1) + r % rep
                            0: every row of a group uses ends[r/rep] unchanged        */
  int32_t has_starts;    /* 0: start = 0 for every row; 1: starts[] is given          */
  int32_t split;         /* CTAs per row in the select kernels: 0 = automatic (from
                            rows, W and the SM count), else a power of two <= 16
                            (a thread-block cluster per row when > 1); reduced when
                            the device cannot schedule it.  32 .. 256 (a power of
                            two): a wide split -- each row is first streamed in
                            `split` parts, each keeping its top-Kb list in device
                            memory the plan owns, and a 16-CTA cluster per row then
                            merges them.  Automatic for very few rows of many
                            blocks: 64 parts when rows * 64 <= SMs, 128 when
                            rows * 128 <= SMs.  A plan with a wide split
                            must not run two calls at once (the lists are shared).  */
} dsa_select_cfg;

typedef struct dsa_select_plan dsa_select_plan;

/* Launch geometry chosen by a plan (for tests and benchmarks). */
typedef struct dsa_plan_desc {
  int32_t threads;           /* threads per CTA                                       */
  int32_t sm_count;          /* SMs on the plan's device                               */
  int64_t nblocks;           /* NB = ceil(W / B)                                       */
  int32_t vector_path;       /* 1: aligned rows stream with 128-bit accesses           */
  int32_t stream_capacity;   /* entries of the streaming block top-k buffer            */
  int32_t per_round;         /* most insertions one streaming round can make           */
  int32_t candidate_capacity;/* (Kb + 1) * B + 1 candidate columns                     */
  int64_t smem_select;       /* dynamic shared memory of the select kernel (bytes)     */
  int64_t smem_topk_cand;    /* ... of the candidate-mode row top-k kernel             */
  int64_t smem_topk_scan;    /* ... of the scan-mode row top-k kernel                  */
  int32_t ctas_per_sm_select;/* resident select CTAs per SM (unclustered kernel)        */
  int32_t grid_select;       /* CTAs per select launch (rows * split)                  */
  int32_t split;             /* CTAs per row chosen by the plan                        */
  int32_t parts;             /* wide split: parts per row of the first launch (0: none) */
} dsa_plan_desc;

/*
 * Build a plan for `cfg` on CUDA device `device`.  Validates the shape first
 * (DSA_ERR_INVALID_ARG / DSA_ERR_UNSUPPORTED without touching CUDA), then
 * reads the device's SM count and shared-memory limit and configures the
 * kernels.  *plan receives a host object freed by dsa_select_destroy;
 * *workspace_bytes (may be NULL) receives the device workspace every call of
 * this plan needs (0 for this build: pass NULL).  A plan with a wide split
 * (see dsa_select_cfg.split) allocates its own device memory for the parts'
 * lists here, rows * parts * (Kb + 1) * 8 bytes, and frees it in
 * dsa_select_destroy; if that allocation fails the plan keeps a cluster per
 * row instead.
 */
int dsa_select_init(const dsa_select_cfg* cfg, int device, dsa_select_plan** plan,
                    size_t* workspace_bytes);

/* Free a plan (NULL is ignored).  No CUDA call is made. */
void dsa_select_destroy(dsa_select_plan* plan);

/* Copy out the plan's launch geometry. */
int dsa_plan_describe(const dsa_select_plan* plan, dsa_plan_desc* out);

/*
 * Candidate selection and live-span mask (steps 1-4), in place.
 *   logits  [rows, W] fp32, element (r, c) at logits[r*row_stride + c*col_stride];
 *           4-byte aligned; rows whose start and column stride give 16-byte
 *           alignment take the 128-bit path.  Read over each row's live span,
 *           written with -inf over the non-kept columns of [0, min(end, W)).
 *   starts  int32 [ceil(rows/rep)] (NULL iff cfg.has_starts == 0).  A negative
 *           start is read as 0.
 *   ends    int32 [ceil(rows/rep)]; may exceed W; end <= start is an empty row.
 *   cand    int32 [rows, Kb + 1] output: the min(Kb, NB) chosen block ids in
 *           ascending order, -1 padding, then the pin (-1 for an empty row).
 *           Block b covers columns [start + b*B, start + (b+1)*B).
 *   workspace  unused by this build (may be NULL).
 */
int dsa_candidate_select(const dsa_select_plan* plan, float* logits, const int32_t* starts,
                         const int32_t* ends, int32_t* cand, void* workspace,
                         struct CUstream_st* stream);

/*
 * Row top-k (step 5): the best K columns of [start, min(end, W)) by value,
 * lower column on ties, as absolute column indices in ascending order with -1
 * padding, into topk int32 [rows, K].
 *   cand == NULL  scan mode: any logits; reads the whole live span.
 *   cand != NULL  candidate mode: logits must be the output of
 *                 dsa_candidate_select with the same bounds and this cand;
 *                 reads only the candidate columns (plus, when fewer than K
 *                 of them beat -inf, the first -inf columns of the span).
 *                 Returns exactly what scan mode returns on those logits.
 */
int dsa_row_topk(const dsa_select_plan* plan, const float* logits, const int32_t* starts,
                 const int32_t* ends, const int32_t* cand, int32_t* topk, void* workspace,
                 struct CUstream_st* stream);

/*
 * Steps 1-5 fused in one launch: the result of dsa_candidate_select followed
 * by dsa_row_topk in candidate mode, without re-reading the candidate list.
 */
int dsa_select_topk(const dsa_select_plan* plan, float* logits, const int32_t* starts,
                    const int32_t* ends, int32_t* cand, int32_t* topk, void* workspace,
                    struct CUstream_st* stream);

/*
 * Consumer step after the row top-k: per row, the ascending union of its
 * top-k indices (topk [rows, K] as dsa_row_topk writes them: an ascending
 * prefix of indices >= 0, then -1) and the last `window` columns of its live
 * span, [max(start, e' - window), e') with e' = min(end, W), written to
 * out int32 [rows, K + window] and padded with -1.  vLLM PR #57459 (Speedup
 * Result) names this step CombineTopkSwaIndicesKernel without defining it;
 * this is the plain reading.  window >= 0; starts/ends as for the other calls.
 */
int dsa_combine_window(const dsa_select_plan* plan, const int32_t* starts, const int32_t* ends,
                       const int32_t* topk, int32_t window, int32_t* out,
                       struct CUstream_st* stream);

/*
 * Indexer logits producer (tensor cores, tcgen05 kind::f8f6f4).
 *
 * The pages describe an FP8 "MQA score for every query/KV pair" written to a
 * [num_q, seq_len] matrix (vLLM PR #48726, Motivation) without the formula.
 * This build computes, for query t and key s in the query's live span
 * [start_t, min(end_t, keys)):
 *     logits[t * out_stride + s] = k_scale[s] * sum_h w[t*heads + h] * max(0, q[t, h, :] . k[s, :])
 * with q, k in OCP FP8 E4M3 and fp32 accumulation; columns outside the live
 * span are not written.  Supported: heads == 64, head_dim == 128.
 *   q        uint8 [queries, 64, 128] (e4m3 bytes), 16-byte aligned
 *   k        uint8 [keys, 128] (e4m3 bytes), 16-byte aligned
 *   k_scale  f32 [keys];  w  f32 [queries, 64]
 *   starts   int32 [queries] or NULL (start 0);  ends  int32 [queries]
 *   logits   f32 [queries, out_stride] (out_stride >= keys)
 * Waits inside the kernel are bounded; dsa_indexer_status() (synchronising)
 * reports DSA_ERR_TIMEOUT once if one gave up, and clears it.
 */
typedef struct dsa_indexer_cfg {
  int32_t queries;
  int32_t keys;
  int32_t heads;
  int32_t head_dim;
  int64_t out_stride;
} dsa_indexer_cfg;

int dsa_indexer_logits(const dsa_indexer_cfg* cfg, const uint8_t* q, const uint8_t* k,
                       const float* k_scale, const float* w, const int32_t* starts,
                       const int32_t* ends, float* logits, struct CUstream_st* stream);

int dsa_indexer_status(void);

/*
 * The producer fused with the selection, the [queries, keys] logits never
 * written.  Each query's logits are the ones dsa_indexer_logits computes
 * (start 0, live span [0, min(end_t, keys))).  Four launches share one record
 * per query in `workspace`: the producer stores each live block's largest
 * logit (4 bytes per block of B keys); the block top-k (pin, packed-column
 * clamp, edge flag) runs on those maxima; the producer recomputes the logits
 * of the kept blocks only, with the same tensor-core instruction and the same
 * arithmetic, so they have the same bits; the row top-k runs on them.  cand
 * and topk are bit-identical to dsa_indexer_logits followed by
 * dsa_select_topk.  No masked logits are produced (there is no logits
 * matrix).  The pages materialise the score matrix (vLLM PR #48726,
 * Motivation; vLLM PR #57459, Summary); the fusion is this library's own.
 *   plan       from dsa_select_init with rows == queries, width == keys,
 *              col_stride 1, has_starts 0, row_repeat 1, block_size in
 *              {1, 2, 4, 8}; any other plan gives DSA_ERR_UNSUPPORTED
 *   cfg        queries == plan rows, keys == plan width, heads 64, head_dim 128
 *   q, k, k_scale, w, ends   as for dsa_indexer_logits (no starts)
 *   workspace  device memory, 16-byte aligned, of at least
 *              dsa_indexer_select_workspace() bytes (per query 4 * ceil(keys /
 *              B) bytes plus about (Kb + 1) * (B + 1) * 4); owned by the caller and
 *              overwritten by every call, so calls that may overlap in time
 *              need workspaces of their own
 *   cand, topk int32 [queries, Kb + 1] and [queries, K], as dsa_select_topk
 * Returns DSA_OK once the launches are queued; bounded-wait timeouts are
 * reported by dsa_indexer_status() as for dsa_indexer_logits.
 */
int dsa_indexer_select_workspace(const dsa_select_plan* plan, size_t* bytes);

int dsa_indexer_select(const dsa_select_plan* plan, const dsa_indexer_cfg* cfg, const uint8_t* q,
                       const uint8_t* k, const float* k_scale, const float* w, const int32_t* ends,
                       void* workspace, size_t workspace_bytes, int32_t* cand, int32_t* topk,
                       struct CUstream_st* stream);

/*
 * Grouped masked sparse attention over the selection.
 *
 * vLLM PR #48726 ("LiteDSA: grouped masked sparse attention"): with H query
 * heads per token, G = 128 / H adjacent tokens form a group whose G x H
 * query/head rows fill one 128-row tensor-core tile; one GEMM runs over the
 * union of the group's selected KV positions, and each token still attends to
 * its own selection only.  The pages fix neither the dimensions nor the
 * formula; this build takes multi-query attention (a token's heads share the
 * selected key and value rows): for token t, head h and its selection A(t),
 *     o[t, h] = sum_{j in A(t)} softmax_j(scale * q[t, h] . k[j]) v[j]
 *     lse[t, h] = ln sum_{j in A(t)} exp(scale * q[t, h] . k[j])
 * and an empty A(t) gives o = 0, lse = -inf.
 *   heads      8 or 16 (G = 16 or 8);  head_dim = value_dim = 128
 *   keys       S: rows of k and v
 *   select     Kc: entries per token in idx, with G * Kc <= 49,152 (a group's
 *              union's token masks are built in shared memory)
 *   idx        int32 [tokens, Kc]: each row's positions in [0, S), strictly
 *              ascending, then -1 for unused entries (the rows dsa_row_topk
 *              and dsa_combine_window write qualify)
 *   q          bf16 [tokens, heads, 128];  k, v  bf16 [keys, 128]
 *   o          f32 [tokens, heads, 128];  lse  f32 [tokens, heads]
 *   workspace  device memory, 16-byte aligned, of at least
 *              dsa_sparse_attention_workspace() bytes; per group of G tokens:
 *              n (int32, padded to 16 bytes) | keys[G * Kc] int32, the union
 *              ascending | masks[G * Kc] uint32, bit g set when token
 *              group * G + g selected that position
 */
typedef struct dsa_attention_cfg {
  int32_t tokens;
  int32_t heads;
  int32_t keys;
  int32_t head_dim;
  int32_t value_dim;
  int32_t select;
} dsa_attention_cfg;

int dsa_sparse_attention_workspace(const dsa_attention_cfg* cfg, size_t* bytes);

/* Only the unions and masks, into workspace (the first launch of
 * dsa_sparse_attention). */
int dsa_group_union(const dsa_attention_cfg* cfg, const int32_t* idx, void* workspace,
                    size_t workspace_bytes, struct CUstream_st* stream);

/* The unions, then the attention (tcgen05, bf16 operands, fp32 accumulation;
 * P is rounded to bf16 for the P V product).  scale: the softmax scale, e.g.
 * 1/sqrt(128).  q, k, v, o 16-byte aligned; v finite.  Bounded-wait timeouts
 * are reported by dsa_sparse_attention_status(). */
int dsa_sparse_attention(const dsa_attention_cfg* cfg, const uint16_t* q, const uint16_t* k,
                         const uint16_t* v, const int32_t* idx, float scale, void* workspace,
                         size_t workspace_bytes, float* o, float* lse, struct CUstream_st* stream);

/*
 * The same attention when each token's selection is a set of position ranges
 * instead of an index list: the structure-aware form of vLLM PR #48726
 * ("LiteDSA: grouped masked sparse attention"), where DeepSeek-V4's C128A path
 * represents its compressed prefix plus sliding window as exact per-query
 * ranges over the group union, derived from positions, without materialising
 * the [tokens, topk + window] combined index matrix.  The pages give no
 * formula; this build's reading: token t attends to every key position in the
 * union of its ranges, with the multi-query attention above.
 *   ranges   int32 [tokens, nranges, 2]: half-open [lo, hi) key positions; an
 *            empty range (lo >= hi) is ignored, positions outside [0, keys)
 *            are dropped, overlapping ranges of a token count once
 *   nranges  1 .. 8 ranges per token
 *   cfg->select: the most positions the ranges of one token cover (sizes each
 *            group's record: G * select <= 2^24; a group whose union exceeds
 *            G * select is cut there)
 *   workspace: dsa_sparse_attention_ranges_workspace() bytes, the record
 *            layout of dsa_sparse_attention (union ascending, token masks)
 * Errors: DSA_ERR_INVALID_ARG for a null or misaligned pointer, a workspace
 * too small or nranges < 1; DSA_ERR_UNSUPPORTED for nranges > 8 or the
 * shapes dsa_sparse_attention does not take.
 */
int dsa_sparse_attention_ranges_workspace(const dsa_attention_cfg* cfg, int32_t nranges, size_t* bytes);

/* Only the unions and masks, into workspace (the first launch of
 * dsa_sparse_attention_ranges). */
int dsa_group_union_ranges(const dsa_attention_cfg* cfg, const int32_t* ranges, int32_t nranges, void* workspace,
                           size_t workspace_bytes, struct CUstream_st* stream);

/* The unions from ranges, then the attention of dsa_sparse_attention. */
int dsa_sparse_attention_ranges(const dsa_attention_cfg* cfg, const uint16_t* q, const uint16_t* k,
                                const uint16_t* v, const int32_t* ranges, int32_t nranges, float scale,
                                void* workspace, size_t workspace_bytes, float* o, float* lse,
                                struct CUstream_st* stream);

/* DSA_ERR_TIMEOUT once after an attention launch gave up a wait (then
 * cleared), else DSA_OK; synchronises the device. */
int dsa_sparse_attention_status(void);

/*
 * dsa_indexer_select without a caller workspace: the fused producer +
 * selection, with its per-query records kept in one fixed array inside this
 * library instead of memory the caller allocates.  The pages describe nothing
 * like it; it exists for callers of this library that cannot allocate device
 * memory when they call: an engine that hands all free device memory to its
 * own pool before serving (a cudaMalloc then fails, or bypasses the pool and
 * fragments it), a plugin whose host framework owns the device allocator and
 * allows no side allocations, or plain C code with no allocator to take a
 * workspace from.  This call allocates nothing: no cudaMalloc, no cudaFree,
 * no allocating library routine.
 *   Limit: the array holds DSA_NOALLOC_SCRATCH_BYTES (8 MiB) on every device
 *   that loads the library, until the process exits.  A plan whose
 *   dsa_indexer_select_workspace() exceeds it gets DSA_ERR_UNSUPPORTED (at
 *   block size 8 and Kb 256: 112 queries of 131,072 keys, 15 of
 *   1,048,576).
 *   Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture begins.  The address is kept with the id of
 *   the context it belongs to; after a device reset the next call sees a new
 *   context and looks the address up again (that call, too, belongs before
 *   any capture).
 *   Sharing: every call on a device uses the same array, and each call
 *   overwrites what the last one left there (nothing in it has to start at
 *   zero: a call writes every part of it that it reads back).  Calls that can
 *   run at the same time on the GPU -- on streams with no ordering between
 *   them -- race on it; keep them on one stream or otherwise ordered.
 * Arguments, results and errors are those of dsa_indexer_select.
 */
#define DSA_NOALLOC_SCRATCH_BYTES (8u << 20)

int dsa_indexer_select_noalloc(const dsa_select_plan* plan, const dsa_indexer_cfg* cfg,
                               const uint8_t* q, const uint8_t* k, const float* k_scale,
                               const float* w, const int32_t* ends, int32_t* cand, int32_t* topk,
                               struct CUstream_st* stream);

/*
 * Paged key/value cache held in 4 bits, and the sparse attention over it.
 *
 * The selection above gives each query row the positions it attends to.  In a
 * server those positions belong to many requests, whose keys and values sit in
 * pages; the calls below keep the pages, store rows in 4 bits and attend to
 * the selected ones.  No page describes this part: it is this library's own
 * design.
 *
 * Layout.  The cache is [pages, page_size, kv_heads] records of
 * DSA_CACHE_RECORD_BYTES = 144 bytes, one per position and key/value head
 * (head_dim = value_dim = 128):
 *     bytes   0 ..  63   key codes, e2m1: dim 2 i in the low nibble of byte i,
 *                        dim 2 i + 1 in the high one
 *     bytes  64 .. 127   value codes, the same
 *     bytes 128 .. 135   key scales, e4m3: byte g scales dims 16 g .. 16 g + 15
 *     bytes 136 .. 143   value scales
 * A key element is code * scale * 2^k_shift, a value element code * scale *
 * 2^v_shift.  slot = page * page_size + offset numbers the positions of the
 * whole cache; request r's position p lies in page tables[r, p / page_size] at
 * offset p % page_size.  16-byte aligned; dsa_cache_bytes() gives its size.
 *
 *   pages      >= 0; pages * page_size < 2^31
 *   page_size  a power of two, 1 .. 4096
 *   kv_heads   1 .. 64
 *   k_shift, v_shift   -32 .. 32: a power of two that keys (values) are
 *              divided by before they are rounded.  One e4m3 scale covers
 *              groups whose largest element is between 0.012 and 2688; smaller
 *              groups become zeros, larger ones are clipped, unless the shift
 *              moves them into that range.
 * A cfg outside these limits gives DSA_ERR_INVALID_ARG (DSA_ERR_UNSUPPORTED
 * for more kv_heads).  Rows are bf16, f16 or f32 (DSA_BF16, DSA_F16, DSA_F32).
 */
#define DSA_CACHE_RECORD_BYTES 144
#define DSA_BF16 0
#define DSA_F16 1
#define DSA_F32 2

typedef struct dsa_cache_cfg {
  int32_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t k_shift;
  int32_t v_shift;
} dsa_cache_cfg;

int dsa_cache_bytes(const dsa_cache_cfg* cfg, size_t* bytes);

/*
 * One step's pages, block tables and slots, from request lengths on the
 * device: for request r, lens[r] is its length after the step and fresh[r] how
 * many of those positions are this step's tokens (the last fresh[r]).
 *   - a request that needs more pages than it holds (ceil(lens / page_size))
 *     takes them from the top of the free stack, in request order and then in
 *     position order; one that needs fewer (finished: lens 0; drafts rejected)
 *     gives its last pages back, so that a step taken back leaves the stack as
 *     it was.  Pages given back are taken again from the next call on.
 *   - token i of the step (request after request, position after position)
 *     gets token_req[i], ends[i] = its position + 1 (the live end that
 *     dsa_select_topk takes with row_repeat 1) and slots[i].  Entries past the
 *     last token get -1, 0 and -1: a padded batch selects, stores and attends
 *     to nothing there.
 *   requests   R, 0 .. 8192;  table_width  P, pages a request may hold
 *   tokens     T, entries of token_req, ends and slots
 *   lens, fresh  int32 [R];  tables int32 [R, P] and held int32 [R] (pages each
 *              request holds now): updated; entries of tables at or past held
 *              are -1 once they have been given back
 *   free_pages int32 [free_capacity], a stack of *free_count page ids, the
 *              next one last; both updated
 *   first      int32 [R + 1]: the requests' first tokens, first[R] their total
 *   status     int32 [4]: code, pages short, tokens, free pages now
 * A step that cannot be taken changes nothing (tables, held, the stack), gives
 * every entry -1, 0 and -1 and first = 0, and leaves its reason in status[0]:
 *   1 more pages are needed than are free (status[1]: how many), or the stack
 *     has no room for those given back;  2 a request needs more than P pages;
 *   3 more tokens than T;  4 a length or count is negative, fresh[r] > lens[r],
 *     or held[r] or *free_count is out of range.
 * Where several hold, 4 comes first, then 2, 3 and 1.  A token whose page id
 * is not in [0, pages) gets slot -1.  One launch; the tensors must not overlap.
 */
int dsa_cache_plan(const dsa_cache_cfg* cfg, int32_t requests, int32_t table_width, int32_t tokens,
                   int32_t free_capacity, const int32_t* lens, const int32_t* fresh, int32_t* tables,
                   int32_t* held, int32_t* free_pages, int32_t* free_count, int32_t* first,
                   int32_t* token_req, int32_t* ends, int32_t* slots, int32_t* status,
                   struct CUstream_st* stream);

/*
 * Store rows: token i's keys and values, k and v [tokens, kv_heads, 128] with
 * k_stride (v_stride) elements from one token to the next, go to record
 * slots[i].  Each group of 16 dims gets scale = e4m3(min(max|x| / 6, 448)) and
 * codes e2m1(x / scale), both rounded to nearest, ties to even, and clipped
 * (infinities too) to the type's largest; x is the element divided by the
 * shift's power of two.  A group that holds a NaN reads back as NaN.
 *   slots   int32 [tokens]; one outside [0, pages * page_size) stores nothing.
 *           A slot named twice in a call holds one of its rows, or parts of
 *           several: give each token its own.
 */
int dsa_cache_write(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype, const void* k, const void* v,
                    int64_t k_stride, int64_t v_stride, const int32_t* slots, uint8_t* cache,
                    struct CUstream_st* stream);

/* Read rows back: k and v [tokens, kv_heads, 128], contiguous and 16-byte
 * aligned; zeros for a slot outside [0, pages * page_size).  With shifts of 0
 * every element is exact in bf16 and f16. */
int dsa_cache_read(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype, const uint8_t* cache,
                   const int32_t* slots, void* k, void* v, struct CUstream_st* stream);

/*
 * Sparse attention over the cache: the form for decode steps and mixed
 * batches.  heads = kv_heads * n query heads, n = 1 .. 128; query head h reads
 * key/value head h / n.  For token t of request token_req[t], with A(t) the
 * positions listed in idx[t],
 *     o[t, h] = sum_{j in A(t)} softmax_j(scale * q[t, h] . k[j]) v[j]
 *     lse[t, h] = ln sum_{j in A(t)} exp(scale * q[t, h] . k[j])
 * and an empty A(t) (no entry, or token_req[t] outside [0, requests)) gives
 * o = 0, lse = -inf.
 *   idx     int32 [tokens, select] (the rows of dsa_row_topk and
 *           dsa_combine_window qualify): positions in any order, entries below 0
 *           anywhere among them unused.  A position at or past table_width *
 *           page_size, or in a page whose id is not in [0, pages), is not
 *           attended to; one listed twice counts twice.
 *   tables  int32 [requests, table_width]
 *   q, o    [tokens, heads, 128] of one type, DSA_BF16 or DSA_F16, 16-byte
 *           aligned;  lse  f32 [tokens, heads]
 *   scale   of any sign; scale * 2^k_shift * log2(e) is finite in f32
 * Scores and sums are held in fp32; q, the softmax weights and the expanded rows
 * enter the products in f16 (the rows exactly, and q but for elements below
 * 2^-26 of a row's largest; a weight is off by 2^-11 of it, or by 2^-32 of the
 * row's largest), o is rounded once.  A NaN key scale makes the rows that attend
 * to its record NaN, o and lse; a NaN value scale its 16 dims of their o, and
 * nothing else.  Few rows split their lists over a cluster of CTAs; the order of
 * every sum is fixed, so results repeat bit for bit.
 */
int dsa_cache_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                        int32_t requests, int32_t table_width, int32_t dtype, const uint8_t* cache,
                        const void* q, const int32_t* idx, const int32_t* token_req,
                        const int32_t* tables, float scale, void* o, float* lse,
                        struct CUstream_st* stream);

/*
 * The same attention for the tokens of one request's prompt chunk, whose
 * neighbours select overlapping positions: G = 128 / n adjacent tokens share
 * the union of their selections, as in dsa_sparse_attention, so that a record
 * is read and expanded once a group.  n = heads / kv_heads = 8 or 16 and
 * G * select <= 49,152.
 *   idx     int32 [tokens, select]: each row's positions strictly ascending,
 *           then -1 (a position listed twice counts once here)
 *   table   int32 [table_width]: the request's block table
 *   workspace  device memory, 16-byte aligned, of at least
 *           dsa_cache_attention_prompt_workspace() bytes
 * Everything else is as in dsa_cache_attention.
 */
int dsa_cache_attention_prompt_workspace(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads,
                                         int32_t select, size_t* bytes);

int dsa_cache_attention_prompt(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                               int32_t table_width, int32_t dtype, const uint8_t* cache, const void* q,
                               const int32_t* idx, const int32_t* table, float scale, void* workspace,
                               size_t workspace_bytes, void* o, float* lse,
                               struct CUstream_st* stream);

/* DSA_ERR_TIMEOUT once after a launch of dsa_cache_attention or
 * dsa_cache_attention_prompt on the current device gave up a wait (then
 * cleared), else DSA_OK; synchronises the device, every stream of it. */
int dsa_cache_attention_status(void);

/*
 * Paged key/value cache held in 16 bits: a step's rotated rows stored, causal
 * attention of its tokens to everything before them, and attention to the pages
 * that each token's queries score highest.  dsa_cache_plan above serves this
 * cache too (its slots, ends, first and tables number positions and pages, not
 * records).  This library's own design.
 *
 * Layout.  k_cache and v_cache [pages, page_size, kv_heads, 128], means [pages,
 * kv_heads, 128], all of cfg's type, each 16-byte aligned.  Request r's position
 * p is row p % page_size of page tables[r, p / page_size].  The means hold each
 * full page's mean key; what they hold of other pages is not read.
 *   pages      >= 0; pages * page_size < 2^31
 *   page_size  16, 32, 64 or 128
 *   kv_heads   1 .. 64
 *   dtype      DSA_BF16 or DSA_F16
 * A cfg outside these limits gives DSA_ERR_INVALID_ARG (DSA_ERR_UNSUPPORTED for
 * other powers of two of page_size and more kv_heads).
 *
 * A step (dsa_kv_attention, dsa_kv_select, dsa_kv_block_attention).  Tokens
 * first[r] .. first[r + 1] - 1 are request r's newest, lens[r] its length with
 * them: token i has position p = lens[r] - first[r + 1] + i.  A request whose length
 * is below its tokens here (or negative) has none: its tokens attend to nothing and
 * have no pages (no plan makes such a step).  Rows of tokens at or past
 * first[requests] are left as they were.  heads = kv_heads * n, n = 1 ..
 * 128; query head h belongs to key/value head h / n.
 *   requests   1 .. 8192 (tokens 0: nothing is read);  table_width >= 0
 *   q          [tokens, heads, 128] with q_stride elements (a multiple of 8)
 *              from one token to the next, 16-byte aligned
 *   first int32 [requests + 1], ascending from 0 up to tokens;  lens int32
 *   [requests];  tables int32 [requests, table_width]
 * A position at or past table_width * page_size, or in a page whose id is not in
 * [0, pages), is not attended to.
 */
typedef struct dsa_kv_cfg {
  int32_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t dtype;
} dsa_kv_cfg;

/*
 * Store a step's rows and rotate its queries.  Token i has position ends[i] - 1
 * and goes to slots[i] (page * page_size + row); its q, k and v rows lie q_stride,
 * k_stride and v_stride elements (multiples of 8) after the token's before it,
 * heads and dims packed, 16-byte aligned.
 *   rotation  pairs (a, b) of the first `rotary` dims (a multiple of 16, 0 .. 128)
 *             become gain * (a cos x - b sin x, b cos x + a sin x) with x =
 *             position * 2 pi * turns[j] / 2^64: dims j and j + rotary / 2 are
 *             pair j, or with neighbours != 0 dims 2 j and 2 j + 1.  turns int64
 *             [rotary / 2]: a frequency as a fraction of 2^64 of a turn a
 *             position, so that the angle of a far position is reduced exactly.
 *             Keys and queries are rotated in f32 and rounded once; other dims
 *             and values are copied.
 *   q_out     [tokens, heads, 128] contiguous; may be q.  heads 0: no queries.
 *   means     NULL: not kept.  A page whose last row is stored by this call gets
 *             the mean of its rows as stored, summed in f32 in a fixed order and
 *             rounded once.
 *   ends      1 <= ends[i]; a token with less is not looked at (its q_out row is
 *             left as it was)
 *   slots     one outside [0, pages * page_size): k and v are not stored.  No slot
 *             twice; where means are kept, tokens that store into one page stand
 *             next to one another in the order of their slots, as in a plan.
 */
int dsa_kv_append(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t rotary, int32_t neighbours,
                  float gain, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const int32_t* ends, const int32_t* slots, const int64_t* turns, void* q_out,
                  void* k_cache, void* v_cache, void* means, struct CUstream_st* stream);

/*
 * Causal attention of a step's tokens: with A(t) the positions 0 .. p of t's
 * request,
 *     o[t, h] = sum_{j in A(t)} softmax_j(scale * q[t, h] . k[j]) v[j]
 *     lse[t, h] = ln sum_{j in A(t)} exp(scale * q[t, h] . k[j])
 * and an empty A(t) gives o = 0, lse = -inf.  Single tokens, drafts and prompt
 * chunks may stand side by side.
 *   o    [tokens, heads, 128] of cfg's type, 16-byte aligned;  lse f32 [tokens, heads]
 *   scale  of any sign; scale * log2(e) is finite in f32
 *   workspace  device memory, 16-byte aligned, of at least
 *              dsa_kv_attention_workspace() bytes; nothing in it has to start at
 *              zero.  Calls that may run at the same time need one each.
 * Scores, sums and outputs are held in f32; the softmax weights, the largest of them
 * between 2^7 and 2^15, are rounded to cfg's type for the second product (bf16 values of
 * more than 2^112 / positions pass the sums' range).  What a row does not attend to --
 * later positions, stale rows of a page -- has no effect on it, whatever it holds (but
 * on the time: a row is computed a second time, by one warp, where a value in a tile
 * that it attends to part of is a NaN or infinite, or, with lists, a score there).  A
 * NaN score makes a row's o and lse NaN, one of +infinity its o NaN and its lse
 * +infinity.  Results repeat bit for bit.
 */
int dsa_kv_attention_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                               int32_t table_width, size_t* bytes);

int dsa_kv_attention(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
                     const void* k_cache, const void* v_cache, const void* q, int64_t q_stride,
                     const int32_t* first, const int32_t* lens, const int32_t* tables, float scale,
                     void* workspace, size_t workspace_bytes, void* o, float* lse, struct CUstream_st* stream);

/*
 * The pages each token's queries score highest: for token t at position p and
 * key/value head g, page j's score is the sum over the group's heads of
 * q[t, h] . means[page j, g].  The first `lead` pages and the last `trail` up to
 * the token's own (p / page_size) are taken always, and of the others before them
 * the best, select pages in all (all there are, if fewer).
 *   idx     int32 [tokens, kv_heads, select]: page numbers within the request,
 *           ascending, then -1
 *   select  1 .. 256;  lead >= 0, trail >= 1, lead + trail <= select.  The own page
 *           of a position past the table is the table's last.
 *   workspace  as above, dsa_kv_select_workspace() bytes
 * Ranks are those of the scores in f64 (which are computed where f32 cannot tell two
 * apart); among equal scores the lower page wins; a NaN score ranks below every
 * other.  A page without a valid id has no score and ranks as a NaN does.  A token
 * for which hundreds of pages come close to its last place takes many times as long
 * as others.
 */
int dsa_kv_select_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                            int32_t table_width, size_t* bytes);

int dsa_kv_select(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
                  int32_t select, int32_t lead, int32_t trail, const void* means, const void* q, int64_t q_stride,
                  const int32_t* first, const int32_t* lens, const int32_t* tables, void* workspace,
                  size_t workspace_bytes, int32_t* idx, struct CUstream_st* stream);

/*
 * dsa_kv_attention with A(t), for a query head of key/value head g, cut down to
 * the positions up to t's own in the pages idx[t, g] lists.
 *   idx  int32 [tokens, kv_heads, select] (the rows of dsa_kv_select qualify):
 *        strictly ascending, then -1;  select 1 .. 4096
 */
int dsa_kv_block_attention_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                                     int32_t table_width, int32_t select, size_t* bytes);

int dsa_kv_block_attention(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                           int32_t table_width, int32_t select, const void* k_cache, const void* v_cache,
                           const void* q, int64_t q_stride, const int32_t* idx, const int32_t* first,
                           const int32_t* lens, const int32_t* tables, float scale, void* workspace,
                           size_t workspace_bytes, void* o, float* lse, struct CUstream_st* stream);

/* DSA_ERR_TIMEOUT once after a launch of dsa_kv_attention, dsa_kv_select or
 * dsa_kv_block_attention on the current device gave up a wait (then cleared),
 * else DSA_OK; synchronises the device, every stream of it. */
int dsa_kv_status(void);

/* Static description of a status code. */
const char* dsa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* DSA_SELECT_H */
