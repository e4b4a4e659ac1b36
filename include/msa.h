/*
 * msa.h - C ABI of libmsa: block-sparse, causal, document-local grouped-query
 * attention (MiniMax Sparse Attention, "MSA") forward and backward on one
 * NVIDIA GB300 (sm_103a).
 *
 * What the library computes is fixed by the flat-attention interface of the
 * NeMo-Automodel PR "feat(minimax-m3): add SM100 MSA sparse attention with
 * custom backward" (sections "Design" and "Supported scope") and by the
 * run_backward contract on the API page "msa_backward_sm100":
 *
 *   Q, dO : bf16 [T, 64, 128]   compact token-major (THD) rows
 *   K, V  : bf16 [T, 4, 128]
 *   q2k   : int32 [4, T, 16]    document-local key-block ids per index head,
 *                               -1 marks an unused slot
 *   doc_offsets : int32 [D+1]   0 = o_0 < o_1 < ... < o_D = T
 *
 * Query head h reads KV head and index head g = h / 16.  Token t = o_d + p of
 * document d attends key o_d + j iff j <= p and floor(j / 128) is one of the
 * values in q2k[g, t, :] (a set: duplicates count once).  Then
 *   s_j = scale * <Q[t,h], K[j,g]>,  LSE[t,h] = ln sum_j exp(s_j),
 *   O[t,h] = sum_j exp(s_j - LSE[t,h]) V[j,g],
 * and the backward returns dQ, dK, dV of L = sum(O * dO).  A row that sees no
 * key gets O = 0, LSE = -inf and zero gradients.  A q2k value < -1 or >= the
 * document's block count is an error (MSA_ERR_BAD_Q2K, detected on device).
 *
 * Conventions for every call:
 *   - All tensor and workspace pointers are DEVICE pointers on the current
 *     CUDA device, contiguous, 16-byte aligned.  The caller owns all memory;
 *     the library never allocates or frees device memory.
 *   - Calls are asynchronous on the given stream (a cudaStream_t; NULL is the
 *     legacy default stream) and never synchronise, except the diagnostics
 *     msa_read_status and msa_plan_export which say so.
 *   - Host-detectable problems (null pointer, bad size, misalignment, small
 *     workspace) return an error before anything is launched.  Problems only
 *     the device can see (bad q2k value, bad document offsets, a pipeline
 *     wait that timed out) set bits of the plan's device status word; later
 *     kernels of the same plan then skip their work.  msa_read_status reads it.
 *   - Gradients are accumulated with floating-point atomics, so results are
 *     not bitwise reproducible from run to run.  There is no deterministic
 *     mode.
 *   - Limits: 1 <= T <= 2^20, 1 <= num_docs <= T.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Stream handle: a cudaStream_t, passed as an opaque pointer. */
typedef struct CUstream_st* msa_stream_t;

typedef enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1,  /* null pointer, T or num_docs out of range, ...  */
  MSA_ERR_UNSUPPORTED = 2,  /* device is not sm_100 / sm_103 class             */
  MSA_ERR_ALIGNMENT = 3,    /* a pointer is not 16-byte aligned                */
  MSA_ERR_WORKSPACE = 4,    /* workspace smaller than the *_workspace_bytes   */
  MSA_ERR_CUDA = 5,         /* a CUDA runtime call failed                      */
  MSA_ERR_BAD_Q2K = 6,      /* device: a q2k slot outside [-1, blocks of doc)  */
  MSA_ERR_BAD_OFFSETS = 7,  /* device: doc_offsets not 0 < ... strictly up .. T */
  MSA_ERR_TIMEOUT = 8,      /* device: a bounded pipeline wait gave up         */
  MSA_ERR_CAPACITY = 9,     /* device: a plan table exceeded its capacity      */
  MSA_ERR_RANGE = 10,       /* device warning: the last backward's 16-bit dQ
                               pool overflowed (dQ holds inf / nan); rerun it
                               with MSA_DQ_ACCUM_BF16 or MSA_DQ_ACCUM_F32      */
  MSA_ERR_BAD_PAGE = 11,    /* device: a page-table entry that is needed lies
                               outside the pool, or a position or a length
                               outside its row of the page table              */
  MSA_ERR_BAD_TREE = 12     /* device: a row of more than 64 drafted tokens, a
                               parent that does not come before its token, or
                               a path that does not ascend                    */
} msa_status;

/* Human-readable name of a status code (static string). */
const char* msa_status_string(msa_status s);

/* Precision of the dQ accumulation pool of msa_backward.  The pages' default
 * is packed FP16 atomics with a BF16 switch for range (section "Supported
 * scope", the MSA_M3_DQ_ACCUM setting); FP32 is the widest and slowest.
 * FP16 saturates above 65504: when the finalize reads a non-finite FP16 pool
 * value it sets MSA_ERR_RANGE in the plan's status word.  That bit is a
 * warning about the last backward only (every backward clears it first) and,
 * unlike the errors, does not make later kernels of the plan skip work. */
typedef enum msa_dq_accum {
  MSA_DQ_ACCUM_F16 = 0,
  MSA_DQ_ACCUM_BF16 = 1,
  MSA_DQ_ACCUM_F32 = 2
} msa_dq_accum;

/* Precision of the forward's O accumulation pool.  The up-to-16 block
 * partials of an output row are added in a pool at a shared row shift; FP32
 * keeps O's rounding to that of the final bf16 store.  MSA_O_ACCUM_BF16 is
 * rejected with MSA_ERR_UNSUPPORTED: an 8-bit mantissa in every addition
 * plus the bf16 store can put O one bf16 ulp (1.6e-2 at |O| in [2, 4)) off
 * the exact result, above the forward's 1e-2 max-abs bar. */
typedef enum msa_o_accum {
  MSA_O_ACCUM_F32 = 0,
  MSA_O_ACCUM_BF16 = 1
} msa_o_accum;

/* Plan-build options.  Pass NULL for the defaults. */
typedef struct msa_plan_options {
  /* Tasks of one (index head, key block) bucket are cut at runs of
   * super_block consecutive query blocks (0 = never cut).  Default 64. */
  int32_t super_block;
  /* An msa_dq_accum value.  Default MSA_DQ_ACCUM_F16. */
  int32_t dq_accum;
  /* An msa_o_accum value; only (0) MSA_O_ACCUM_F32 is accepted. */
  int32_t o_accum;
  /* Dense octets of the forward: an aligned run of 8 tokens in query block
   * b whose tokens see different blocks runs as one tile over all blocks
   * 0 .. b, each token's rows masked to its own blocks, when b + 1 <=
   * dense_blocks (instead of through the pooled tasks).  0 selects the
   * default, 32; -1 turns dense octets off; 1 .. 64 set the bound; other
   * values give MSA_ERR_INVALID_ARG. */
  int32_t dense_blocks;
  int32_t reserved[4];
} msa_plan_options;

/*
 * The execution plan derived from q2k and the document layout: per index
 * head and key block, the queries that selected it (the k2q CSR), and the
 * task table of 128-row tiles (8 queries x 16 heads of one index head against
 * one key block) that the forward and backward kernels walk.  The pages call
 * these the CSR and scheduling metadata and, on the API page
 * msa_backward_sm100, the backward's task rows, one 128-row tile each,
 * grouped by (batch, index head, key block).
 *
 * A plain struct of device pointers into the caller's plan workspace and of
 * host-side capacities.  Fill it with msa_build_plan; do not edit it.  It
 * stays valid while the workspace and the q2k / doc_offsets buffers live and
 * may be reused by any number of msa_forward / msa_backward calls on the same
 * T, q2k and documents.  All counts live on the device.
 */
typedef struct msa_plan {
  int64_t T;
  int32_t num_docs;
  int32_t super_block;
  int32_t dq_accum;
  int32_t o_accum;
  int32_t dense_blocks; /* the bound in effect (0: no dense octets)     */
  int64_t nb_cap;     /* bound on the number of 128-key blocks            */
  int64_t tri_cap;    /* bound on (index head, doc, key block, query block) */
  int64_t nnz_cap;    /* bound on CSR entries                              */
  int64_t task_cap;   /* bound on tasks                                    */
  const int32_t* q2k;
  const int32_t* doc_offsets;
  int64_t* header;    /* device: status and counts                         */
  int32_t* doc_info;  /* device: [num_docs][4] start, length, blocks, block base */
  int64_t* doc_tri;   /* device: [num_docs+1] prefix of per-doc count entries */
  int32_t* cnt;       /* device: [tri_cap] queries per count entry          */
  int32_t* off;       /* device: [tri_cap] exclusive prefix of cnt          */
  int32_t* col;       /* device: [nnz_cap] query tokens, sorted per entry   */
  int32_t* tcnt;      /* device: [tri_cap] tasks per count entry            */
  int32_t* toff;      /* device: [tri_cap] exclusive prefix of tcnt         */
  int32_t* tasks;     /* device: [task_cap][4] task records                 */
  int32_t* scan_tmp;  /* device: scan scratch                               */
  int64_t scan_tmp_len;
  /* The forward's octet groups: aligned runs of 8 tokens (document positions
   * 8k .. 8k+7, one block b) whose tokens all see the same selected blocks,
   * or whose block range 0 .. b is short (dense octets, each token masked to
   * its own blocks); their tiles are accumulated block after block in one
   * place, without the pool. */
  int64_t item_cap;   /* bound on octet-group items                        */
  uint8_t* grouped;   /* device: [4][T] 1 = the token's octet is grouped    */
  int32_t* items;     /* device: [item_cap][36] group items (msa_plan_export_groups) */
  int32_t* fflag;     /* device: [task_cap] task has an ungrouped query      */
  int32_t* fpos;      /* device: [task_cap] exclusive prefix of fflag        */
  int32_t* ftasks;    /* device: [task_cap][4] the forward's pooled tasks    */
  int32_t* rows;      /* device: [4 T] the (token t, index head g) pairs
                       * outside the octet groups, as 4 t + g, in no
                       * particular order (the pooled path's rows)           */
} msa_plan;

/* Bytes of plan workspace needed for T tokens in num_docs documents.
 * Host only, no CUDA call. */
msa_status msa_plan_workspace_bytes(int64_t T, int32_t num_docs, size_t* bytes);

/*
 * Build the plan on the device (no host synchronisation): validate the
 * document offsets and q2k, invert q2k into the k2q CSR (queries ascending
 * within each bucket), cut the buckets into tasks and count the attended
 * (query, head, key) triples.
 *   q2k          device int32 [4, T, 16]
 *   doc_offsets  device int32 [num_docs + 1]
 *   workspace    device, >= msa_plan_workspace_bytes(T, num_docs)
 *   out          host struct, filled on success
 * Device-side validation failures set MSA_ERR_BAD_Q2K / MSA_ERR_BAD_OFFSETS in
 * the status word (see msa_read_status); forward and backward then do no work.
 */
msa_status msa_build_plan(const int32_t* q2k, const int32_t* doc_offsets, int64_t T,
                          int32_t num_docs, const msa_plan_options* opts, void* workspace,
                          size_t workspace_bytes, msa_stream_t stream, msa_plan* out);

/*
 * msa_build_plan with the plan tables in device memory owned by the library,
 * for callers that cannot allocate device memory where they need a plan (a
 * memory manager that forbids allocation at that point, a hook that is handed
 * only the input buffers).  The pages have no counterpart of this call.
 *   - The tables live in one static 16 MiB device array that every GPU which
 *     loads the library keeps until the process exits.  A problem is
 *     accepted while msa_plan_workspace_bytes(T, num_docs) <= 16 MiB (about
 *     T <= 21400 tokens, a little more or less with the number of
 *     documents); larger ones are rejected with MSA_ERR_WORKSPACE after the
 *     argument checks and before any CUDA call.
 *   - Each call looks the array's device address up on the current device
 *     (cudaGetSymbolAddress); the first call on a device initialises the
 *     library's module there, so make it before any stream capture.
 *   - Every call reuses the same array: the returned plan is valid until the
 *     next msa_build_plan_static call on that device, and calls (or uses of
 *     the plan) that overlap on the GPU race.  Nothing else is allocated.
 * Arguments, validation and errors otherwise as msa_build_plan.
 */
msa_status msa_build_plan_static(const int32_t* q2k, const int32_t* doc_offsets, int64_t T,
                                 int32_t num_docs, const msa_plan_options* opts,
                                 msa_stream_t stream, msa_plan* out);

/* Bytes of forward workspace for a plan (host only).  Dominated by the fp32
 * O pool, T x 64 x 128 x 4 bytes. */
msa_status msa_forward_workspace_bytes(const msa_plan* plan, size_t* bytes);

/*
 * Forward (the pages' flat sparse forward: O [T,64,128] and LSE [T,64]).
 *   q  device bf16 [T,64,128]; k, v device bf16 [T,4,128]
 *   softmax_scale   e.g. 1/sqrt(128)
 *   o   device bf16 [T,64,128] (written)
 *   lse device fp32 [T,64] natural-log LSE (written; -inf for keyless rows)
 *   workspace device, >= msa_forward_workspace_bytes(plan)
 */
msa_status msa_forward(const msa_plan* plan, const void* q, const void* k, const void* v,
                       float softmax_scale, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, msa_stream_t stream);

/* Bytes of backward workspace for a plan (host only). */
msa_status msa_backward_workspace_bytes(const msa_plan* plan, size_t* bytes);

/*
 * Backward (the pages' launch sequence: delta = rowsum(dO * O) -> zero the
 * gradient pools -> main KV-parallel backward -> BF16 finalize), see
 * msa_backward_sm100 run_backward.  O and LSE are the forward's outputs.
 *   dq device bf16 [T,64,128]; dk, dv device bf16 [T,4,128] (written; compact
 *   token order, zero for rows that receive no gradient)
 */
msa_status msa_backward(const msa_plan* plan, const void* q, const void* k, const void* v,
                        const void* o, const float* lse, const void* dout, float softmax_scale,
                        void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                        msa_stream_t stream);

/* Synchronises the stream and returns the plan's device status (MSA_OK if no
 * device-side error was recorded): the lowest-numbered error, else
 * MSA_ERR_RANGE if the last backward's FP16 dQ pool overflowed.  For tests
 * and diagnostics. */
msa_status msa_read_status(const msa_plan* plan, msa_stream_t stream);

/* Plan counts after synchronising the stream: counts[0] = key blocks NB,
 * [1] = CSR entries, [2] = tasks, [3] = attended (query, head, key) triples,
 * [4] = count entries, [5] = octet-group items, [6] = tasks of the forward's
 * pooled list.  Host array of 7 int64. */
msa_status msa_plan_counts(const msa_plan* plan, msa_stream_t stream, int64_t* counts);

/*
 * Copy the plan tables to host memory after synchronising the stream (for
 * the bit-exact plan tests).  Each destination may be NULL to skip it.
 *   col   int32 [nnz]  query tokens, grouped by task order
 *   tasks int32 [ntasks][4]: {first col index, first key token,
 *         key count | query count << 8 | index head << 12,
 *         index head * nb_cap + global key block}
 * Capacities are element counts; too small -> MSA_ERR_INVALID_ARG.
 */
msa_status msa_plan_export(const msa_plan* plan, msa_stream_t stream, int32_t* col,
                           int64_t col_capacity, int32_t* tasks, int64_t task_capacity);

/*
 * Copy the forward's octet-group tables to host memory after synchronising
 * the stream (for the plan tests).  Each destination may be NULL to skip it.
 *   grouped uint8 [4][T]: 1 where the token's octet is grouped
 *   items   int32 [n_items][36]: first token of octet A, of octet B (-1 if
 *           none), queries of A | of B << 4 | index head << 8 | blocks << 12
 *           | dense << 20, document index, then for a uniform item the
 *           blocks ascending, -1 padded to 32 words, for a dense one (blocks
 *           0 .. b) each token's 64-bit block mask as a low and a high word
 *           (tokens of A, then of B; 32 words); items are ordered by
 *           decreasing work (blocks x octets)
 *   ftasks  int32 [n_ftasks][4]: the task records (as in msa_plan_export) of
 *           the tasks with at least one ungrouped query, in task order
 * Capacities are element counts of the first dimension (T for grouped, which
 * must be >= T); too small -> MSA_ERR_INVALID_ARG.
 */
msa_status msa_plan_export_groups(const msa_plan* plan, msa_stream_t stream, uint8_t* grouped,
                                  int64_t grouped_capacity, int32_t* items,
                                  int64_t item_capacity, int32_t* ftasks,
                                  int64_t ftask_capacity);

/*
 * Compaction of padded packed rows into the compact THD layout, and back
 * (the steps either side of the operation when documents arrive packed into
 * fixed-length rows with trailing padding: NeMo-Automodel PR "feat(minimax-m3):
 * add SM100 MSA sparse attention with custom backward", section "Design" -
 * padding tokens are dropped before the flat attention call and the output is
 * scattered back).  The pages print no interface for them; these are plain
 * row gathers.
 *
 *   x        [B][S][row_bytes] bytes, row b's tokens 0..row_len[b]-1 are real
 *   row_len  int32 [B] device; each value must lie in [0, S] (values outside
 *            are clamped into it)
 *   y        [T][row_bytes] bytes, T = sum of row_len, rows in (b, s) order
 *   row_offsets int32 [B+1] device: exclusive prefix sum of row_len
 *            (written by msa_pack_thd, read by msa_unpack_bshd)
 * row_bytes must be a positive multiple of 16 and all pointers 16-byte
 * aligned; B >= 1, S >= 1, B * S < 2^31.  The caller sizes y for T rows (it
 * knows the lengths; T <= B * S always suffices).  msa_unpack_bshd writes
 * zeros into the padding rows of x.  Both are asynchronous on the stream.
 * Errors: MSA_ERR_INVALID_ARG (null pointer, bad sizes), MSA_ERR_ALIGNMENT,
 * MSA_ERR_CUDA (launch failure).
 */
msa_status msa_pack_thd(const void* x, int32_t B, int32_t S, int32_t row_bytes,
                        const int32_t* row_len, void* y, int32_t* row_offsets,
                        msa_stream_t stream);
msa_status msa_unpack_bshd(const void* y, int32_t B, int32_t S, int32_t row_bytes,
                           const int32_t* row_len, const int32_t* row_offsets, void* x,
                           msa_stream_t stream);

/*
 * Block selection: the index scorer and top-16 choice that produce q2k (the
 * step upstream of the plan: NeMo-Automodel PR "feat(minimax-m3): add SM100
 * MSA sparse attention with custom backward", sections "Summary" and
 * "Design" - an indexer picks, per query and index head, the top-16
 * document-local key blocks).  The pages give no scoring formula; this call
 * implements the plainest reading:
 *   summary(g, d, v) = mean of the index keys ik[j, g, :] of document block v
 *   score(t, g, v)   = dot(iq[t, g, :], summary(g, d, v))  for v = 0 .. b,
 * b = the query's own block.  With b + 1 <= 16 all candidates are selected;
 * otherwise the 16 best by (score descending, block ascending), and with
 * force_local != 0 blocks 0 and b are always kept (plus the 14 best of
 * 1 .. b-1).  Slots hold the blocks in ascending order, then -1.  Scores are
 * fp32: block sums key by key divided by the key count, dot products channel
 * by channel with fused multiply-adds (a fixed order, so the ranking is
 * reproducible).
 *   iq, ik       bf16 [T][4][dim] device, dim in {8, 16, ..., 128}; finite
 *   doc_offsets  int32 [num_docs+1] device, valid as for msa_build_plan
 *   q2k          int32 [4][T][16] device (output)
 *   workspace    msa_select_workspace_bytes(T, num_docs, dim) bytes, 16-byte
 *                aligned (block summaries)
 * Asynchronous on the stream.  Errors: MSA_ERR_INVALID_ARG, MSA_ERR_ALIGNMENT,
 * MSA_ERR_WORKSPACE, MSA_ERR_CUDA.
 */
msa_status msa_select_workspace_bytes(int64_t T, int32_t num_docs, int32_t dim, size_t* bytes);
msa_status msa_select_blocks(const void* iq, const void* ik, int64_t T, int32_t dim,
                             const int32_t* doc_offsets, int32_t num_docs, int32_t force_local,
                             int32_t* q2k, void* workspace, size_t workspace_bytes,
                             msa_stream_t stream);

/*
 * Serving: a paged key-value cache
 * --------------------------------
 * A model trained with this attention is run token by token from a cache in
 * pages.  A step of a batch of rows (sequences) is
 *
 *   msa_paged_append   rotate the new tokens' keys (and queries) by their
 *                      positions, write keys and values into the cache
 *   msa_paged_index    write the new tokens' index keys, renew block means
 *   msa_paged_select   the top-16 blocks of each row's newest token (q2k)
 *   msa_paged_decode   attention of each row's newest token over the cache:
 *                      over all keys, or over the blocks of q2k
 *
 * A prompt goes through append and index in one call for all its tokens.  If
 * it begins at position 0 and has the shape that these calls take (64 query and
 * 4 key heads of 128 channels, bf16), the rotated queries and keys that append
 * hands back go through msa_select_blocks, msa_build_plan and msa_forward.
 * There is no call that selects for all tokens of a prompt behind a cached
 * prefix at once.  Each such token can be a row of its own in select and
 * decode, with the same pages and its own length, once all of them have been
 * appended and indexed; the prefix is then read once for each token.  select
 * is right for such rows with force_local alone: the mean of a token's own
 * block already holds the keys behind it.  Over every key, up to 64 of them
 * are one row of msa_paged_tree (below), which reads the prefix once.
 *
 * Rows and pages.  Token j of row r lives in page page_table[r][j / S], slot
 * j % S, S the page size.  A row's table entries past its tokens are never
 * read.  Pages may be shared between rows for reading.  A page id outside
 * [0, num_pages) that is needed, a position or length outside the row's
 * table, sets MSA_ERR_BAD_PAGE in the status word and what it concerns is
 * left out as each call says; nothing outside the given buffers is touched.
 *
 * Status.  `status` is a device word of the caller's, zero at first, to which
 * the calls OR (1 << msa_status) (msa_paged_read_status reads it); it is
 * never cleared by the library, and no call does less because it is set.
 *
 * Calls are asynchronous on the stream, allocate nothing and can be captured
 * into a CUDA graph (make one such call on the device before, which loads the
 * kernels); sizes that change from step to step (positions, lengths) are read
 * on the device.  Inputs and outputs must not overlap except where a call says
 * so.  Keys, values and queries that are used are finite; what lies in a page
 * where no token has been written may be anything.
 */
typedef enum msa_dtype { MSA_BF16 = 0, MSA_F16 = 1 } msa_dtype;

/* Keys and values in pages, each [num_pages][page_size][kv_heads][head_dim]
 * with the given strides (in elements: of a page, of a token in a page, of a
 * head; a head's channels are contiguous), so head-major pages work as well.
 * page_size is a power of two up to 1024, kv_heads 1 .. 64, head_dim 64 or
 * 128; strides are positive multiples of 8, k and v 16-byte aligned. */
typedef struct msa_paged_cache {
  void* k;
  void* v;
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;       /* an msa_dtype */
  int64_t* status;     /* device word */
} msa_paged_cache;

/* Index keys in pages, bf16 [num_pages][page_size][heads][dim] with strides
 * as above (dim 8, 16, .. 128; heads 1 .. 64; page_size a power of two up to
 * 1024), and the means of 128-key blocks, fp32 [slots][heads][dim]
 * contiguous, slots = num_pages * max(1, page_size / 128).  A block's mean is
 * kept with the page of the last key it has so far: slot = page id, or for
 * pages of more than 128 tokens page id * (page_size / 128) + block in page.
 * Rows that share a page thus share the means of the blocks that end in it. */
typedef struct msa_paged_index_cache {
  void* keys;
  int64_t key_stride[3];
  float* means;
  int64_t num_pages;
  int32_t page_size;
  int32_t heads;
  int32_t dim;
  int32_t reserved;
  int64_t* status;
} msa_paged_index_cache;

/* Page table of a call: int32 [rows][width] device, rows `stride` entries
 * apart (stride >= width); 1 <= rows <= 65536, 1 <= width,
 * width * page_size <= 2^30. */
typedef struct msa_page_table {
  const int32_t* pages;
  int64_t stride;
  int32_t rows;
  int32_t width;
} msa_page_table;

/* Synchronises the stream and returns the lowest-numbered status set in the
 * device word (MSA_OK if none). */
msa_status msa_paged_read_status(const int64_t* status, msa_stream_t stream);

/*
 * Append.  The call's tokens are compact: row r owns tokens row_offsets[r]
 * .. row_offsets[r+1]-1, which go to positions start_pos[r], start_pos[r]+1,
 * ...  Tokens at row_offsets[rows] and behind (padding of a captured batch)
 * are skipped: q, k and v hold T tokens, whatever the padding's values, and
 * nothing is written for it.
 *   k, v   [T][kv_heads][head_dim] of the cache's type, tokens k_stride /
 *          v_stride elements apart (multiples of 8)
 *   q      [T][q_heads][head_dim] or NULL, tokens q_stride elements apart
 *   inv_freq fp32 [rotary_dim / 2] device, or NULL for no rotation
 *          (rotary_dim is then ignored); rotary_dim a multiple of 16, at most
 *          head_dim
 *   interleaved 0: channel i pairs with i + rotary_dim / 2; 1: 2 i with 2 i + 1
 *   q_out  contiguous [T][q_heads][head_dim], rotated q (required with q; may
 *          be q itself when q is contiguous)
 *   k_out  contiguous [T][kv_heads][head_dim] rotated keys, or NULL
 * Pair i of a token at position p turns by p * inv_freq[i] (the product and
 * its reduction in 64 bits, the rotation in 32, one rounding); channels from
 * rotary_dim on are copied.  A token whose place is bad is skipped
 * (MSA_ERR_BAD_PAGE); offsets that do not start at 0, decrease or pass T set
 * MSA_ERR_BAD_OFFSETS, and tokens that no row owns are skipped: a row owns
 * those of its tokens that lie below T, and none if its offset is negative
 * (where offsets decrease, one token may be two rows', and which of them
 * append takes is not defined).  Two tokens
 * of one call must not have the same place.  1 <= T <= 2^20.
 */
msa_status msa_paged_append(const msa_paged_cache* cache, const msa_page_table* table,
                            const int32_t* row_offsets, const int32_t* start_pos, int64_t T,
                            const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const void* q, int64_t q_stride, int32_t q_heads,
                            const float* inv_freq, int32_t rotary_dim, int32_t interleaved,
                            void* q_out, void* k_out, msa_stream_t stream);

/*
 * Index keys of new tokens (tokens, rows and padding as for append):
 *   ik  bf16 [T][heads][dim], tokens ik_stride elements apart (a multiple of 8)
 * Writes them into their pages and the mean of every block that got a token:
 * the fp32 sum of the block's keys up to the row's last new token, in
 * order of position, divided by their number - the summary that
 * msa_select_blocks forms.  A block one of whose pages is bad is left out
 * with all its tokens (MSA_ERR_BAD_PAGE).
 */
msa_status msa_paged_index(const msa_paged_index_cache* cache, const msa_page_table* table,
                           const int32_t* row_offsets, const int32_t* start_pos, int64_t T,
                           const void* ik, int64_t ik_stride, msa_stream_t stream);

/*
 * Block selection for one new token of each row, the one at kv_len[r] - 1:
 * scores, candidates, force_local and ties as for msa_select_blocks, with the
 * same fp32 operations in the same order, so that both calls choose the same
 * blocks for the same keys.
 *   iq      bf16 [rows][heads][dim] contiguous; finite
 *   kv_len  int32 [rows] device, tokens of each row, the new one included;
 *           0 marks a row that is not in use (its slots are all -1)
 *   q2k     int32 [heads][rows][16] (written)
 * The means of the scored blocks must be there (msa_paged_index).  A block
 * whose page is bad is not chosen (MSA_ERR_BAD_PAGE); a row with a bad length
 * gets -1 in all slots.
 */
msa_status msa_paged_select(const msa_paged_index_cache* cache, const msa_page_table* table,
                            const int32_t* kv_len, const void* iq, int32_t force_local,
                            int32_t* q2k, msa_stream_t stream);

/* Bytes of decode workspace for `rows` rows and q_heads query heads (host
 * only; an upper bound for every device of this kind). */
msa_status msa_paged_decode_workspace_bytes(const msa_paged_cache* cache, int32_t rows,
                                            int32_t q_heads, size_t* bytes);

/*
 * Attention of one token of each row over the cache.
 *   q       [rows][q_heads][head_dim] contiguous, of the cache's type;
 *           q_heads = kv_heads * n, 1 <= n <= 16; query head h reads key head
 *           h / n
 *   kv_len  int32 [rows] device: row r attends keys 0 .. kv_len[r]-1 (the
 *           new token's key, at kv_len[r]-1, has been appended)
 *           rows * kv_heads * width * page_size of the table <= 2^36; what is
 *           launched follows the table's width, so a table much wider than the
 *           rows need costs few short rows without q2k 1 to 2 us
 *   q2k     int32 [kv_heads][rows][16] device, or NULL: of these keys only
 *           those whose block (key / 128) is in the set q2k[g][r][:], -1 = an
 *           unused slot.  Other values outside [0, blocks of the row) set
 *           MSA_ERR_BAD_Q2K and are left out.
 *   o       [rows][q_heads][head_dim] contiguous, of the cache's type
 *   lse     fp32 [rows][q_heads] natural log
 *   workspace  device, 16-byte aligned, >= msa_paged_decode_workspace_bytes;
 *           needs no initialisation; calls that may overlap in time (on two
 *           streams, in graphs replayed side by side) need one each
 * Results are the same from call to call on one device: how the keys are split
 * depends on the lengths, the sizes (the table's width is one of them) and the
 * device alone.  Two devices of one kind may split them differently, and results
 * then differ by the rounding of 32-bit sums.
 * MSA_ERR_TIMEOUT in the status word: a bounded wait of the kernel gave up, and
 * outputs of that call are missing.
 * A row that sees no key (kv_len 0, no slot used) gets O = 0, LSE = -inf; so
 * does a row whose length is bad.  Keys in a bad page are left out.  What
 * lies in a page past a row's length does not matter, whatever it is.
 */
msa_status msa_paged_decode(const msa_paged_cache* cache, const msa_page_table* table,
                            const int32_t* kv_len, const void* q, int32_t q_heads,
                            float softmax_scale, const int32_t* q2k, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Norm and rotation of queries and keys, head by head: what stands between the
 * projections and the attention, in training (msa_forward) and in serving
 * (msa_paged_append without inv_freq, msa_paged_tree, msa_paged_decode).
 *   n = 1 / sqrt(mean(x^2) + eps) over a head's channels, y = x n w,
 * then pair i of a token at position p turns by p * inv_freq[i] as in
 * msa_paged_append; channels from rotary_dim on are not turned.
 *   q, k   [T][q_heads / k_heads][head_dim] of `dtype`, tokens q_stride /
 *          k_stride elements apart (multiples of 8, a token's heads contiguous:
 *          slices of one projection will do); head_dim 64 or 128, heads 1 .. 1024
 *   q_weight, k_weight  [head_dim] of weight_dtype, an msa_dtype or MSA_F32
 *   positions int32 [T] device, any values; NULL without inv_freq
 *   inv_freq  fp32 [rotary_dim / 2], or NULL for no rotation (rotary_dim is then
 *          ignored); rotary_dim a multiple of 16, at most head_dim
 *   interleaved as for msa_paged_append
 *   q_out, k_out  contiguous; q_out may be q itself and k_out k itself where that is
 *          contiguous, else they must not overlap the inputs or one another
 * Sums, norms and rotation are 32 bits, angles 64, and each result is rounded
 * once.  eps >= 0, finite (with eps = 0 a head of zeros gives NaN, as the formula
 * does); 1 <= T <= 2^20.
 *
 * The backward takes the gradients dq_out, dk_out (contiguous) of the results,
 * with q and k as the forward got them, and returns
 *   g = dy turned back, dx = n (g w - u mean(g w u)), dw = sum over tokens and
 *   heads of g u,  u = x n,
 * dq, dk contiguous of `dtype`, dq_weight and dk_weight fp32 [head_dim].  dq, dk
 * must not overlap the inputs.  The same call on the same device gives the same
 * bits.  workspace: device, 16-byte aligned, >= msa_norm_rope_workspace_bytes,
 * one for calls that may overlap in time.
 * Errors: MSA_ERR_INVALID_ARG, MSA_ERR_ALIGNMENT (tensors 16 bytes, weights,
 * positions and inv_freq their element), MSA_ERR_WORKSPACE, MSA_ERR_CUDA.
 */
#define MSA_F32 2 /* weight_dtype alone */
typedef struct msa_norm_rope_args {
  const void* q;
  const void* k;
  int64_t q_stride;
  int64_t k_stride;
  const void* q_weight;
  const void* k_weight;
  const int32_t* positions;
  const float* inv_freq;
  int64_t T;
  int32_t q_heads;
  int32_t k_heads;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t dtype;        /* an msa_dtype */
  int32_t weight_dtype;
  float eps;
} msa_norm_rope_args;
msa_status msa_norm_rope(const msa_norm_rope_args* args, void* q_out, void* k_out,
                         msa_stream_t stream);
msa_status msa_norm_rope_workspace_bytes(int32_t head_dim, size_t* bytes);
msa_status msa_norm_rope_backward(const msa_norm_rope_args* args, const void* dq_out,
                                  const void* dk_out, void* dq, void* dk, float* dq_weight,
                                  float* dk_weight, void* workspace, size_t workspace_bytes,
                                  msa_stream_t stream);

/*
 * Drafted tokens
 * --------------
 * Several new tokens of a row in one step.  Row r's tokens row_offsets[r] ..
 * row_offsets[r+1]-1 (at most 64; T in all, what lies behind row_offsets[rows]
 * is padding) form a tree: token j continues token parents[j] of its row, a
 * number below j, or what is cached (-1).  The row's token j lies in the cache
 * behind the kv_len[r] tokens that are there to stay, at slot kv_len[r] + j;
 * its position in the text is kv_len[r] plus its depth.  A step is
 *
 *   msa_norm_rope     (or a rotation of the caller's) with those positions
 *   msa_paged_append  without inv_freq, start_pos = kv_len: keys and values
 *   msa_paged_select  a row for each token, with kv_len its row's: the blocks
 *                     of the cached tokens that it attends (q2k)
 *   msa_paged_tree    attention
 *   msa_tree_verify   which tokens stay, and the token behind them
 *   msa_paged_compact moves those together; kv_len grows by their number
 *   msa_paged_index   index keys of the tokens that stay
 *
 * With parents NULL every token continues the one before it: a chain of drafts,
 * or up to 64 tokens of a prompt behind a cached prefix.
 *
 * msa_paged_tree: attention of such tokens.  Token t of row r sees the cached
 * keys 0 .. kv_len[r]-1 (with q2k those in blocks of its own q2k[g][t][:]), and
 * of the drafted ones itself, its parent, its parent's parent and so on.
 *   q       [T][q_heads][head_dim] contiguous, of the cache's type;
 *           q_heads = kv_heads * n, 1 <= n <= 16; query head h reads key head
 *           h / n
 *   row_offsets int32 [rows + 1], kv_len int32 [rows], parents int32 [T] or
 *           NULL, all device; rows * kv_heads * width * page_size of the table,
 *           times ceil(n / 4), <= 2^34
 *   q2k     int32 [kv_heads][T][16] device, or NULL: every cached key.  -1 = an
 *           unused slot; other values outside [0, blocks of the kv_len[r] cached
 *           tokens) set MSA_ERR_BAD_Q2K and are left out
 *   o       [T][q_heads][head_dim] contiguous, of the cache's type
 *   lse     fp32 [T][q_heads] natural log
 *   workspace  device, 16-byte aligned, >= msa_paged_tree_workspace_bytes for
 *           these rows, T and q_heads;
 *           needs no initialisation; one for each of the calls that may overlap
 *           in time
 * Weights are rounded to the cache's type before the product with the values
 * (the sum under them is not); all else is 32 bits.  Results are the same from
 * call to call on one device.
 * Keys that a token does not see may hold anything, and so may the values of
 * drafted tokens that it does not see.  The cached tokens' values are finite: with
 * q2k one that is not may reach all tokens of its row.
 * Values of a bf16 cache that are seen are at most 2^60 in size: weights reach 2^30
 * before they are scaled down, and the sums of 2^30 keys have to stay inside 32 bits.
 * Beyond, a result may be infinite where its exact value is not.
 * Nothing is written for padding.  A row of more than 64 tokens
 * (MSA_ERR_BAD_TREE) and a row whose kv_len plus tokens do not fit its part of
 * the table (MSA_ERR_BAD_PAGE) get O = 0, LSE = -inf.  A bad parent is taken as
 * -1 (MSA_ERR_BAD_TREE).  Offsets as for msa_paged_append; a row whose offsets
 * are negative, decrease or pass T has no tokens (MSA_ERR_BAD_OFFSETS).  Keys in
 * a bad page are left out (MSA_ERR_BAD_PAGE); a token all of whose keys are gets
 * O = 0, LSE = -inf.  MSA_ERR_TIMEOUT as for msa_paged_decode.  1 <= T <= 2^20.
 */
msa_status msa_paged_tree_workspace_bytes(const msa_paged_cache* cache, int32_t rows, int64_t T,
                                          int32_t q_heads, size_t* bytes);
msa_status msa_paged_tree(const msa_paged_cache* cache, const msa_page_table* table,
                          const int32_t* row_offsets, const int32_t* kv_len,
                          const int32_t* parents, int64_t T, const void* q, int32_t q_heads,
                          float softmax_scale, const int32_t* q2k, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities.  A row's
 * token 0 stands already; the walk begins there.  At token c it tries the tokens
 * whose parent is c, in order of their number, and goes on from the first that it
 * keeps.  With x = tokens[j], p = target[c], q = draft[c], S = 1 and r = p at first:
 *   with draft     keep j if u[j] q(x) < r(x) f, f = fp32(1 / S); else
 *                  r = max(r f - q, 0) for every token, S = sum of r.  f = 0 where
 *                  1 / S passes fp32's range: so little is left that it is nothing
 *   without        (drafts that were not drawn) keep j if r(x) > 0 and
 *                  u[j] S < r(x); else S = S - r(x), r(x) = 0
 * Where none is kept (there may be no child), the row's last token is drawn: the
 * first x of r(0) + .. + r(x) > u_last[row] * (the sum of r).  r all zero: p itself
 * is taken for it.  With u uniform on [0, 1) and drafts drawn from q independently
 * of one another the row's tokens are distributed as the target's.  r is 32 bits,
 * rounded after each operation; sums are 64 bits (up to 2^-40 of the sum), and so
 * are the comparisons.
 *   target  fp32 [T][vocab] device, rows target_stride elements apart: row t the
 *           distribution behind token t, not negative, sum 1; any alignment of 4
 *   draft   the same for the drafting model, draft_stride; or NULL
 *   tokens  int32 [T], u fp32 [T] (what they hold for tokens 0 does not matter)
 *   parents int32 [T] or NULL (a chain), u_last fp32 [rows]
 *   path    int32 [rows][max_path]: the numbers, within the row, of token 0 and the
 *           kept ones, ascending, then -1.  1 <= max_path <= 64; a walk ends at
 *           max_path tokens
 *   count   int32 [rows]: how many they are
 *   last    int32 [rows]: the token behind them; -1 if p has no positive value or
 *           its sum is not finite
 * A token whose parent does not come before it, or that is not in [0, vocab), is
 * not tried.  A row without tokens, of more than 64, or with offsets that decrease
 * or lie outside [0, T] gets count 0, path -1, last -1.
 * 1 <= rows <= 65536, 1 <= T <= 2^20, 1 <= vocab <= 2^24.
 * Asynchronous, no workspace, the same answer from call to call.  Errors:
 * MSA_ERR_INVALID_ARG, MSA_ERR_ALIGNMENT, MSA_ERR_CUDA.
 */
msa_status msa_tree_verify(const float* target, int64_t target_stride, const float* draft,
                           int64_t draft_stride, const int32_t* tokens, const int32_t* parents,
                           const int32_t* row_offsets, int32_t rows, int64_t T, int32_t vocab,
                           const float* u, const float* u_last, int32_t max_path, int32_t* path,
                           int32_t* count, int32_t* last, msa_stream_t stream);

/*
 * Moves the kept tokens of each row together: keys and values at slot kv_len[r] +
 * path[r][i] go to slot kv_len[r] + i, for i = 0 .. count[r]-1, within the row's
 * pages; nothing else in the cache changes.
 *   path    int32 [rows][path_width] device, rows contiguous, 1 <= path_width <= 64;
 *           path[r][0 .. count[r]-1] ascend strictly from 0 or more
 *   count   int32 [rows] device
 *   new_len int32 [rows] device (written, not kv_len itself): kv_len[r] + count[r]
 * A row whose count is not in [0, path_width] or whose path does not ascend
 * (MSA_ERR_BAD_TREE), or one of whose tokens has a bad place (MSA_ERR_BAD_PAGE),
 * is left as it is, new_len = kv_len.  No token that moves may lie in a page of
 * another row.
 */
msa_status msa_paged_compact(const msa_paged_cache* cache, const msa_page_table* table,
                             const int32_t* kv_len, const int32_t* path, int32_t path_width,
                             const int32_t* count, int32_t* new_len, msa_stream_t stream);

/*
 * Kernel timing for benchmarks.  While enabled, every kernel the library
 * launches is bracketed by CUDA events on its launch stream.  msa_profile_read
 * synchronises and returns, for the kernel family named (e.g. "fwd_main",
 * "bwd_main"), the launch count and the summed device time since the last
 * reset.  msa_launch_count returns the number of kernels the library has
 * launched since it was loaded.
 */
msa_status msa_profile_enable(int32_t on);
msa_status msa_profile_reset(void);
msa_status msa_profile_read(const char* name, int64_t* launches, double* total_ms);
int64_t msa_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* MSA_H_ */
