/*
 * dsa.h -- C ABI of the B200 (sm_100a) DeepSeek Sparse Attention hot path.
 *
 * The path has three stages, each a call below, plus one call that runs all
 * three for a decode step:
 *
 *   1. dsa_indexer_scores  lightning-indexer scores with the causal mask
 *        I[t,s] = sum_h w[t,h] * ReLU(q_I[t,h,:] . k_I[s,:])
 *      ("DeepSeek-V3.2-Exp - Keep top-k positions", Indexer.forward listing,
 *       the fp8_index call and "index_score += mask"; the head sum is the fix
 *       in "[WIP] deepseek v32", mlx-lm PR #512).
 *   2. dsa_topk  keep each query's min(k, valid) highest-scoring positions
 *      (same page, the M^sel formula and "topk(min(index_topk, end_pos))").
 *   3. dsa_sparse_mla  absorbed MLA over only the selected latent rows
 *      ("DeepSeek-V3.2-Exp - Apply sparse mask", MQA decode listing:
 *       scores = q.[kv||pe] * scale, the -inf index mask, softmax, P.kv).
 *
 * Shapes and layouts (all device pointers, row-major, no padding unless said):
 *   H_I = 64 indexer heads, D_I = 128 indexer dim, D_QK = 576 (512 latent ||
 *   64 rope), D_V = 512, H = MLA heads (1..128).
 *   offsets  int32 [B+1], device.  Sequence b owns rows [offsets[b],
 *            offsets[b+1]) of BOTH caches; end_pos_b = offsets[b+1]-offsets[b].
 *            Its T query rows sit at absolute positions end_pos_b - T + t.
 *   kv_rows  number of rows the caches were allocated with (>= offsets[B]);
 *            bounds every cache read.
 *   q_idx    [B,T,64,128] bf16, or e4m3 codes (uint8) when idx_dtype=DSA_E4M3
 *   w        [B,T,64] fp32 per-head weights; for e4m3 the per-(t,h) q scale
 *            is already multiplied in, as the listing does before fp8_index
 *   k_idx    [kv_rows,128] bf16 or e4m3 codes;  k_scale [kv_rows] fp32 (e4m3 only)
 *   scores   fp32, row (b,t) starts at scores + (b*T+t)*ld_scores
 *   indices  int32 [B,T,k], sequence-local positions, ascending, -1 padded
 *   q        [B,T,H,576] bf16 absorbed query;  kv [kv_rows,576] bf16
 *   out      [B,T,H,512] bf16 or fp32;  lse [B,T,H] fp32 natural-log, optional
 *
 * Ownership and errors.  The caller allocates and owns every buffer, the
 * workspace included; the library allocates nothing and keeps no state between
 * calls.  Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 * legacy default stream).  Argument errors are returned before anything is
 * launched.  A launch failure returns DSA_ERR_CUDA.  Problems only the device
 * can see (offsets that break the bounds above, an index outside [0,end_pos),
 * a pipeline wait that ran out of time) are written as a DSA status code into
 * *dev_status (device int32, optional, never cleared by the library) and the
 * affected row is skipped or zeroed; read it after synchronising.
 * Device pointers must be 16-byte aligned.
 */
#ifndef DSA_H
#define DSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or enum       */
  DSA_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. H > 128)  */
  DSA_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than required; device: shared by two calls at once */
  DSA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed         */
  DSA_ERR_TIMEOUT = 5,     /* device: a pipeline wait ran out of time   */
  DSA_ERR_BAD_INDEX = 6,   /* device: an index outside [0, end_pos)     */
  DSA_ERR_BAD_OFFSETS = 7  /* device: offsets exceed kv_rows / ld / T   */
} dsa_status_t;

enum { DSA_BF16 = 0, DSA_E4M3 = 1, DSA_F32 = 2 };

/* Largest k accepted by dsa_topk / dsa_sparse_mla (index_topk = 2048). */
#define DSA_MAX_TOPK 2048
/* Largest MLA head count (the 128 heads of the decode listing). */
#define DSA_MAX_HEADS 128

/* Human-readable name of a status code; never NULL. */
const char* dsa_status_string(int status);

/* ABI version of this library (major*100 + minor). */
int dsa_version(void);

/*
 * Stage 1 -- indexer scores ("Keep top-k positions", Indexer.forward: the
 * fp8_index call over k_cache[:end_pos] and "index_score += mask").
 * Writes, for every row (b,t) and every s < end_pos_b:
 *   scores[(b*T+t)*ld_scores + s] = s <= end_pos_b-T+t
 *       ? sum_h w[b,t,h] * ReLU(q_I[b,t,h,:] . k_I[offsets[b]+s,:]) (* k_scale for e4m3)
 *       : -inf
 * Entries at s >= end_pos_b are not touched.  ld_scores >= max end_pos, a
 * multiple of 4.  Bytes read: the key cache once, q_I and w once.
 */
int dsa_indexer_scores(const void* q_idx, const float* w, const void* k_idx,
                       const float* k_scale, int idx_dtype, const int32_t* offsets,
                       int B, int T, int64_t kv_rows, float* scores, int64_t ld_scores,
                       int32_t* dev_status, void* stream);

/*
 * Stage 2 -- top-k ("Keep top-k positions": topk(min(index_topk, end_pos))
 * and M^sel).  For row (b,t) the valid positions are s < min(end_pos_b,
 * end_pos_b-T+t+1) (the causal prefix); it keeps k_eff = min(k, #valid) of
 * them, ordered by larger score first and then lower position (-0.0 == +0.0),
 * and writes them ascending into indices[(b*T+t)*k ...], then -1 up to k.
 * Deterministic: the same scores always give the same indices.  1 <= k <= 2048.
 */
int dsa_topk(const float* scores, int64_t ld_scores, const int32_t* offsets, int B, int T,
             int k, int32_t* indices, int32_t* dev_status, void* stream);

/*
 * Stage 3 -- sparse absorbed MLA ("Apply sparse mask", MQA decode listing).
 * For each row r=(b,t), head h, the selected positions j (indices >= 0):
 *   l_j = scale * q[r,h,:576] . kv[offsets[b]+j, :576];  p = softmax_j(l)
 *   out[r,h,:] = sum_j p_j * kv[offsets[b]+j, :512];  lse[r,h] = log sum_j exp(l_j)
 * Rows with no selected position get out = 0, lse = -inf.  Indices outside
 * [0,end_pos_b) are treated as empty and reported as DSA_ERR_BAD_INDEX.
 * workspace: dsa_sparse_mla_workspace_size(B,T,H,k) bytes (may be 0 -> NULL ok).
 */
size_t dsa_sparse_mla_workspace_size(int B, int T, int H, int k);
int dsa_sparse_mla(const void* q, const void* kv, const int32_t* offsets, const int32_t* indices,
                   int B, int T, int H, int k, float scale, int64_t kv_rows, void* out,
                   int out_dtype, float* lse, void* workspace, size_t ws_bytes,
                   int32_t* dev_status, void* stream);

/*
 * The whole decode step (T = 1): stages 1 -> 2 -> 3 on `stream`, scores and
 * indices kept in the workspace.  max_end_pos bounds every end_pos_b (it sets
 * the workspace's score pitch).  Same layouts as above with T = 1.  When
 * max_end_pos <= k every sequence keeps all of its positions, so stages 1 and
 * 2 are skipped (the workspace's scores and indices are then not written) and
 * stage 3 attends to each whole cache.
 * workspace: dsa_decode_step_workspace_size(B, max_end_pos, k, H) bytes.
 */
size_t dsa_decode_step_workspace_size(int B, int max_end_pos, int k, int H);
/*
 * Kernels one dsa_decode_step call launches for these sizes (the indexer and
 * the selection are skipped when max_end_pos <= k: every position is then
 * kept whatever the scores, as the MLX port does below the top-k size).
 * -1 for invalid sizes.  Useful to budget CUDA-graph nodes.
 */
int dsa_decode_step_launches(int B, int max_end_pos, int k, int H);
int dsa_decode_step(const void* q_idx, const float* w, const void* k_idx, const float* k_scale,
                    int idx_dtype, const void* q, const void* kv, const int32_t* offsets, int B,
                    int max_end_pos, int64_t kv_rows, int k, int H, float scale, void* out,
                    int out_dtype, float* lse, void* workspace, size_t ws_bytes,
                    int32_t* dev_status, void* stream);

/*
 * Cache write of the newest tokens ("Keep top-k positions", Indexer.forward:
 * k_cache[start:end] = k after act_quant; the latent cache write of the MLA
 * listing).  For every sequence b and new token t < T, the row
 * offsets[b+1] - T + t (the sequence's last T rows) of each cache gets:
 *   kv_cache  <- kv_new[b,t,:576] (bf16 copy)                 if kv_new != NULL
 *   k_idx_cache <- k_new[b,t,:128]                            if k_new  != NULL
 *     bf16 (idx_dtype DSA_BF16): copied;
 *     e4m3 (DSA_E4M3): act_quant of the 128-vector -- scale = amax/448 in fp32
 *     (1 when amax = 0), codes = nearest e4m3 of x/scale (ties to even,
 *     saturating), the scale stored in k_scale_cache[row].
 * k_new [B,T,128] bf16, kv_new [B,T,576] bf16 (device, 16-byte aligned).
 * Offsets that break the bounds are reported in *dev_status and skipped.
 */
int dsa_cache_append(const void* k_new, const void* kv_new, const int32_t* offsets, int B, int T,
                     int idx_dtype, void* k_idx_cache, float* k_scale_cache, void* kv_cache,
                     int64_t kv_rows, int32_t* dev_status, void* stream);

/*
 * Indexer pre-stage ("Keep top-k positions", Indexer.forward, before
 * act_quant): for every 128-vector x[r, v, :] (bf16; r < n_rows, v <
 * vec_per_row -- the 64 heads of a query row, or one key per row)
 *   1. rotary embedding of the rope part, entries 0..63, not interleaved:
 *      entry i < 32 pairs with entry i + 32 and (a, b) becomes
 *      (a*cos - b*sin, a*sin + b*cos), cos/sin = rope_cos/rope_sin[pos[r], i]
 *      (the freqs_cis table, [rope_len, 32] fp32, row-major); the result is
 *      rounded to bf16;
 *   2. rotate_activation: the Walsh-Hadamard transform of the 128 entries in
 *      Sylvester order, scaled by 128^-1/2, rounded to bf16 into y[r, v, :].
 * y may equal x.  x, y, rope_cos, rope_sin 16-byte aligned (device).  A
 * position outside [0, rope_len) leaves that row's vectors untouched and is
 * reported in *dev_status as DSA_ERR_BAD_INDEX.
 */
int dsa_indexer_prestage(const void* x, const int32_t* pos, int n_rows, int vec_per_row, const float* rope_cos,
                         const float* rope_sin, int rope_len, void* y, int32_t* dev_status, void* stream);

/*
 * act_quant of the indexer queries for the e4m3 path (Indexer.forward:
 * q_fp8, q_scale = act_quant(q) and weights * q_scale): for every row and
 * head the 128-vector q_idx[row,h,:] (bf16) becomes e4m3 codes
 * q_idx_e4m3[row,h,:] with the rule of dsa_cache_append, and
 * w_out[row,h] = w[row,h] * scale (fp32).  n_rows = B*T.
 */
int dsa_quantize_queries(const void* q_idx, const float* w, int n_rows, void* q_idx_e4m3, float* w_out,
                         void* stream);

/*
 * Host <-> device copies done by a kernel (not a copy engine), so that a step
 * fed from host buffers stays one chain of kernel launches on `stream`.
 * dsa_copy_host_to_device: dst (device) <- src_host; dsa_copy_device_to_host:
 * dst_host <- src (device).  The host buffer must be page-locked and mapped
 * into the device's address space as one allocation (cudaHostAlloc, or
 * torch's pin_memory); this is checked at both ends of the range and anything
 * else returns DSA_ERR_INVALID_ARG, as do null pointers, pointers not 16-byte
 * aligned and sizes that are not a multiple of 16.  bytes = 0 does nothing.
 * The copy waits for the previous kernel in the stream; the host may read
 * dst_host once the stream has been synchronised.  The caller keeps
 * ownership of both buffers.
 */
int dsa_copy_host_to_device(void* dst, const void* src_host, size_t bytes, void* stream);
int dsa_copy_device_to_host(void* dst_host, const void* src, size_t bytes, void* stream);

/*
 * Stage 3 without a caller workspace.  The paper has no counterpart: this is
 * a convenience of this library, not a step of the method.
 *
 * For callers that cannot allocate device memory where they issue the step
 * (a plugin inside a runtime that owns all device memory and offers no
 * allocator, a serving loop whose memory is fixed at start-up, code that may
 * not call cudaMalloc on that path).  Same arguments, layouts and results as
 * dsa_sparse_mla, minus the workspace: the split partials live in a scratch
 * array of DSA_NOALLOC_SCRATCH_BYTES (32 MiB) built into the library, which
 * every GPU that loads the library holds until the process exits.
 *   - A call that needs more scratch than that (dsa_sparse_mla_workspace_size
 *     above the limit; e.g. 128..147 rows at H = 128, k = 2048) returns
 *     DSA_ERR_WORKSPACE before launching anything.
 *   - The first call on each device looks the scratch address up with
 *     cudaGetSymbolAddress (with that device current); make that first call
 *     before any stream capture.  It allocates nothing, ever.
 *   - All calls on a device share the one scratch array: calls that may run
 *     concurrently on the GPU (different streams, no ordering between them)
 *     race and corrupt each other's results.  Order them on one stream.
 *   - Nothing in the scratch needs to start at zero: every value a call reads
 *     was written earlier in the same call.
 */
#define DSA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int dsa_sparse_mla_noalloc(const void* q, const void* kv, const int32_t* offsets,
                           const int32_t* indices, int B, int T, int H, int k, float scale,
                           int64_t kv_rows, void* out, int out_dtype, float* lse,
                           int32_t* dev_status, void* stream);

/*
 * Test hook for the device-side timeout path.  The paper has no counterpart:
 * it exists so that a test can make a pipeline wait run out on purpose
 * without faulting or hanging the GPU.
 *
 * The next n_launches attention launches in this process (from
 * dsa_sparse_mla, dsa_decode_step, dsa_sparse_mla_noalloc, dsa_paged_mla or
 * dsa_paged_weights) initialise their query barrier with one expected arrival
 * more than will ever come, and limit every pipeline wait to wait_limit_ns
 * (1 ms to 1 s).  The wait runs out; the kernel stops its pipeline, waits
 * (bounded) for its own copies and tensor
 * core work, releases its tensor memory and writes DSA_ERR_TIMEOUT into
 * *dev_status.  The output of such a launch is undefined; the launches after
 * it run normally.  n_launches = 0 cancels.  Returns DSA_ERR_INVALID_ARG for
 * a negative count or a limit outside the range.  Launches captured in a
 * CUDA graph keep the setting they were captured with.
 * With DSA_STALL_AT_PRODUCT added to n_launches, a dsa_paged_mla launch stalls
 * later: scores run, messages between SMs are on their way, and the first
 * product with the values is never issued.
 */
#define DSA_STALL_AT_PRODUCT (1 << 30)
int dsa_debug_stall_attention(int n_launches, uint64_t wait_limit_ns);

/*
 * ---------------------------------------------------------------- paged cache
 *
 * A latent cache in pages, for serving: the attention of new tokens over the
 * whole of it (layers without an indexer, contexts below the top-k length),
 * the attention weight that each slot collects, and the eviction of the slots
 * that collect least.  The paper has no counterpart: the formulas are those
 * of dsa_sparse_mla over every position.
 *
 *   kv_pages   [n_pages, page_size, 576] bf16, the pool of all sequences.
 *              page_size is a multiple of 16, n_pages * page_size <= 2^31 - 4096.
 *   page_table int32, row b at page_table + b * ld_table (ld_table >=
 *              max_pages): slot s of sequence b is row
 *              page_table[b, s / page_size] * page_size + s % page_size of the
 *              pool.  Entries behind a sequence's last page are not read.
 *   lens       int32 [B]: slots in use, the T newest tokens included (they sit
 *              in the last T slots; query row t sees the slots s <= lens[b] -
 *              T + t).  0 is an empty sequence (a padded batch) and fine
 *              everywhere; a length outside [0, max_pages * page_size] is
 *              reported as DSA_ERR_BAD_OFFSETS and treated as 0.
 *   acc, pos   fp32 and int32, row b at acc + b * ld_slots: attention weight
 *              collected by, and position of the token in, each slot.
 *              16-byte aligned, ld_slots a multiple of 4 and >= every length.
 * A page number outside [0, n_pages) is reported as DSA_ERR_BAD_INDEX; its
 * slots count as masked.  Slots behind a sequence's length, and pages that no
 * table names, are never written, and what they hold (NaN included) never
 * reaches a result.  All sizes that change from step to step are read on the
 * device, so one captured CUDA graph serves growing and shrinking sequences.
 */

/*
 * Cache write of the T newest tokens of every sequence: slot lens[b] - T + t
 * gets kv_new[b,t,:576], and, where the arrays are given (NULL: left out),
 * acc = 0 and pos = end_pos[b] - T + t.  end_pos int32 [B]: tokens seen so far
 * by the sequence, evicted ones included; needed with pos.  Two sequences may
 * share pages for reading, not the pages written here.
 * 0 < lens[b] < T is reported as DSA_ERR_BAD_OFFSETS and the sequence skipped.
 */
int dsa_paged_append(const void* kv_new, const int32_t* lens, const int32_t* page_table, int64_t ld_table,
                     int max_pages, int B, int T, int page_size, int64_t n_pages, void* kv_pages, float* acc,
                     int32_t* pos, const int32_t* end_pos, int64_t ld_slots, int32_t* dev_status, void* stream);

/*
 * Absorbed MLA of the T newest tokens over the whole paged cache (q, out, lse
 * and scale as for dsa_sparse_mla):
 *   l_s = scale * q[b,t,h,:576] . kv(b,s)[:576],  s <= lens[b] - T + t;  p = softmax_s(l)
 *   out[b,t,h,:] = sum_s p_s * kv(b,s)[:512];  lse[b,t,h] = log sum_s exp(l_s)
 * Rows that see no slot, or whose scores are all -inf, get lse = -inf and
 * out = 0.  (A slot that holds infinities and has weight 0 gives NaN or 0 in
 * their columns; a score of NaN or +inf gives NaN.)
 * The cache is read once per 128 (token, head) rows of a sequence.  The work
 * is divided by the lengths found on the device, so ragged batches need no
 * padding and no plan.  The result does not depend on what else runs; the same
 * inputs give the same bits.
 * Roundings: p is rounded to bf16 before its product with kv (half a step,
 * 2^-8), whatever the output's type; the sum of p that divides it is not.  All
 * sums are fp32, with one exception: with bf16 output and tiles of more than 32
 * rows, the partial sums of a row that several SMs share are stored as scaled
 * fp16 (2^-11) before they are added up.
 * workspace: dsa_paged_mla_workspace_size(B, T, H) bytes, for the current
 * device; its contents need not survive between calls, and calls that may run
 * at the same time (two graphs, two streams) need one each.  Two that share one
 * all the same give wrong results (reported as DSA_ERR_WORKSPACE where it
 * shows), and touch nothing outside their own arrays.
 */
size_t dsa_paged_mla_workspace_size(int B, int T, int H);
int dsa_paged_mla(const void* q, const void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages,
                  const int32_t* lens, int B, int T, int H, int page_size, int64_t n_pages, float scale, void* out,
                  int out_dtype, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * Attention weight that every slot collects from these query rows:
 *   acc_out[b,s] = decay * acc[b,s] + sum_{t,h : s <= lens[b]-T+t} exp(scale * q[b,t,h,:] . kv(b,s) - lse[b,t,h])
 * for s < lens[b]; the other entries of acc_out are not touched.  lse comes
 * from dsa_paged_mla with the same q, scale and cache; rows with lse = -inf
 * add nothing.  acc may be NULL (zeros); acc_out may be acc.  A slot on a bad
 * page gets decay * acc.  The sums' order is fixed: the same inputs always
 * give the same bits.
 */
int dsa_paged_weights(const void* q, const void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages,
                      const int32_t* lens, const float* lse, int B, int T, int H, int page_size, int64_t n_pages,
                      float scale, float decay, const float* acc, float* acc_out, int64_t ld_slots,
                      int32_t* dev_status, void* stream);

/*
 * Which slots stay when every sequence is cut to `budget` slots, and the row
 * moves that close the gaps.  Of sequence b the n = min(budget, lens[b])
 * first slots stay in this order: protected slots (pos >= end_pos[b] -
 * recent; none when recent = 0) before the others, then larger acc, then the
 * lower slot; NaN counts as less than everything, -0 as 0.  Survivors below n
 * stay where they are; the i-th free slot below n takes the i-th survivor at
 * or above n:
 *   new_lens[b] = n,  n_moves[b] = number of moves (<= min(n, lens[b] - n)),
 *   move_dst[b,i] (ascending), move_src[b,i] (ascending), -1 from n_moves[b]
 *   up to ld_moves.
 * Attention does not depend on the order of the slots, so nothing else has to
 * move: the plan touches min(n, evicted) rows at most.  pos and end_pos may
 * be NULL when recent = 0.  0 <= recent <= budget, budget >= 1.  A length
 * outside [0, ld_slots], or more than ld_moves moves, is reported as
 * DSA_ERR_BAD_OFFSETS; that sequence keeps its length and moves nothing.
 * The outputs must not overlap the inputs, but new_lens may be lens.
 * ld_slots above DSA_MAX_PLAN_SLOTS returns DSA_ERR_UNSUPPORTED.
 */
#define DSA_MAX_PLAN_SLOTS (6 << 20)
int dsa_evict_plan(const float* acc, const int32_t* pos, const int32_t* lens, const int32_t* end_pos, int B,
                   int64_t ld_slots, int budget, int recent, int32_t* new_lens, int32_t* n_moves, int32_t* move_dst,
                   int32_t* move_src, int64_t ld_moves, int32_t* dev_status, void* stream);

/*
 * Carries a plan out: for i < n_moves[b] the cache row (and acc, pos where
 * given, NULL: left out) of slot move_src[b,i] goes to slot move_dst[b,i].
 * Moves run in parallel: no slot may be the destination of two moves or the
 * source of one and the destination of another (a plan's never are).  Moves
 * with a slot outside the page list (or ld_slots) or on a bad page are
 * reported as DSA_ERR_BAD_INDEX and left out; an n_moves outside
 * [0, ld_moves] is reported as DSA_ERR_BAD_OFFSETS and its sequence skipped.
 */
int dsa_paged_move(void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages, int page_size,
                   int64_t n_pages, const int32_t* n_moves, const int32_t* move_dst, const int32_t* move_src,
                   int64_t ld_moves, int B, float* acc, int32_t* pos, int64_t ld_slots, int32_t* dev_status,
                   void* stream);

/*
 * Where, inside a decode-step workspace, the step leaves its intermediates
 * (byte offsets; the scores pitch is returned in *ld_scores).  For tests and
 * tools that want to look at stage outputs; the layout may change between
 * versions.
 */
int dsa_decode_step_workspace_layout(int B, int max_end_pos, int k, int H, size_t* scores_off,
                                     int64_t* ld_scores, size_t* indices_off, size_t* mla_off);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H */
