/*
 * fab.h -- C ABI of libfab, the fused attention backward library for one
 * NVIDIA GB300 GPU (sm_103a).
 *
 * The operation is ggml_flash_attn_back: given the forward's inputs q, k, v,
 * the upstream gradient d of the forward output, a softmax scale and an
 * optional causal flag and/or additive f16 mask, return dQ, dK and dV as f32,
 * packed into one buffer.  Sources, by page and section:
 *   - the ggml_flash_attn_back constructor (PowerInfer ggml.c): shape
 *     asserts (k rows match q rows, H % Hkv == 0), f32 result type, and the
 *     packed offsets offs_k = PAD(elem_q*4, 16), offs_v = offs_k +
 *     PAD(elem_k*4, 16), end = offs_v + PAD(elem_v*4, 16);
 *   - the ggmlR test file test-flash-attn-back.R: the call shape
 *     (q, k, v, mask, d, scale), layouts q [DK,N,H,B], k [DK,M,Hkv,B],
 *     v [DV,M,Hkv,B], forward output and d [DV,H,N,B], mask f16 [M,N]
 *     added after scaling (attn_ref), contiguous GQA groups, the causal mask
 *     (query n attends keys 0..n), rows with no finite score giving zero
 *     output, and a zero-filled packed buffer whose padding stays 0;
 *   - the labml "Flash Attention" page, sections "Forward pass", "Flash
 *     Attention Optimization" (online softmax) and "Backward pass": the
 *     gradient formulas, with D_i = dO_i . O_i.
 *
 * Layout convention: every tensor is contiguous in ggml ne order (ne[0]
 * fastest), e.g. q[i, n, h, b] is at i + DK*(n + N*(h + H*b)).
 *   q    [DK, N, H, B]     k [DK, M, Hkv, B]     v [DV, M, Hkv, B]
 *   o, d [DV, H, N, B]     (the forward output and its gradient)
 *   lse  [N, H, B] f32     (natural-log row log-sum-exp of the scaled,
 *                           masked scores; +inf for a row with no finite score)
 *   mask [M, N] f16        (mask[m + M*n] is added to score(n, m); shared by
 *                           every head and batch; only -inf and finite values
 *                           are defined)
 *   packed f32: [dQ as q | 0 pad | dK as k | 0 pad | dV as v | 0 pad],
 *               byte offsets from fab_packed_offsets().
 * Causal masking is top-left: query n attends keys m <= n (also when N != M).
 * When both `causal` and a mask are given, both apply.
 *
 * Ownership and execution: the caller owns every buffer.  Device pointers
 * must point to device memory of the current device and be 16-byte aligned.
 * The library never allocates, frees or synchronises: each compute entry point
 * validates its arguments on the host, enqueues kernels on `stream` and
 * returns.  A status other than FAB_OK means nothing was enqueued, except
 * FAB_ERR_CUDA, which reports a launch error (the stream state is then the
 * CUDA runtime's).  Device-side waits are bounded: a wait that runs out sets
 * an error word that fab_last_device_error() returns as FAB_ERR_TIMEOUT.
 *
 * Supported on the GPU: dtype FAB_F32 (any DK, DV <= 256), FAB_BF16 and
 * FAB_F16 (tensor-core path when DK == DV and DK is 64 or 128, with P and dS
 * rounded to the input type for their products; any DK, DV <= 256
 * otherwise).  Anything else returns FAB_ERR_UNSUPPORTED; there is no CPU
 * fallback.  ALiBi and logit soft-capping are not part of this ABI.
 */
#ifndef FAB_H
#define FAB_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FAB_EXPORT __attribute__((visibility("default")))
#else
#define FAB_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FAB_OK = 0,
  FAB_ERR_INVALID = 1,     /* null/misaligned pointer, bad dims, H % Hkv != 0; or see fab_last_device_error */
  FAB_ERR_UNSUPPORTED = 2, /* valid op, but no GPU kernel for these dims/dtype */
  FAB_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required */
  FAB_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  FAB_ERR_TIMEOUT = 5      /* a device-side wait ran out (see fab_last_device_error) */
} fab_status;

typedef enum {
  FAB_F32 = 0,  /* q, k, v, d, o are float32 */
  FAB_BF16 = 1, /* q, k, v, d, o are bfloat16 */
  FAB_F16 = 2   /* q, k, v, d, o are float16 (IEEE binary16) */
} fab_dtype;

/* Sizes in ggml terms: B batches, H query heads, Hkv key/value heads
 * (H % Hkv == 0; query head h uses key/value head h / (H / Hkv)), N queries,
 * M keys, DK query/key width, DV value width.  All must be positive. */
typedef struct {
  int64_t B, H, Hkv, N, M, DK, DV;
} fab_dims;

/* An opaque cudaStream_t; NULL is the legacy default stream. */
typedef void* fab_stream;

/* Library version, major*10000 + minor*100 + patch. */
FAB_EXPORT int fab_version(void);

/* Human-readable text for a fab_status value; never NULL. */
FAB_EXPORT const char* fab_status_string(int status);

/* Byte offsets of the dK and dV slices and the total size of the packed
 * result (the ggml_flash_attn_back constructor's offs_k, offs_v, end).
 * Returns FAB_ERR_INVALID for bad dims (the outputs are then untouched). */
FAB_EXPORT int fab_packed_offsets(const fab_dims* dims, size_t* off_k, size_t* off_v, size_t* end);

/* Total packed bytes (== end above), or 0 for bad dims. */
FAB_EXPORT size_t fab_packed_bytes(const fab_dims* dims);

/* Device workspace bytes fab_backward needs: D_i = rowsum(dO * O), f32
 * [N,H,B], then, for a call with a mask, the mask's live-tile maps (a byte
 * per 128 x 128 tile, nonzero where some mask entry is not -inf, by query
 * tile rows then by key tile rows, each row padded to 16 bytes; the
 * tensor-core passes skip the tiles before the first and after the last live
 * tile of each row, which changes no result bit; a workspace that ends after
 * D_i skips nothing), each part a multiple of 256 bytes.  0 for bad dims. */
FAB_EXPORT size_t fab_backward_workspace_bytes(const fab_dims* dims, int dtype);

/* Device workspace bytes fab_backward needs when called without o and lse
 * (it then recomputes them): D_i and the live-tile maps as above, then O
 * (`dtype`, [DV,H,N,B]) and LSE (f32, [N,H,B]), each part a multiple of 256
 * bytes.  0 for bad dims. */
FAB_EXPORT size_t fab_backward_recompute_workspace_bytes(const fab_dims* dims, int dtype);

/* Forward pass saving what the backward needs (labml "Flash Attention",
 * "Forward pass" and "Flash Attention Optimization"; ggmlR attn_ref):
 *   o[:, h, n, b] = sum_m softmax_m(scale * q_n . k_m + mask[m + M*n]) v_m
 *   lse[n, h, b]  = log sum_m exp(scale * q_n . k_m + mask[m + M*n])
 * q, k, v: device, `dtype`; mask: device f16 [M,N] or NULL; o: device,
 * `dtype`, [DV,H,N,B]; lse: device f32 [N,H,B].  A query row with no finite
 * score gets o = 0 and lse = +inf. */
FAB_EXPORT int fab_forward_lse(const void* q, const void* k, const void* v, const uint16_t* mask, int causal, float scale,
                    int dtype, const fab_dims* dims, void* o, float* lse, fab_stream stream);

/* Backward pass (ggml_flash_attn_back; labml "Backward pass"):
 *   dV_m = sum_n P_nm dO_n,  dP_nm = dO_n . V_m,  D_n = dO_n . O_n,
 *   dS_nm = P_nm (dP_nm - D_n),  dQ_n = scale sum_m dS_nm K_m,
 *   dK_m = scale sum_n dS_nm Q_n,
 * with P recomputed from q, k, mask, causal, scale and the saved lse; dK and
 * dV are summed over each GQA group's query heads.  o and lse must come from
 * fab_forward_lse on the same inputs; or both be NULL, as in
 * ggml_flash_attn_back, whose operands are q, k, v, the mask and d alone:
 * the call then enqueues fab_forward_lse into the workspace first (exactly one
 * of them NULL is FAB_ERR_INVALID).  d: device, `dtype`, [DV,H,N,B].
 * workspace: device, >= fab_backward_workspace_bytes() bytes (with o and lse
 * NULL: fab_backward_recompute_workspace_bytes()), contents overwritten.  packed_out: device f32, fab_packed_bytes() bytes, fully
 * overwritten (padding written as 0).  Where the tensor-core kernels apply
 * (bf16 or f16, DK == DV in {64, 128}) it enqueues fab_backward_query_pass then
 * fab_backward_key_pass; otherwise fab_backward_preprocess then
 * fab_backward_main. */
FAB_EXPORT int fab_backward(const void* q, const void* k, const void* v, const void* d, const void* o, const float* lse,
                 const uint16_t* mask, int causal, float scale, int dtype, const fab_dims* dims, void* workspace,
                 size_t workspace_bytes, float* packed_out, fab_stream stream);

/* First half of fab_backward (labml "Backward pass", D_i = dO_i . O_i):
 * writes D into the workspace, zeroes the padding of packed_out and, where the
 * main kernel accumulates dQ, the dQ slice.  Same arguments as fab_backward
 * minus those the preprocess does not read. */
FAB_EXPORT int fab_backward_preprocess(const void* d, const void* o, int dtype, const fab_dims* dims, void* workspace,
                            size_t workspace_bytes, float* packed_out, fab_stream stream);

/* Second half of fab_backward: the gradient kernels proper.  Requires the
 * workspace and packed_out as fab_backward_preprocess left them. */
FAB_EXPORT int fab_backward_main(const void* q, const void* k, const void* v, const void* d, const float* lse,
                      const uint16_t* mask, int causal, float scale, int dtype, const fab_dims* dims,
                      const void* workspace, size_t workspace_bytes, float* packed_out, fab_stream stream);

/* The two tensor-core passes that make up fab_backward for bf16 or f16 inputs
 * with DK == DV in {64, 128} (labml "Backward pass"); FAB_ERR_UNSUPPORTED
 * otherwise.  Same arguments as fab_backward.
 * fab_backward_query_pass: D_i = dO_i . O_i into the workspace, the dQ slice
 * of packed_out (dQ_n = scale sum_m dS_nm K_m, recomputing S and dP per query
 * tile) and the padding of packed_out.
 * fab_backward_key_pass: the dK and dV slices of packed_out, reading D_i
 * from the workspace (written by the query pass or fab_backward_preprocess);
 * it does not read o. */
FAB_EXPORT int fab_backward_query_pass(const void* q, const void* k, const void* v, const void* d, const void* o,
                            const float* lse, const uint16_t* mask, int causal, float scale, int dtype,
                            const fab_dims* dims, void* workspace, size_t workspace_bytes, float* packed_out,
                            fab_stream stream);
FAB_EXPORT int fab_backward_key_pass(const void* q, const void* k, const void* v, const void* d, const float* lse,
                          const uint16_t* mask, int causal, float scale, int dtype, const fab_dims* dims,
                          const void* workspace, size_t workspace_bytes, float* packed_out, fab_stream stream);

/* Largest B*H*N that fab_backward_noalloc accepts (query rows times heads
 * times batches): its fixed scratch holds one float per such row. */
#define FAB_NOALLOC_MAX_ROWS 1048576

/* fab_backward for callers that cannot allocate device memory (o and lse
 * must be given: the fixed scratch holds D_i and, when they fit after it, the
 * mask's live-tile maps, not a recomputed O and LSE), for example
 * code whose device memory belongs to another allocator, or code that must not
 * call cudaMalloc (which can synchronise the device) on its path.  The pages
 * have no counterpart; the operation and every argument are those of
 * fab_backward minus the workspace.  The workspace lives instead in a fixed
 * device array inside the library: FAB_NOALLOC_MAX_ROWS floats (4 MiB), held
 * on every GPU that loads the library until the process exits.  Returns
 * FAB_ERR_WORKSPACE when B*H*N exceeds FAB_NOALLOC_MAX_ROWS; allocates and
 * frees nothing.  The first call on a device looks up the array's device
 * address with that device current; make that first call before any stream
 * capture.  The address is kept for the life of the process: after a
 * cudaDeviceReset of that device, do not call this entry point there again.  Calls on one device share the array, so two calls that may run
 * at the same time on the GPU (on unordered streams) race; order them.  No
 * part of the array needs clearing between calls. */
FAB_EXPORT int fab_backward_noalloc(const void* q, const void* k, const void* v, const void* d, const void* o,
                                    const float* lse, const uint16_t* mask, int causal, float scale, int dtype,
                                    const fab_dims* dims, float* packed_out, fab_stream stream);

/* ---- Around the attention: query/key norms with the position rotation ----
 *
 * A projection leaves one row of H*DK queries, Hkv*DK keys and Hkv*DV values
 * for each token, heads contiguous inside a row.  fab_qk_norm_rope turns those
 * rows into fab_forward_lse's q, k and v; fab_qk_norm_rope_backward turns the
 * slices of fab_backward's packed result into the gradient of the rows.
 * With x a head's row, w its weights and r = 1 / sqrt(mean(x^2) + eps):
 *   n = r x w (or n = x without weights),  y = R(pos) n,
 * where R rotates pair i < rot / 2 by the angle whose cosine and sine are
 * cos[i + rot/2*pos] and sin[i + rot/2*pos]: y_a = n_a cos - n_b sin,
 * y_b = n_b cos + n_a sin, with (a, b) = (i, i + rot/2), or (2i, 2i + 1) when
 * `interleaved` is nonzero.  Columns from rot on are not rotated.  Arithmetic
 * is f32, rounded once to the output's type. */
typedef struct {
  int64_t B, N;          /* sequences, tokens in each */
  int64_t H, Hkv;        /* query heads (< 2^31), key/value heads (H % Hkv == 0) */
  int64_t DK, DV;        /* query/key width, value width (<= 256) */
  int64_t rot;           /* rotated columns of q and k: even, 0 .. DK */
  int64_t P;             /* positions held by cos and sin (read when rot > 0) */
  int64_t ldq, ldk, ldv; /* elements from one token's row to the next in q, k, v:
                            q[i, h, n, b] is at i + DK*h + ldq*(n + N*b) */
  int64_t ldgq, ldgk, ldgv; /* the same for gq, gk, gv (backward only) */
} fab_rope_dims;

/* q, k, v: device, `dtype`, rows as above, aligned to their element only (v
 * may be NULL with v_out NULL).  wq, wk: device, `dtype`, [DK], or NULL: that
 * operand is not normalised.  cos, sin: device f32 [rot/2, P].  pos: device
 * int32 [N,B], or NULL: token n is at position n (N <= P).  A position
 * outside 0 .. P-1 is reported by fab_last_device_error as FAB_ERR_INVALID
 * and its token's q_out and k_out are then meaningless.  q_out [DK,N,H,B],
 * k_out [DK,N,Hkv,B], v_out [DV,N,Hkv,B]: `dtype`, as fab_forward_lse reads
 * them; they must not overlap the inputs. */
FAB_EXPORT int fab_qk_norm_rope(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                                const float* cos, const float* sin, const int32_t* pos, float eps, int interleaved,
                                int dtype, const fab_rope_dims* dims, void* q_out, void* k_out, void* v_out,
                                fab_stream stream);

/* Device workspace bytes of fab_qk_norm_rope_backward (partial sums of the
 * weights' gradients); 0 for bad dims. */
FAB_EXPORT size_t fab_qk_norm_rope_backward_workspace_bytes(const fab_rope_dims* dims);

/* With g = R(pos)^T dy and u = g w:  dw = sum over rows of g r x,
 *   dx = r (u - r x mean(u r x))   (dx = g where there are no weights).
 * dq, dk, dv: device f32, [DK,N,H,B], [DK,N,Hkv,B], [DV,N,Hkv,B] (dv NULL with
 * gv NULL).  q, k: the forward's inputs; each is read only when its weights
 * are given, and may be NULL otherwise.  gq, gk, gv: `dtype`, rows of ldgq,
 * ldgk, ldgv elements, aligned to their element only; only the heads' columns
 * are written.  gwq, gwk: device f32 [DK], overwritten (NULL exactly where the
 * weights are).  Sums run in an order that depends on the sizes alone: two
 * calls give the same bits. */
FAB_EXPORT int fab_qk_norm_rope_backward(const float* dq, const float* dk, const float* dv, const void* q,
                                         const void* k, const void* wq, const void* wk, const float* cos,
                                         const float* sin, const int32_t* pos, float eps, int interleaved, int dtype,
                                         const fab_rope_dims* dims, void* workspace, size_t workspace_bytes, void* gq,
                                         void* gk, void* gv, float* gwq, float* gwk, fab_stream stream);

/* ---- The same attention served from a paged key/value cache ----
 *
 * A cache is an array of pages, each holding `page` key (or value) rows of
 * every key/value head: k_cache [DK, page, Hkv, pages], v_cache [DV, page, Hkv,
 * pages].  Sequence b holds lens[b] tokens; token m of it lies in row m % page
 * of page table[m / page + max_pages*b].  One call works on the T new tokens of
 * B sequences laid end to end: sequence b owns tokens starts[b] ..
 * starts[b+1]-1 (starts has B + 1 ascending entries, the first 0), and they are
 * the last of its lens[b] tokens: lens counts them already, for both calls
 * below.  A sequence may have no new token, and tokens from starts[B] on are
 * padding: nothing is written for them.  starts, lens and table are device
 * int32 and are read when the kernels run, so a captured call follows their
 * contents.  A page number outside 0 .. pages-1, a token past max_pages*page
 * or starts that do not ascend within 0 .. T touch no memory outside the
 * arguments; fab_last_device_error reports FAB_ERR_INVALID, and what was
 * computed for those tokens is meaningless. */
typedef struct {
  int64_t B, T;          /* sequences, rows of new tokens (T may be 0; < 2^31 - 256) */
  int64_t H, Hkv;        /* query heads (< 2^31), key/value heads (H % Hkv == 0) */
  int64_t DK, DV;        /* query/key width, value width (<= 256) */
  int64_t page;          /* rows of a page */
  int64_t pages;         /* pages of the cache */
  int64_t max_pages;     /* entries of a sequence's row of the table */
  int64_t rot, P;        /* as in fab_rope_dims (fab_paged_append only) */
  int64_t ldq, ldk, ldv; /* as in fab_rope_dims, by token (fab_paged_append only) */
} fab_paged_dims;

/* Writes the new tokens' keys and values into the cache and their queries into
 * q_out [DK,H,T], norms and rotation as in fab_qk_norm_rope, each token at
 * its place in its sequence (token i of the n new ones is at position
 * lens[b] - n + i, which must be in 0 .. P-1).  q, k, v: [DK,H] rows of ldq, ...
 * elements by token, aligned to their element only; q_out and the caches must not
 * overlap them.  No other row of the caches or of q_out is touched.  A row of the cache that two tokens of one call map
 * to gets either of them. */
FAB_EXPORT int fab_paged_append(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                                const float* cos, const float* sin, float eps, int interleaved, const int32_t* starts,
                                const int32_t* lens, const int32_t* table, int dtype, const fab_paged_dims* dims,
                                void* q_out, void* k_cache, void* v_cache, fab_stream stream);

/* Device workspace bytes of fab_paged_attention on the current device; 0 for bad
 * dims (which fab_paged_attention itself refuses), and for short calls that need
 * none (of few sequences whose rows of the table hold few keys; workspace may then
 * be NULL).  Ask for each call's own sizes: one of fewer tokens can need a
 * workspace where one of more needs none. */
FAB_EXPORT size_t fab_paged_attention_workspace_bytes(const fab_paged_dims* dims, int dtype);

/* Attention of the new tokens over their sequences' caches: token i of the n
 * new ones of sequence b sees keys m < lens[b], and with `causal` only
 * m <= lens[b] - n + i (the last token sees all: aligned at the end, unlike
 * fab_forward_lse's top-left rule).  q [DK,H,T], o [DV,H,T]: `dtype`; lse f32
 * [T,H] (natural log), or NULL.  A token that sees no key gets o = 0 and
 * lse = +inf.  Cache rows from lens[b] on are never read into a result, whatever
 * they hold; rows before it have to be finite: a later token's value takes part in
 * an earlier one's sum with weight 0, which a NaN or an infinity survives.
 * bf16 and f16 calls with DK and DV multiples of 8 up to 128 and pages of a
 * multiple of 8 rows run on the tensor cores, which take the softmax weights of
 * the second product in `dtype`, rounded one by one, as in fab_forward_lse (their
 * sum is not rounded); every other call keeps them in f32.  Scores, maxima, sums and
 * unfinished outputs are f32 in both.  o and lse must not overlap the inputs.
 * workspace: device, fab_paged_attention_workspace_bytes() bytes, contents
 * overwritten; calls that may overlap on the GPU need one each. */
FAB_EXPORT int fab_paged_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* starts,
                                   const int32_t* lens, const int32_t* table, int causal, float scale, int dtype,
                                   const fab_paged_dims* dims, void* workspace, size_t workspace_bytes, void* o,
                                   float* lse, fab_stream stream);

/* ---- Drafted trees ----
 *
 * A draft is a tree of tokens that go on from what a sequence's cache holds: the
 * new tokens of fab_paged_append and fab_paged_attention, of which each sees its
 * ancestors and not the other branches.  Who sees whom is a row of `words`
 * 32-bit words for each of the T tokens: bit j % 32 of word j / 32 of token i's
 * row is set where token i sees new token j of its sequence; only bits j <= i
 * count.  words is at least the largest sequence's new tokens / 32, rounded up (a
 * sequence of more is reported as FAB_ERR_INVALID, its results are meaningless).
 * One step is fab_paged_reserve, fab_draft_tree, then for each layer
 * fab_paged_append_tree and fab_paged_attention_tree, then fab_paged_accept. */

/* Words of a row that fab_draft_tree takes at most (16,384 new tokens). */
#define FAB_DRAFT_MAX_WORDS 512

/* seen [words,T] (device int32, 16-byte aligned): each token's own bit and its
 * ancestors'.  parents [T] (device int32): token i of a sequence follows its token
 * parents[i] < i, or, -1, what the cache held before; anything else is reported
 * as FAB_ERR_INVALID and taken as -1.  starts as above; rows of tokens from
 * starts[B] on are left as they were.  seen may be parents itself where words is 1, and
 * overlaps neither otherwise.  Words past FAB_DRAFT_MAX_WORDS are
 * FAB_ERR_UNSUPPORTED. */
FAB_EXPORT int fab_draft_tree(const int32_t* starts, const int32_t* parents, int64_t B, int64_t T, int64_t words,
                              int32_t* seen, fab_stream stream);

/* fab_paged_append of a draft: token i is written where fab_paged_append writes
 * it, and rotated by the position lens[b] - n + (new tokens before it that it
 * sees): its place on its path. */
FAB_EXPORT int fab_paged_append_tree(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                                     const float* cos, const float* sin, float eps, int interleaved,
                                     const int32_t* starts, const int32_t* lens, const int32_t* table,
                                     const int32_t* seen, int64_t words, int dtype, const fab_paged_dims* dims,
                                     void* q_out, void* k_cache, void* v_cache, fab_stream stream);

/* fab_paged_attention of a draft, causal: token i sees the keys before the
 * sequence's new tokens, and of those the j <= i whose bits are set.  A token
 * without a key gets o = 0 and lse = +inf.  Rows before lens[b] have to be finite,
 * those of branches that a token does not see too.  Types, widths, roundings and the
 * workspace (fab_paged_attention_workspace_bytes) are fab_paged_attention's. */
FAB_EXPORT int fab_paged_attention_tree(const void* q, const void* k_cache, const void* v_cache, const int32_t* starts,
                                        const int32_t* lens, const int32_t* table, const int32_t* seen, int64_t words,
                                        float scale, int dtype, const fab_paged_dims* dims, void* workspace,
                                        size_t workspace_bytes, void* o, float* lse, fab_stream stream);

/* ---- Rows and pages of a cache, in all layers at once ---- */

/* A cache of `layers` layers that share one table: layer l's keys are the cache
 * [DK, page, Hkv, pages] from element l*ldk on, its values from l*ldv on (ldk, ldv
 * at least a layer's elements; not read for one layer).  B * max_pages is at
 * most 2^30, layers * Hkv at most 2^24. */
typedef struct {
  int64_t B;             /* sequences (rows of the table) */
  int64_t T, words;      /* new tokens, words of a row of `seen` (fab_paged_accept only) */
  int64_t Hkv, DK, DV;   /* key/value heads, key width, value width (<= 256) */
  int64_t page;          /* rows of a page */
  int64_t pages;         /* pages of the cache */
  int64_t max_pages;     /* entries of a sequence's row of the table */
  int64_t layers;
  int64_t ldk, ldv;
} fab_cache_dims;

/* Keeps one path of each draft: last[b] is the number (among the new tokens of
 * sequence b) of the last token accepted, -1 for none.  The tokens that it sees up to
 * itself become the sequence's next ones: their rows move, in order, to the places
 * from lens[b] - n on, in every layer, and lens_out[b] = lens[b] - n + how many they
 * are (lens[b] for a sequence without new tokens, whose last[b] is not read).  What the rows behind
 * them hold afterwards is not defined; no other row is written.  starts,
 * lens (counting the draft), table, seen, last: device int32 as the calls before
 * had them; lens_out: device int32 [B], not overlapping them.  No two sequences may
 * share a page that holds new tokens.  A last[b] outside -1 .. n-1, or lens, starts
 * and pages out of range, are reported as FAB_ERR_INVALID, and touch nothing outside
 * the arguments. */
FAB_EXPORT int fab_paged_accept(const int32_t* starts, const int32_t* lens, const int32_t* table, const int32_t* seen,
                                const int32_t* last, int dtype, const fab_cache_dims* dims, void* k_cache,
                                void* v_cache, int32_t* lens_out, fab_stream stream);

/* Device workspace bytes of fab_paged_reserve; 0 for bad dims. */
FAB_EXPORT size_t fab_paged_reserve_workspace_bytes(const fab_cache_dims* dims);

/* Hands out the pages of a cache.  table [max_pages,B]: entries that hold no page
 * are -1.  refs [pages] (16-byte aligned): how many entries of the table name each
 * page, 0: it is free.  Both are read and brought up to date.  Row b afterwards
 * has room for lens[b] tokens and holds the first kept[b] (lens[b] where that is
 * less) of the row source[b] as it was before the call (source NULL: of itself;
 * source[b] = -1: of none):
 *   - the entries of those tokens' pages are carried over, and shared where
 *     several rows continue one (a fork);
 *   - where lens[b] > kept[b] and the last of those pages is partly filled, it will be
 *     written, and may then belong to no other row: the lowest such row keeps it if
 *     all rows that hold it would write it, every other gets a fresh page with
 *     its kept[b] % page rows copied, in every layer;
 *   - further entries up to lens[b] are fresh pages, those behind are -1, and pages
 *     that no entry names any more are free (lens[b] = 0 frees a row).
 * Fresh pages are the free ones, lowest first, in order of row and entry, those
 * that this call frees among them.  spare [1], no part of the other arrays, gets the
 * number of pages left free, below zero the number that were missing: the last
 * entries in that order are then -1, and what a copy among them should have held is
 * lost.
 * source, kept, lens: device int32 [B].  kept[b] past what the row source[b] holds,
 * or any of them out of range, are reported as FAB_ERR_INVALID (the rows concerned are
 * meaningless; nothing outside the arguments is touched).  So are references too low
 * for the table, by the call in which that matters: where a page that a row holds on to
 * would be handed out or written by another, or a count falls below zero.  References
 * above what the table says stand for holders besides it: for as long as they are there
 * the page is not written, handed out or freed.  fab_cache_dims' T and words are not read.
 * workspace: device, fab_paged_reserve_workspace_bytes() bytes, contents overwritten;
 * calls that may overlap on the GPU need one each. */
FAB_EXPORT int fab_paged_reserve(int32_t* table, int32_t* refs, const int32_t* source, const int32_t* kept,
                                 const int32_t* lens, int dtype, const fab_cache_dims* dims, void* k_cache,
                                 void* v_cache, void* workspace, size_t workspace_bytes, int32_t* spare,
                                 fab_stream stream);

/* Synchronises `stream`, then returns and clears the device-side error word
 * of the current device: FAB_OK, FAB_ERR_TIMEOUT (a bounded wait inside a
 * kernel ran out; that kernel's outputs are invalid), FAB_ERR_INVALID (a
 * position, page number, start or other index that a kernel read from device
 * memory was out of range) or FAB_ERR_CUDA. */
FAB_EXPORT int fab_last_device_error(fab_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FAB_H */
