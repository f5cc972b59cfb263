/*
 * rope.h -- C ABI of the MI355X (gfx950) RoPE apply library, librope_amd.so.
 *
 * Each operation is one call that validates its arguments on the host and then enqueues
 * hand-written HIP kernels on the caller's stream:
 *
 *   rope_partial_inplace           in-place partial RoPE (interleave or half mode) on a BSND tensor
 *   rope_partial_inplace_backward  its gradient with respect to x, in place on the gradient
 *   rope_with_cos_sin_cache        RoPE of query/key rows with cos/sin gathered from a cache by
 *                                  position; rope or mrope mode; GPT-NeoX or GPT-J style
 *   rope_with_cos_sin_cache_v2     the same with the cacheMode argument (sectioned or
 *                                  interleaved mrope stitching)
 *   rope_append_paged_cache        rotates a batch's new keys (and queries) by position and
 *                                  appends keys and values to a paged cache
 *   rope_latent_attention_paged    attention of those queries over the paged cache where keys and
 *                                  values come from one latent row a token (absorbed form)
 *   rope_latent_attention          the expanded form, for prompts and training: a key and value
 *                                  of every head and one rotated key part shared by the heads
 *   rope_latent_attention_backward
 *                                  its gradients
 *   rope_append_paged_cache_q8     rotates a batch's new keys (and queries) by position and writes
 *                                  keys and values to a paged cache of 8-bit codes with a scale
 *                                  for each block of tokens and head
 *   rope_attention_paged_q8        grouped-query attention over that cache
 *   rope_copy_pages                copies listed pages of any number of caches
 *   rope_fork_pages                the page tables, holds and copies of a batch whose sequences
 *                                  continue those of another (beams, samples, sequences that end)
 *   rope_compact_pages             moves the pages in use to the lowest numbers
 *
 * Pages defining the operations:
 *   [IPRM] "CANN ops-transformer 的 aclnnInplacePartialRotaryMul 算子：Inplace 部分旋转位置编码
 *           接口详解与实现剖析"
 *   [RSCC] "CANN ops-transformer 旋转位置编码算子 RopeWithSinCosCache 深度解析：cache 化 RoPE 的
 *           计算原理与 aclnn 两段式调用实战"
 * Both pages describe a two-phase interface (workspace size, then execute).  Their kernels
 * need no workspace here, so the two phases are one call.  Where the attention calls need one,
 * a function beside them gives its size and the caller passes it.
 *
 * Common rules
 *  - Memory: every tensor `data` pointer is device memory (or memory the GPU can address)
 *    owned by the caller.  The library never allocates, frees, retains a pointer after the
 *    call returns, or synchronizes.  Host arrays (partial_slice, mrope_section) are read
 *    during the call only.
 *  - Stream: `stream` is a hipStream_t (NULL = the null stream of the current device).  The
 *    kernels run on the current HIP device: the stream and every tensor must belong to it
 *    (hipSetDevice first when several GPUs are in use).  The
 *    call returns once the work is enqueued; results are visible after the stream is
 *    synchronized.  The library is stateless and reentrant; calls that touch the same
 *    buffers must be ordered by the caller (same stream or events).
 *  - Arithmetic (of the rotations; the attention calls state theirs): operands are raised to float32, each product and each sum of the formulas
 *    is one float32 operation (no fused multiply-add), and the result is rounded once to
 *    the tensor dtype (round to nearest even).  Data outside the rotated range is never
 *    converted: it is left untouched (in-place op) or copied bit for bit (cache op).
 *  - Errors: a non-zero status means nothing was enqueued and no buffer was touched
 *    (except ROPE_ERR_RUNTIME, which reports a failed launch).  rope_last_error() gives a
 *    text for the last failing call of the calling thread.
 *  - Determinism: every output element is written by exactly one GPU lane with no atomics,
 *    so repeated calls give bit-identical results ([IPRM §约束说明], [RSCC §约束说明]).  (The counts of
 *    rope_fork_pages are sums of integers, which no order changes.)
 */
#ifndef ROPE_AMD_H
#define ROPE_AMD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a tensor description. */
typedef enum {
  ROPE_F32 = 0,  /* IEEE binary32 */
  ROPE_F16 = 1,  /* IEEE binary16 */
  ROPE_BF16 = 2, /* bfloat16 */
  ROPE_I64 = 3,  /* int64 (positions) */
  ROPE_I8 = 4,   /* int8 codes of a cache in 8 bits */
  ROPE_E4M3 = 5  /* 8-bit floating point codes, 4 exponent and 3 mantissa bits, no infinities */
} rope_dtype;

/* Status codes.  The two parameter codes are the ones of [IPRM §返回值与错误码];
 * ROPE_ERR_RUNTIME has no value on the pages (library-defined). */
enum {
  ROPE_OK = 0,
  ROPE_ERR_PARAM_NULLPTR = 161001, /* a required tensor (or its data) is NULL          */
  ROPE_ERR_PARAM_INVALID = 161002, /* dtype / shape / attribute / layout not supported */
  ROPE_ERR_RUNTIME = 361001        /* the HIP launch failed                           */
};

/* A strided tensor view.  shape[] and stride[] hold `ndim` entries (1..4); strides are in
 * elements.  `data` may be NULL only when the tensor has no elements.  Every entry point
 * refuses (ROPE_ERR_PARAM_INVALID) a view with more than 2^53 elements or whose furthest
 * element lies 2^53 or more elements from its first: no buffer is that large. */
typedef struct {
  void *data;
  rope_dtype dtype;
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} rope_tensor;

/*
 * rope_partial_inplace -- in-place partial RoPE.
 *
 * Defined in [IPRM §计算原理与公式] and [IPRM §partial_slice 局部旋转机制]: on the slice
 * x[..., start:end) of the last dim (indices below count from `start`), x = x*cos +
 * x_rotate*sin.  Interleave mode (rotary_mode 1): x_rotate = (-x2, x1) interleaved per pair,
 * so each pair (x[2i], x[2i+1]) becomes
 *     x[2i]   = x[2i]*cos[2i]     - x[2i+1]*sin[2i]
 *     x[2i+1] = x[2i+1]*cos[2i+1] + x[2i]*sin[2i+1]
 * Half mode (rotary_mode 0; [IPRM §参数说明] lists it as not yet enabled on its hardware,
 * enabled here): x1, x2 are the two halves of the slice, x_rotate = cat(-x2, x1), so with
 * h = L/2 each pair (x[i], x[i+h]) becomes
 *     x[i]   = x[i]*cos[i]     - x[i+h]*sin[i]
 *     x[i+h] = x[i+h]*cos[i+h] + x[i]*sin[i+h]
 * Elements in [0, start) and [end, D) are never read or written.
 *
 * x      [B, S, N, D] (BSND), contiguous, F32 / F16 / BF16; read and written in place.
 * cos,   [Bc, Sc, Nc, L] with L = end - start, contiguous, both of one dtype: x's dtype or
 * sin    F32 (F32 with half-precision x is the mixed case of [IPRM §返回值与错误码]).
 *        Each of Bc, Sc, Nc is 1 (broadcast) or equal to x's B, S, N; this covers the BSND,
 *        BS1D, B1ND, B11D and 111D layouts of [IPRM §约束说明].
 * rotary_mode    1 (interleave) or 0 (half); any other value is ROPE_ERR_PARAM_INVALID.
 * partial_slice  host array {start, end}; NULL with partial_slice_len 0 means [0, D).
 *                0 <= start <= end <= D and end - start even; start == end returns
 *                ROPE_OK at once without launching anything (and without checking cos/sin's
 *                last dim).  start may be odd.
 * Constraints (else ROPE_ERR_PARAM_INVALID): 4-D tensors, D even and D <= 1024, cos and
 * sin of one shape whose last dim is L, contiguous tensors, and x sharing no memory with
 * cos or sin (cos and sin may be one tensor).  NULL x/cos/sin, or NULL data
 * of a non-empty tensor, gives ROPE_ERR_PARAM_NULLPTR.  An x with no elements is a no-op.
 */
int rope_partial_inplace(const rope_tensor *x, const rope_tensor *cos, const rope_tensor *sin,
                         int64_t rotary_mode, const int64_t *partial_slice,
                         int64_t partial_slice_len, void *stream);

/*
 * rope_partial_inplace_backward -- gradient of rope_partial_inplace with respect to x, in place
 * on the incoming gradient g.
 *
 * [IPRM §Python 接口与自动微分]: the training path computes the gradient of x with a backward
 * op; cos and sin get no gradient; empty tensors and empty slices are no-ops.  The pages give
 * no formula: on each slice pair (j, k) -- (2i, 2i+1) in interleave mode, (i, i+L/2) in half
 * mode -- the forward map is y = [[c_j, -s_j], [s_k, c_k]] x, so its gradient is the transpose,
 *     g[j] = g[j]*cos[j] + g[k]*sin[k]
 *     g[k] = g[k]*cos[k] - g[j]*sin[j]
 * and elements outside [start, end) pass the gradient through unchanged (never touched).
 * Arguments, layouts, validation, error codes and the no-op rules are those of
 * rope_partial_inplace, with g in the place of x.
 */
int rope_partial_inplace_backward(const rope_tensor *g, const rope_tensor *cos,
                                  const rope_tensor *sin, int64_t rotary_mode,
                                  const int64_t *partial_slice, int64_t partial_slice_len,
                                  void *stream);

/*
 * rope_with_cos_sin_cache -- RoPE with a cos/sin cache ([RSCC §设计动机]).
 *
 * For each token t: cos/sin are gathered from cos_sin_cache[position] and split in halves
 * (first rotaryDim/2 columns cos, last rotaryDim/2 sin).  Every head of query, then of key,
 * has its first rotaryDim elements rotated and the remaining headSize - rotaryDim copied:
 *   GPT-NeoX (is_neox_style != 0, [RSCC §rotate_half（GPT-NeoX style）旋转模式]):
 *       x1 = x[0 : rd/2], x2 = x[rd/2 : rd]
 *   GPT-J    (is_neox_style == 0, [RSCC §rotate_interleaved（GPT-J style）旋转模式]):
 *       x1 = x[0 : rd : 2], x2 = x[1 : rd : 2], outputs interleaved back
 *   o1 = x1*cos - x2*sin,  o2 = x2*cos + x1*sin.
 *
 * positions      INT64. rope mode: [T]. mrope mode: [m, T] with m = mrope_section_len.
 *                Any non-negative strides.  Every value must lie in [0, maxSeqLen) -- a
 *                precondition ([RSCC §约束说明]) that is not checked (that would need a device
 *                synchronization); a value outside it is clamped into range on the device, so
 *                the call never reads outside the cache but its output is then meaningless.
 * query_in       [T, Nq*headSize], key_in [T, Nk*headSize]: F32 / F16 / BF16, unit inner
 *                stride, any non-negative row stride (the qStride/kStride of the pages).
 * cos_sin_cache  [maxSeqLen, rotaryDim], same dtype, unit inner stride, any row stride.
 * mrope_section  host array or NULL.  NULL (length 0) -> rope mode.  Otherwise 3 or 4
 *                non-negative entries; entry 0 > 0 selects mrope ([RSCC §rope 模式：标准位置编码]),
 *                where 2*sum == rotaryDim and the list is one of {16,24,24}, {8,12,12},
 *                {24,20,20}, {11,11,10}, {16,16,16,16} ([RSCC §入参校验逻辑]).  Element i of
 *                cos/sin then comes from the position row k whose section holds i
 *                ([RSCC §mrope 模式：多模态位置编码]).  Entry 0 == 0 -> rope mode.
 * head_size      headSize; a positive multiple of 64 bytes (32 elements for F16/BF16, 16 for
 *                F32); rotaryDim (= cache width) is a multiple of 64 bytes too and
 *                <= headSize ([RSCC §约束说明]).
 * query_out,     contiguous, same shapes and dtype as the inputs.  An output may be its own
 * key_out        input exactly (same pointer and layout); any other overlap between an
 *                output and another tensor is rejected.
 * Errors: NULL tensors -> ROPE_ERR_PARAM_NULLPTR; wrong dtype, rank, empty inputs, token
 * count mismatch, output shape mismatch, bad mropeSection or alignment -> ROPE_ERR_PARAM_INVALID.
 */
int rope_with_cos_sin_cache(const rope_tensor *positions, const rope_tensor *query_in,
                            const rope_tensor *key_in, const rope_tensor *cos_sin_cache,
                            const int64_t *mrope_section, int64_t mrope_section_len,
                            int64_t head_size, int is_neox_style,
                            const rope_tensor *query_out, const rope_tensor *key_out,
                            void *stream);

/*
 * rope_with_cos_sin_cache_v2 -- rope_with_cos_sin_cache with the cacheMode argument
 * ([RSCC §V2 接口：cacheMode 扩展]), which picks how mrope stitches cos/sin from the position
 * rows:
 *   cache_mode 0  sectioned: element i comes from the row whose section holds i (exactly
 *                 rope_with_cos_sin_cache, which is this call with cache_mode 0);
 *   cache_mode 1  interleaved, 3-section lists only: every element starts from row 0; then
 *                 the elements i < 3*mropeSection[1] with i % 3 == 1 come from row 1 and
 *                 those with i % 3 == 2 from row 2 (index i in [0, rotaryDim/2), the same
 *                 for the cos and the sin half).
 * cache_mode must be 0 or 1, and 0 with the list {16,16,16,16}; anything else gives
 * ROPE_ERR_PARAM_INVALID (checked in rope mode too, where the value changes nothing).
 * Every other argument, layout and rule is that of rope_with_cos_sin_cache.
 */
int rope_with_cos_sin_cache_v2(const rope_tensor *positions, const rope_tensor *query_in,
                               const rope_tensor *key_in, const rope_tensor *cos_sin_cache,
                               const int64_t *mrope_section, int64_t mrope_section_len,
                               int64_t head_size, int is_neox_style, int64_t cache_mode,
                               const rope_tensor *query_out, const rope_tensor *key_out,
                               void *stream);

/*
 * rope_append_paged_cache -- rotate by position, append to a paged cache.
 *
 * For token t with cos_sin_cache row [c | s] of positions[t] (split in halves as in
 * rope_with_cos_sin_cache), every key head, and every query head if there is a query, has its
 * elements [rot_start, rot_start + rotaryDim) rotated, rotaryDim = cache width:
 *       o1 = x1*c - x2*s,  o2 = x2*c + x1*s
 * with pairs (i, i + rotaryDim/2) of the slice for is_neox_style != 0 and (2i, 2i+1) otherwise;
 * the rest of a head, and the value, are copied bit for bit.  Keys and values are written to
 * row slots[t] % pageSize of page slots[t] / pageSize.
 *
 * positions      INT64 [T], any non-negative stride; out-of-range values are clamped as in
 *                rope_with_cos_sin_cache.
 * slots          INT64 [T], any non-negative stride.  A slot below 0 or beyond the last page's
 *                last row is skipped (padding tokens; their queries are still rotated).  The
 *                slots in range must be distinct -- a precondition that is not checked: a slot
 *                given twice ends up with elements of either token.
 * query          [T, Nq, Dq] or NULL, with query_out [T, Nq, Dq] (NULL exactly if query is).
 * key            [T, Nk, D]; value [T, Nk, Dv] or NULL, with its cache NULL exactly if it is.
 * cos_sin_cache  [maxSeqLen, rotaryDim], rotaryDim even and positive.
 * key_cache      [pages, pageSize, Nk, D], value_cache [pages, pageSize, Nk, Dv].
 * All floating-point tensors share one dtype, F32, F16 or BF16.  Every one may have any
 * non-negative strides with unit inner stride (columns of one projection's output, caches that
 * keep heads before rows, or keys and values in one allocation); 16-byte aligned rows, slices and
 * widths take wide accesses.  query_out may be the query itself (same view).  Outputs whose
 * strides reach an element twice, and any other overlap with an output, are refused
 * (ROPE_ERR_PARAM_INVALID).  T = 0 is a no-op.
 */
int rope_append_paged_cache(const rope_tensor *positions, const rope_tensor *slots,
                            const rope_tensor *query, const rope_tensor *key,
                            const rope_tensor *value, const rope_tensor *cos_sin_cache,
                            int64_t query_rot_start, int64_t key_rot_start, int is_neox_style,
                            const rope_tensor *query_out, const rope_tensor *key_cache,
                            const rope_tensor *value_cache, void *stream);

/*
 * rope_latent_attention_paged -- attention over a paged cache of latent rows, absorbed form.
 *
 * A cached token j of a sequence is one row c_j of latent_dim + 64 elements: a latent part and a
 * rotated tail.  The row is the key, its latent part the value, of every head.  Query token i
 * (of n, in a sequence of len cached tokens, its own n among them) sees rows j < len - n + 1 + i:
 *       s_j = scale * <query[i, h], c_j>,   p = softmax_j(s),   out[i, h] = sum_j p_j c_j[0 : latent_dim]
 *       lse[i, h] = log sum_j exp(s_j)
 * Products accumulate in float32; maxima, sums and outputs are float32 until one rounding to the
 * output's dtype; the weights p are rounded to the dtype for the second product.  A query that
 * sees no row gets zeros and lse = -infinity.  Rows past len may hold anything: they reach no
 * result.  A row that a sequence's last query sees and an earlier one does not has weight 0 for
 * the earlier one, so a NaN or infinity in it makes that query's output NaN too.
 *
 * query          [T, heads, latent_dim + 64], F16 or BF16, unit inner stride, rows on 16-byte
 *                boundaries, any non-negative strides.
 * latent_cache   [pages, pageSize, latent_dim + 64], same dtype, same rule for rows; any pageSize.
 * page_table     INT64 [B, maxPages]: pages of each sequence, in order, any non-negative strides.
 *                Entries in use must lie in [0, pages): not checked; others are clamped, so
 *                that nothing outside the cache is read, and give meaningless results.
 * seq_lens       INT64 [B]: cached tokens, clamped to [0, maxPages * pageSize].
 * query_offsets  INT64 [B + 1], ascending: sequence b's queries are rows offsets[b] to
 *                offsets[b+1] of query and out; rows outside all of them are left as they are.
 *                Out-of-range values are clamped; where they descend, the call writes no result.
 *                NULL: T / B queries each (T % B == 0).
 * latent_dim     128, 256 or 512.     scale   finite, |scale| < 2^127.
 * out            [T, heads, latent_dim] contiguous, 16-byte aligned; lse F32 [T, heads]
 *                contiguous, or NULL.  Outputs may not overlap anything else.
 * workspace      device memory of at least rope_latent_attention_paged_workspace() bytes, 16-byte
 *                aligned, free for this call from its enqueueing to its end: calls that may run
 *                at the same time need one each.  Its contents need not be initialised.
 * Results do not depend on timing: every sum is taken in a fixed order.
 */
int64_t rope_latent_attention_paged_workspace(int64_t num_tokens, int64_t num_heads,
                                              int64_t latent_dim, int64_t num_sequences);
int rope_latent_attention_paged(const rope_tensor *query, const rope_tensor *latent_cache,
                                const rope_tensor *page_table, const rope_tensor *seq_lens,
                                const rope_tensor *query_offsets, int64_t latent_dim,
                                double scale, const rope_tensor *out, const rope_tensor *lse,
                                void *workspace, int64_t workspace_bytes, void *stream);

/*
 * rope_latent_attention -- latent attention, expanded form.
 *
 * Head h of query token i (of n, in a sequence with m key tokens) attends to its sequence's keys:
 *       s_ij = scale * (<query[i, h, 0 : dim], key[j, h]> + <query[i, h, dim : dim + 64], key_rope[j]>)
 *       p = softmax_j(s),  out[i, h] = sum_j p_ij value[j, h],  lse[i, h] = log sum_j exp(s_ij)
 * With causal != 0 query i sees keys j < m - n + 1 + i (the last query sees them all), else all.
 * Precision as in rope_latent_attention_paged.  A query that sees no key gets zeros and
 * lse = -infinity.  A NaN or infinity in a token reaches results of its own sequence only, there
 * also those of queries that do not see the token.
 *
 * query      [Tq, heads, dim + 64], key [Tk, heads, dim], key_rope [Tk, 64], value
 *            [Tk, heads, dim]: F16 or BF16, one dtype, dim 64 or 128, unit inner stride, rows on
 *            16-byte boundaries, any other non-negative strides (key and value may be the two
 *            parts of one projection's rows), a token's below 32 MiB.
 * query_offsets, key_offsets   INT64 [B + 1] each, ascending: sequence b is query rows
 *            query_offsets[b] to [b+1] and key rows key_offsets[b] to [b+1]; rows outside are
 *            left as they are; out-of-range values are clamped.  Where they descend, the call's results
 *            are not defined (sequences may then share rows, which are written in no fixed order),
 *            but no access leaves the tensors, and rows outside the first and the largest offset
 *            are left as they are.  Both NULL: num_sequences sequences of Tq / B and Tk / B tokens.
 * num_sequences   B; may be 0 when there are offsets.
 * out        [Tq, heads, dim] contiguous, 16-byte aligned; lse F32 [Tq, heads] contiguous.
 * A call whose kernels would need 2^32 threads is refused: with t = Tq / 128 + B tiles (B times the
 * tiles of a sequence without offsets), heads * t * 256 has to stay below; of the backward call also
 * heads * t * 512 with Tk in the place of Tq, and (Tq + Tk) * 16.
 */
int rope_latent_attention(const rope_tensor *query, const rope_tensor *key,
                          const rope_tensor *key_rope, const rope_tensor *value,
                          const rope_tensor *query_offsets, const rope_tensor *key_offsets,
                          int64_t num_sequences, double scale, int causal, const rope_tensor *out,
                          const rope_tensor *lse, void *stream);

/*
 * rope_latent_attention_backward -- gradients of rope_latent_attention with respect to query, key,
 * key_rope (summed over the heads) and value, for the gradient `grad` [Tq, heads, dim] of out.
 * out and lse are the forward call's; of out only the description is used (<grad, out> would carry
 * its rounding into the gradients, so it is computed again, in float32).  Gradients are contiguous,
 * 16-byte aligned, of their input's shape and dtype, each summed in float32 in a fixed order and
 * rounded once (the probabilities and their gradients are rounded to the dtype between the products,
 * in F16 after an exact scaling that keeps them in its range, whatever the size of grad).  The
 * probabilities are taken again from lse, so their relative error grows with it, by some
 * 2^-22 |lse|: below a bfloat16 step for |lse| up to 10^4.  Rows outside all sequences get zero
 * gradients.  workspace: at least rope_latent_attention_backward_workspace() bytes, under the rules
 * of rope_latent_attention_paged's.
 */
int64_t rope_latent_attention_backward_workspace(int64_t query_tokens, int64_t key_tokens,
                                                 int64_t num_heads);
int rope_latent_attention_backward(
    const rope_tensor *grad, const rope_tensor *query, const rope_tensor *key,
    const rope_tensor *key_rope, const rope_tensor *value, const rope_tensor *out,
    const rope_tensor *lse, const rope_tensor *query_offsets, const rope_tensor *key_offsets,
    int64_t num_sequences, double scale, int causal, const rope_tensor *dquery,
    const rope_tensor *dkey, const rope_tensor *dkey_rope, const rope_tensor *dvalue,
    void *workspace, int64_t workspace_bytes, void *stream);

/*
 * rope_append_paged_cache_q8 -- rotate by position, append to a paged cache in 8 bits.
 *
 * A cached key (or value) element is code * scale: the codes lie in a cache [pages, pageSize, Nk, D]
 * of I8 or E4M3, and every block of pageSize / blocks tokens of a page and every head has one
 * float32 scale in [pages, blocks, Nk].  Sequence b's new tokens are rows token_offsets[b] to
 * token_offsets[b+1] of key, value and query; they are the last ones of its seq_lens[b] tokens, so
 * the i-th of n goes to place p = seq_lens[b] - n + i: row p % pageSize of page
 * page_table[b, p / pageSize].  Rotation is that of rope_append_paged_cache, in float32, and keys are
 * coded from its unrounded results.
 *
 * For each block and head that takes new tokens, with top = the largest |x| of the new elements:
 *       need = max(top / 127, 2^-120)                                      I8
 *       need = the smallest power of two >= max(top / 448, 2^-120)         E4M3
 *       scale = need, or the larger of need and the present scale where the block holds earlier
 *               tokens of the sequence; their codes are then round(code * (old scale / scale))
 *       code = round(x * (1 / scale))       (to nearest even; every step is one float32 operation,
 *                                            top / 127 a product with the float32 nearest 1/127)
 * Powers of two keep E4M3 codes exact when a scale grows, down to the type's subnormal numbers;
 * I8 codes of the block's earlier tokens lose up to half a step each time.  Scales outlive tokens
 * that are taken back (a smaller seq_lens): only a block's first token starts a scale anew.
 * Non-finite elements: E4M3 codes them as NaN and leaves them out of top; I8, which has no NaN, sets
 * the scale of the block and head to NaN, and so all its tokens.  Rows behind the last token are
 * left as they are.
 *
 * positions      INT64 [T], as in rope_append_paged_cache.
 * query          [T, Nq, Dq] or NULL, with query_out [T, Nq, Dq] (NULL exactly if query is; it may
 *                be the query itself).  All tokens' queries are rotated.
 * key            [T, Nk, D]; value [T, Nk, Dv]; cos_sin_cache [maxSeqLen, rotaryDim].  One dtype,
 *                F32, F16 or BF16.  Dv may be 0 (a cache of keys alone): value_scales then get the
 *                scales of top = 0.
 * key_cache, value_cache    [pages, pageSize, Nk, D] and [.., Dv], I8 or E4M3, one of the two.
 * key_scales, value_scales  F32 [pages, blocks, Nk]; blocks divides pageSize.  A block has fewer than
 *                2^30 elements of a head.
 * page_table     INT64 [B, maxPages]; seq_lens INT64 [B], clamped to [0, maxPages * pageSize].
 *                Tokens before place 0, and tokens whose page is not in [0, pages) (padding), are
 *                skipped.  A page that takes tokens belongs to one sequence only -- a precondition
 *                that is not checked (rope_fork_pages keeps it).
 * token_offsets  INT64 [B + 1], ascending; out-of-range values are clamped to [0, T], and rows outside
 *                all sequences are not appended.  Where they descend, what is appended is not defined,
 *                but no access leaves the tensors.  NULL: T / B tokens each (T % B == 0).
 * Any non-negative strides with unit inner stride (scales: any non-negative strides).  Outputs whose
 * strides reach an element twice, and any other overlap with an output, are refused.  T = 0 is a no-op.
 */
int rope_append_paged_cache_q8(const rope_tensor *positions, const rope_tensor *query,
                               const rope_tensor *key, const rope_tensor *value,
                               const rope_tensor *cos_sin_cache, const rope_tensor *page_table,
                               const rope_tensor *seq_lens, const rope_tensor *token_offsets,
                               int64_t query_rot_start, int64_t key_rot_start, int is_neox_style,
                               const rope_tensor *query_out, const rope_tensor *key_cache,
                               const rope_tensor *value_cache, const rope_tensor *key_scales,
                               const rope_tensor *value_scales, void *stream);

/*
 * rope_attention_paged_q8 -- grouped-query attention over a paged cache in 8 bits.
 *
 * Head h of query token i (of n, in a sequence of len cached tokens, its own n among them) attends to
 * the tokens j < len - n + 1 + i of key head h / (heads / Nk):
 *       s_j = scale * key_scale_j * <query[i, h], key_code_j>,   p = softmax_j(s)
 *       out[i, h] = sum_j p_j value_scale_j value_code_j,        lse[i, h] = log sum_j exp(s_j)
 * Codes are exact in the query's dtype; products accumulate in float32; maxima, sums and outputs are
 * float32 until one rounding to the output's dtype; the weights p_j value_scale_j are rounded to the
 * dtype for the second product.  (F16: relative to the largest value scale that the query sees, so that
 * none leaves its range; a weight is off by half a step of its own, or 2^-35 of that scale.)  A query
 * that sees no token gets zeros and lse = -infinity.  Tokens that a query does not see reach nothing of
 * its results, whatever their codes and scales: rows past len, and the tokens of later queries.
 *
 * query          [T, heads, D], F16 or BF16, D 64, 128 or 256, heads a multiple of Nk, unit inner
 *                stride, rows on 16-byte boundaries, any non-negative strides.
 * key_cache, value_cache    [pages, pageSize, Nk, D], I8 or E4M3, one of the two; unit inner stride,
 *                rows on 16-byte boundaries, a token's stride below 2^24; any pageSize.
 * key_scales, value_scales  F32 [pages, blocks, Nk], any non-negative strides; blocks divides pageSize.
 * page_table, seq_lens, query_offsets, out [T, heads, D], lse, scale and workspace: as in
 *                rope_latent_attention_paged (pages out of range are clamped), the workspace of at
 *                least rope_attention_paged_q8_workspace() bytes.
 * Results do not depend on timing: every sum is taken in a fixed order.  Tiles are sized by the mean
 * number of queries of a call: sequences that decode and long pieces of prompts are faster in two calls.
 */
int64_t rope_attention_paged_q8_workspace(int64_t num_tokens, int64_t num_heads,
                                          int64_t num_key_heads, int64_t head_size,
                                          int64_t num_sequences);
int rope_attention_paged_q8(const rope_tensor *query, const rope_tensor *key_cache,
                            const rope_tensor *value_cache, const rope_tensor *key_scales,
                            const rope_tensor *value_scales, const rope_tensor *page_table,
                            const rope_tensor *seq_lens, const rope_tensor *query_offsets,
                            double scale, const rope_tensor *out, const rope_tensor *lse,
                            void *workspace, int64_t workspace_bytes, void *stream);

/*
 * rope_copy_pages -- page targets[i] of every cache becomes a copy of its page sources[i].
 *
 * caches         num_caches descriptions [pages, ...] of 1 to 4 dims and any of the dtypes, all of the
 *                same number of pages: the keys, values and scales of all layers.  A page has to be
 *                one dense block of memory, its dimensions in any order, pages any stride apart.
 * sources, targets   INT64 [N], any non-negative stride.  A pair with a number outside [0, pages) is
 *                skipped (padding).  Targets in range have to be distinct, and no target the source
 *                of another pair -- preconditions that are not checked: such pages end up with parts
 *                of either.
 */
int rope_copy_pages(const rope_tensor *sources, const rope_tensor *targets,
                    const rope_tensor *caches, int64_t num_caches, void *stream);

/*
 * rope_fork_pages -- the next step's sequences continue this step's.
 *
 * New row i continues sequence p = parents[i] with all its seq_lens[p] tokens, and is to take grow[i]
 * tokens more.  Sequences that no row continues end.  ref_counts[page] is the number of holds on a
 * page: the rows of page_table that list it, and any others (a cache of shared beginnings may hold
 * pages too); pages without holds are free.
 *   - Full pages are shared.  A last page that is not full goes to the first row that continues its
 *     sequence if it has no other hold (ref_counts 1 or less); every other such row gets a copy of
 *     its tokens in a new page, in all caches.
 *   - New pages are taken for grow[i] tokens.
 *   - New pages are the lowest numbers with ref_counts 0, dealt to the rows in order, to a row its
 *     copied page first.  Pages that this call frees are free for the next one.
 *   - page_table_out[i] lists the row's pages, then -1; seq_lens_out[i] = seq_lens[p] + grow[i];
 *     ref_counts_out are the holds afterwards.  All of a row's tokens have to fit page_table_out:
 *     grow is cut there.
 *   - shortage[0] is the number of pages that were wanted and not there; -1 stands for them in
 *     page_table_out, and where it is not 0, rows with such an entry cannot go on.
 * The sequences of one batch may be freed, forked, reordered and extended by one call, without the
 * host's knowing their lengths.
 *
 * page_table     INT64 [B, maxPages]; seq_lens INT64 [B], clamped to [0, maxPages * pageSize].
 *                Entries in use outside [0, pages) stay and count nowhere.
 * parents        INT64 [R]; outside [0, B): an empty row of length 0, which gets no pages (a sequence that
 *                begins continues one of length 0).     grow  INT64 [R] or NULL (0); below 0: 0.
 * ref_counts     INT64 [pages];  page_size: tokens of a page.
 * caches         as in rope_copy_pages, num_caches may be 0.  Of two forms a copied page gets only the
 *                part that holds the row's tokens, where the second dimension is the outermost of a page:
 *                [pages, page_size, ...] of 3 or 4 dims, whose second dimension is taken for the page's
 *                tokens, and F32 [pages, n, m], n a divisor of page_size, taken for the scales of n blocks
 *                of tokens (rope_append_paged_cache_q8's).  All others are copied whole, [pages, heads,
 *                pageSize, ...] and [pages, 2, ...] among them.  A cache that has one of the two forms and is
 *                something else (as many heads as a page has tokens, outermost; F32 scales of a page's n
 *                heads) is to be described as [pages, elements]: with 2 dims it is copied whole.
 * page_table_out INT64 [R, maxPages or more], seq_lens_out INT64 [R], shortage INT64 [1]: apart from
 *                all inputs.
 * ref_counts_out INT64 [pages], may be ref_counts itself.
 * workspace      at least rope_fork_pages_workspace() bytes, under the rules of
 *                rope_latent_attention_paged's.
 */
int64_t rope_fork_pages_workspace(int64_t num_sequences, int64_t num_rows, int64_t num_pages);
int rope_fork_pages(const rope_tensor *page_table, const rope_tensor *seq_lens,
                    const rope_tensor *parents, const rope_tensor *grow,
                    const rope_tensor *ref_counts, int64_t page_size, const rope_tensor *caches,
                    int64_t num_caches, const rope_tensor *page_table_out,
                    const rope_tensor *seq_lens_out, const rope_tensor *ref_counts_out,
                    const rope_tensor *shortage, void *workspace, int64_t workspace_bytes,
                    void *stream);

/*
 * rope_compact_pages -- the pages in use (ref_counts above 0) become pages 0 to live - 1.
 *
 * The k-th page in use from number `live` on moves, in all caches, to the k-th free page below it.
 * page_map[page] is the new number of a page in use and -1 of a free one; page_table_out[b, j] is
 * page_map of the entry (entries outside [0, pages) stay); ref_counts_out are the holds under the new
 * numbers; live[0] the number of pages in use.  What the moved pages held before stays in their old
 * places, now free.
 *
 * page_table     INT64 [B, maxPages], page_table_out the same shape; it may be page_table itself.
 * ref_counts, ref_counts_out INT64 [pages], the latter may be ref_counts itself; page_map INT64
 * [pages], live INT64 [1].  caches as in rope_copy_pages, num_caches may be 0.
 */
int64_t rope_compact_pages_workspace(int64_t num_pages);
int rope_compact_pages(const rope_tensor *page_table, const rope_tensor *ref_counts,
                       const rope_tensor *caches, int64_t num_caches,
                       const rope_tensor *page_table_out, const rope_tensor *ref_counts_out,
                       const rope_tensor *page_map, const rope_tensor *live, void *workspace,
                       int64_t workspace_bytes, void *stream);

/* Text describing the last failing call on the calling thread ("" if none).  The pointer
 * stays valid until the next call on this thread. */
const char *rope_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_AMD_H */
