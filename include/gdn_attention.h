/*
 * gdn_attention.h -- C ABI of the softmax-attention operators that stand next
 * to the gated delta rule in a hybrid model: the norm and rotation of query
 * and key heads (with its backward), the append to a paged key/value cache and
 * the attention of decode tokens or drafted token trees over that cache.
 *
 * Return codes, the error message, the launch count and the device status word
 * are those of gdn_prefill.h (gdn_last_error, gdn_last_launch_count,
 * gdn_prefill_check). Every call enqueues on `stream` (a cudaStream_t as void*)
 * and returns; host-detectable errors launch nothing. Pointers are device
 * addresses on the current device unless marked host; all 16-bit and 32-bit
 * element tensors are 16-byte aligned and row strides are multiples of 8
 * elements. Buffers stay valid until the stream has passed the call.
 */
#ifndef GDN_ATTENTION_H
#define GDN_ATTENTION_H

#include "gdn_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations and caches. */
enum { GDN_BF16 = 0, GDN_F16 = 1, GDN_F32 = 2 };

/* The rotation of a head's first `rot` values by a token's position p: value
 * pair i (0 <= i < rot / 2) is turned by the angle whose cosine and sine are
 * cos[p * stride + i], sin[p * stride + i] (fp32, `positions` rows).
 *   rot         : a multiple of 8, <= head_dim; 0 (or a NULL struct): no rotation
 *   interleaved : 0 -> pair i is (x[i], x[i + rot/2]); 1 -> (x[2i], x[2i+1])
 * A row whose position is outside [0, positions) is skipped and reported by
 * gdn_prefill_check as GDN_ERR_DEVICE_STATUS. cos and sin are 16-byte aligned
 * and stride is a multiple of 4, >= rot / 2. */
typedef struct {
  const float* cos;
  const float* sin;
  int64_t stride;
  int32_t positions;
  int32_t rot;
  int32_t interleaved;
} gdn_rope_t;

/* Row strides in elements: q and k inputs, their outputs, and (backward only)
 * the incoming gradients. NULL means packed rows. */
typedef struct {
  int64_t q, k, q_out, k_out, q_grad, k_grad;
} gdn_norm_strides_t;

/* RMS norm of every head row of q and k, then the rotation, in one pass:
 *     r = 1 / sqrt(mean(x^2) + eps),  y = rotate(x r w, position)
 *   q, k       : [rows][nq][d] and [rows][nkv][d], `dtype` elements. Either may be
 *                absent (NULL with a head count of 0).
 *   q_weight, k_weight : fp32 [d], shared by all heads; NULL means ones.
 *   positions  : int32 [rows]; may be NULL without a rotation.
 *   q_out, k_out : the same type and shape; may be the inputs themselves.
 * d is 64 or 128. Arithmetic is fp32, rounded once. One launch. */
int gdn_head_norm_rope(const void* q, const void* k, const int32_t* positions, const gdn_rope_t* rope,
                       const float* q_weight, const float* k_weight, float eps, void* q_out, void* k_out, int rows,
                       int nq, int nkv, int d, int dtype, const gdn_norm_strides_t* strides, void* stream);

/* Backward of gdn_head_norm_rope. q, k, positions, rope, weights and eps as
 * given to the forward.
 *   q_grad, k_grad : dL/dq_out, dL/dk_out, `dtype` elements.
 *   dq, dk         : dL/dq, dL/dk, `dtype` elements (strides q_out, k_out); dq may be
 *                    q_grad itself, dk k_grad.
 *   dq_weight, dk_weight : fp32 [d], overwritten with the sums over all rows and
 *                    heads; NULL where not wanted. The sums are fp32 in a fixed order:
 *                    the same inputs give the same bits.
 *   workspace      : gdn_head_norm_rope_backward_workspace_bytes() bytes, 256-byte
 *                    aligned, or NULL to allocate it stream-ordered.
 * Two launches (one without weight gradients). */
size_t gdn_head_norm_rope_backward_workspace_bytes(int rows, int nq, int nkv, int d);
int gdn_head_norm_rope_backward(const void* q, const void* k, const int32_t* positions, const gdn_rope_t* rope,
                                const float* q_weight, const float* k_weight, float eps, const void* q_grad,
                                const void* k_grad, void* dq, void* dk, float* dq_weight, float* dk_weight, int rows,
                                int nq, int nkv, int d, int dtype, const gdn_norm_strides_t* strides, void* workspace,
                                size_t workspace_bytes, void* stream);

/* A paged key/value cache and the batch that uses it. Token t of sequence b
 * lives at place t % page_size of page block_table[b * table_stride + t / page_size];
 * head h of it at k + page * k_page + place * k_token + h * k_head (strides in
 * elements, multiples of 8; v likewise), d contiguous values. A call's new rows
 * are packed: rows [cu_rows[b], cu_rows[b+1]) belong to sequence b (cu_rows[0] = 0,
 * non-decreasing, cu_rows[B] = rows), or row b to sequence b where cu_rows is
 * NULL (then rows == B). New row i of sequence b is token ctx_lens[b] + i of it.
 * Entries of block_table past a sequence's tokens are not read. Malformed
 * cu_rows or ctx_lens, and page numbers outside [0, num_pages), are found on the
 * device and reported by gdn_prefill_check as GDN_ERR_DEVICE_STATUS: the rows or
 * sequences concerned are not written; to the attention, a token on such a page
 * has a key and a value of zeros. */
typedef struct {
  void* k;
  void* v;
  int64_t k_page, k_token, k_head;
  int64_t v_page, v_token, v_head;
  int32_t num_pages, page_size;
  const int32_t* block_table; /* [B][max_pages] */
  int64_t table_stride;
  int32_t max_pages;
  int32_t B, rows;
  const int32_t* ctx_lens; /* [B] tokens of each sequence before this call's rows */
  const int32_t* cu_rows;  /* [B + 1] or NULL */
} gdn_paged_t;

/* Write the new rows' keys and values into the cache; the keys are normed
 * (norm = 1; k_weight fp32 [d] or NULL for ones) and rotated on the way, the
 * values copied. positions: int32 [rows], or NULL to rotate each row by its
 * token index ctx_lens[b] + i (drafted tokens of a tree give their depth
 * instead). k, v: [rows][nkv][d] at row strides k_stride, v_stride (0: packed);
 * dtype GDN_BF16 or GDN_F16, that of the cache. One launch. */
int gdn_paged_append(const void* k, const void* v, const gdn_paged_t* cache, const int32_t* positions,
                     const gdn_rope_t* rope, int norm, const float* k_weight, float eps, int nkv, int d, int dtype,
                     int64_t k_stride, int64_t v_stride, void* stream);

/* Attention of the new rows over the cache:
 *     out[row, h] = sum_t softmax_t(scale q[row, h] . k[t, h / (nq/nkv)]) v[t, h / (nq/nkv)]
 * over the tokens t that the row sees: all ctx_lens[b] tokens of its sequence's
 * context, and of the new tokens ctx_lens[b] + j (already in the cache) those
 * whose bit j % 64 of mask[row * mask_words + j / 64] is set, so a row sees
 * itself only if its own bit is set; with mask NULL those with j <= i. A row
 * that sees no token gives zeros. Bits past the sequence's rows, and new tokens
 * past 64 * mask_words, count as unseen.
 *   q, out   : [rows][nq][d] at row strides q_stride, out_stride (0: packed);
 *              dtype GDN_BF16 or GDN_F16, that of the cache. out overlaps no input.
 *   max_rows : an upper bound on the rows of one sequence, by which the kernel is
 *              chosen; a wrong one costs time, not correctness. 0: `rows`.
 *   workspace: gdn_tree_attention_workspace_bytes() bytes, 256-byte aligned, or NULL
 *              to allocate it stream-ordered. Calls that overlap need one each.
 * d is 64 or 128. Products take 16-bit operands (the softmax's weights are
 * rounded to dtype for the second product; fp16 weights below 2^-31 of a row's
 * largest count as zero there), scores, statistics and sums are fp32. The keys and values of every token below ctx_lens[b] + (rows of b) must
 * be finite, seen or not; what lies past them, in a page or outside, is not
 * used. The same inputs give the same bits. At most two launches. */
size_t gdn_tree_attention_workspace_bytes(int nq, int nkv, int d);
int gdn_tree_attention(const void* q, const gdn_paged_t* cache, const uint64_t* mask, int mask_words, float scale,
                       void* out, int nq, int nkv, int d, int dtype, int64_t q_stride, int64_t out_stride,
                       int max_rows, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H */
