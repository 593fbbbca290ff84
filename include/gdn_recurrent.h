/*
 * gdn_recurrent.h -- C ABI of the operators that stand around and beside the
 * gated delta rule in a linear-attention layer: the short causal convolution
 * before the recurrence (with its backward), the selective state space scan
 * (the recurrence with a scalar decay and no erase) for prompts and for single
 * tokens, and the layer norm after it, gated or not (with its backward).
 *
 * Return codes, the error message, the launch count and the device status word
 * are those of gdn_prefill.h (gdn_last_error, gdn_last_launch_count,
 * gdn_prefill_check). Every call enqueues on `stream` (a cudaStream_t as void*)
 * and returns; host-detectable errors launch nothing. Pointers are device
 * addresses on the current device; tensors are 16-byte aligned and row strides
 * (in elements) are multiples of 8 unless said otherwise. Buffers stay valid
 * until the stream has passed the call. Arithmetic is fp32 unless said
 * otherwise, and each output is rounded once. Element types are GDN_BF16,
 * GDN_F16 and GDN_F32 of gdn_attention.h.
 *
 * Batches: dense (cu_seqlens NULL) B sequences of T tokens, row b*T + t; or
 * packed, B sequences in `T` rows in total, sequence s with the rows
 * [cu_seqlens[s], cu_seqlens[s+1]): cu_seqlens is int32 [B+1] on the device,
 * rises from 0 and ends at T or before; rows behind its end are neither read
 * nor written. Sequences of no token keep their state. A sequence whose
 * offsets fall, or pass T, writes nothing, and gdn_prefill_check reports
 * GDN_ERR_DEVICE_STATUS.
 */
#ifndef GDN_RECURRENT_H
#define GDN_RECURRENT_H

#include "gdn_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The causal convolution of each of D channels with `width` taps:
 *     y[t] = bias + sum_j weight[j] x[t - (width-1) + j],  out = y sigmoid(y) (silu = 1) or y
 *   x, out  : [rows][D] `dtype` elements at row strides x_stride, out_stride (0: D).
 *             out overlaps no input.
 *   weight  : fp32 [D][width], width 2, 3 or 4; bias: fp32 [D] or NULL.
 *   state   : the width-1 inputs before each sequence's first, `dtype` elements
 *             [B][width-1][D], overwritten with the last width-1 (old state and new
 *             inputs together); with state_is_table = 1 a device array of B device
 *             pointers, each to a 16-byte aligned [width-1][D]. NULL: zeros, and
 *             nothing is kept.
 * A table's pointers differ from one another. D is a multiple of 8 up to 2^26. One launch (two where a sequence that has a state may be
 * longer than a thread's strip of rows). */
int gdn_causal_conv(const void* x, const float* weight, const float* bias, void* state, void* out, int B, int T,
                    int D, int width, int silu, int dtype, int state_is_table, int64_t x_stride, int64_t out_stride,
                    const int32_t* cu_seqlens, void* stream);

/* Backward of gdn_causal_conv. x, weight, bias, silu as given to the forward.
 *   h0       : the state that the forward started from, [B][width-1][D], or NULL
 *   dout     : dL/dout; dST: dL/d(state after the call), [B][width-1][D], or NULL
 *   dx       : dL/dx, `dtype` elements; overlaps no input
 *   dweight, dbias : fp32 [D][width], [D], overwritten; NULL where not wanted. Sums in
 *              a fixed order: the same inputs give the same bits.
 *   dh0      : dL/dh0, [B][width-1][D], or NULL
 *   workspace: gdn_causal_conv_backward_workspace_bytes(rows, ...) bytes, 256-byte
 *              aligned, or NULL to allocate it stream-ordered. Calls that overlap
 *              need one each.
 * One launch, and another for the weights' gradients and dh0. */
size_t gdn_causal_conv_backward_workspace_bytes(int rows, int D, int width);
int gdn_causal_conv_backward(const void* x, const float* weight, const float* bias, const void* h0, const void* dout,
                             const void* dST, void* dx, float* dweight, float* dbias, void* dh0, int B, int T, int D,
                             int width, int silu, int dtype, int64_t x_stride, int64_t dout_stride, int64_t dx_stride,
                             const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes, void* stream);

/* Row strides in elements, and how the steps are given:
 *   dt        : any stride >= nv; the elements are fp32, or bf16 with dt_bf16 = 1
 *   softplus  : 1 -> the step is log(1 + e^(dt + dt_bias)); 0 -> dt + dt_bias
 *   state_is_table : as in gdn_strides_t
 * NULL: packed rows, fp32 dt, softplus, a contiguous state. */
typedef struct {
  int64_t q, k, v, dt, out;
  int32_t state_is_table;
  int32_t dt_bf16;
  int32_t softplus;
} gdn_ssm_options_t;

/* The selective state space scan of every sequence and value head h, with key
 * and query head h / (nv / nk) (in state space terms q is C, k is B, v is x):
 *     d = step(dt_t + dt_bias[h]);  S_t = e^(d a[h]) S_{t-1} + k_t (d v_t)^T
 *     o_t = S_t^T q_t + skip[h] v_t
 *   q, k     : bf16 [rows][nk][dk];  v, out : bf16 [rows][nv][dv]; out overlaps no input
 *   a        : fp32 [nv], <= 0;  dt_bias, skip : fp32 [nv] or NULL (zeros). Steps are >= 0.
 *   state    : fp32 [B][nv][dk][dv] (or a table of B pointers to [nv][dk][dv], each
 *              16-byte aligned, no two the same), read as S_0 and overwritten with
 *              the last S.
 *   dk, dv   : 64 or 128 each.
 * Chunks of 128 tokens on the tensor cores: products take bf16 operands and sum in
 * fp32; the state is fp32, its updates keep 16 bits of each term. Steps, decays and
 * their sums are fp32. q, k and v of a sequence's own tokens must be finite (a value
 * that is not reaches the whole chunk's outputs); what lies behind a sequence need not.
 * Chunks may be summed up to 5e21 times above or below their size: the sums over 128
 * tokens of |q.k| d |v| and of |k| d |v| stay below 6e16, beyond which outputs and state
 * may be infinite; of d |v| and state elements below 6e-17 outputs may take less than
 * 8 bits, or nothing.
 * The same inputs give the same bits. Packed batches of more than 32 sequences run in
 * their given order, without segments: long ones go first in them, or into a call of
 * their own.
 *   workspace: gdn_ssm_scan_workspace_bytes() bytes, 256-byte aligned, or NULL to
 *              allocate it stream-ordered. Calls that overlap need one each. It may be 0:
 *              segments of long sequences take it, where there are few heads for the SMs.
 * One launch, or two with segments. */
size_t gdn_ssm_scan_workspace_bytes(int B, int T, int nk, int nv, int dk, int dv, int varlen);
int gdn_ssm_scan(const void* q, const void* k, const void* v, const void* dt, const float* a, const float* dt_bias,
                 const float* skip, void* state, void* out, int B, int T, int nk, int nv, int dk, int dv,
                 const gdn_ssm_options_t* options, const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes,
                 void* stream);

/* One token of every sequence: row b of q, k, v, dt and out belongs to sequence b.
 * out may be v itself (with its stride), and overlaps no other input. One launch. */
int gdn_ssm_decode(const void* q, const void* k, const void* v, const void* dt, const float* a, const float* dt_bias,
                   const float* skip, void* state, void* out, int B, int nk, int nv, int dk, int dv,
                   const gdn_ssm_options_t* options, void* stream);

/* Row strides in elements; NULL: packed rows of groups * dim. */
typedef struct {
  int64_t x, gate, out, dout, dgate; /* out: that of dx in the backward */
} gdn_layer_norm_strides_t;

/* Norm of each of `groups` groups of `dim` values in every row:
 *     h = (u - mean(u)) / sqrt(mean((u - mean(u))^2) + eps);  out = h weight + bias
 * with u = x; with rms = 1 the mean is taken as 0. With a gate z, out is multiplied
 * by silu(z) = z sigmoid(z), or, with gate_first = 1, u = x silu(z).
 *   x, gate, out : [rows][groups][dim] `dtype` elements; gate may be NULL; out may be x
 *                  or gate itself (with its stride)
 *   weight, bias : fp32 [dim], shared by the groups; NULL for ones, zeros
 * dim is a multiple of 8 up to 8192. One launch. */
int gdn_layer_norm(const void* x, const void* gate, const float* weight, const float* bias, float eps, void* out, int rows,
                   int groups, int dim, int dtype, int rms, int gate_first, const gdn_layer_norm_strides_t* strides,
                   void* stream);

/* Backward of gdn_layer_norm. x, gate, weight, bias and the rest as given to it.
 *   dx, dgate      : dL/dx, dL/dgate, `dtype` elements; dgate wherever there is a gate.
 *                    Each may be x, dout or gate itself (with its stride), not both the same.
 *   dweight, dbias : fp32 [dim], overwritten with the sums over rows and groups, in a
 *                    fixed order; NULL where not wanted.
 *   workspace      : gdn_layer_norm_backward_workspace_bytes() bytes, 256-byte aligned,
 *                    or NULL to allocate it stream-ordered; one for each of calls that overlap.
 * One launch, and another for the weights' gradients. */
size_t gdn_layer_norm_backward_workspace_bytes(int rows, int groups, int dim);
int gdn_layer_norm_backward(const void* x, const void* gate, const float* weight, const float* bias, float eps,
                            const void* dout, void* dx, void* dgate, float* dweight, float* dbias, int rows, int groups,
                            int dim, int dtype, int rms, int gate_first, const gdn_layer_norm_strides_t* strides,
                            void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_RECURRENT_H */
