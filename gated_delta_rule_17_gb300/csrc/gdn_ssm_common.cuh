// The selective state space scan: the recurrence of the state with a scalar decay per head,
//
//     d_t = softplus(dt_t + dt_bias);   S_t = e^{d_t a} S_{t-1} + k_t (d_t v_t)^T;   o_t = S_t^T q_t + skip v_t
//
// with S [dk][dv] in fp32, and nv / nk value heads to a query and key head.
#pragma once
#include "gdn_row_common.cuh"

namespace gdn {

struct SsmParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const void* dt;        // fp32, or bf16 where dt_bf16
  const float* a;        // [nv]
  const float* dt_bias;  // [nv] or null
  const float* skip;     // [nv] or null
  void* state;           // float[B][nv][dk][dv], or float*[B] where state_is_table
  __nv_bfloat16* out;
  int64_t q_stride, k_stride, v_stride, dt_stride, out_stride;
  Rows batch;
  int nk, nv;
  int state_is_table, dt_bf16, softplus;
  unsigned* status;
};

// The step d of a row and head.
__device__ __forceinline__ float ssm_step_of(const SsmParams& p, int64_t row, int h, float bias) {
  const int64_t at = row * p.dt_stride + h;
  const float z = (p.dt_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.dt)[at]) : static_cast<const float*>(p.dt)[at]) + bias;
  return p.softplus ? fmaxf(z, 0.f) + log1pf(__expf(-fabsf(z))) : z;
}

template <int DK, int DV>
__device__ __forceinline__ float* ssm_state(const SsmParams& p, int s, int h) {
  float* base = p.state_is_table ? static_cast<float* const*>(p.state)[s] : static_cast<float*>(p.state) + static_cast<int64_t>(s) * p.nv * DK * DV;
  return base + static_cast<int64_t>(h) * DK * DV;
}

// ---- one token -----------------------------------------------------------------------
// Bound by the state's way through HBM, once in and once out (64 KB each for 128 x 128); a CTA has a
// sequence and head, a thread 16 float4 of the state in registers: rows r, r + ROWS, ... of four columns.
// 256 sequences of 32 heads of 128 x 128: 155 us, 6.95 TB/s, the measured copy rate and a little more.
template <int DK, int DV>
constexpr int ssm_threads = DK * DV / 64;

template <int DK, int DV>
__global__ void __launch_bounds__(ssm_threads<DK, DV>) gdn_ssm_decode_kernel(const SsmParams p) {
  constexpr int THREADS = ssm_threads<DK, DV>, LANES = DV / 4, ROWS = THREADS / LANES;
  static_assert(DK == 16 * ROWS, "16 rows a thread");
  __shared__ float s_k[DK], s_q[DK];
  __shared__ __align__(16) float s_part[ROWS][DV];
  const int tid = threadIdx.x, col = 4 * (tid % LANES), r0 = tid / LANES;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.nv)), b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.nv));
  const int kh = h / (p.nv / p.nk);
  tc::grid_dependency_wait();
  float* S = ssm_state<DK, DV>(p, b, h) + col;
  float4 s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = *reinterpret_cast<const float4*>(S + (i * ROWS + r0) * DV);
  for (int i = tid; i < DK; i += THREADS) {
    s_k[i] = __bfloat162float(p.k[b * p.k_stride + kh * DK + i]);
    s_q[i] = __bfloat162float(p.q[b * p.q_stride + kh * DK + i]);
  }
  const float d = ssm_step_of(p, b, h, p.dt_bias ? p.dt_bias[h] : 0.f), decay = __expf(d * p.a[h]);
  float v[4];
  load4(p.v + b * p.v_stride + h * DV + col, v);
  const float4 dv = make_float4(d * v[0], d * v[1], d * v[2], d * v[3]);
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = i * ROWS + r0;
    const float kk = s_k[r], qq = s_q[r];
    s[i].x = fmaf(kk, dv.x, decay * s[i].x);
    s[i].y = fmaf(kk, dv.y, decay * s[i].y);
    s[i].z = fmaf(kk, dv.z, decay * s[i].z);
    s[i].w = fmaf(kk, dv.w, decay * s[i].w);
    *reinterpret_cast<float4*>(S + r * DV) = s[i];
    o.x = fmaf(qq, s[i].x, o.x);
    o.y = fmaf(qq, s[i].y, o.y);
    o.z = fmaf(qq, s[i].z, o.z);
    o.w = fmaf(qq, s[i].w, o.w);
  }
  *reinterpret_cast<float4*>(&s_part[r0][col]) = o;
  __syncthreads();
  if (tid < LANES) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const float4 t = *reinterpret_cast<const float4*>(&s_part[j][col]);
      f[0] += t.x;
      f[1] += t.y;
      f[2] += t.z;
      f[3] += t.w;
    }
    const float skip = p.skip ? p.skip[h] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fmaf(skip, v[i], f[i]);
    store4(p.out + b * p.out_stride + h * DV + col, f);
  }
}

}  // namespace gdn
