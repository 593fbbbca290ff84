// The scan over prompts, token by token: a CTA has a sequence and head with its state in registers, as
// the single-token kernel has it. The plainest kernel that is right.
#pragma once
#include "gdn_ssm_common.cuh"

namespace gdn {

template <int DK, int DV>
__global__ void __launch_bounds__(ssm_threads<DK, DV>) gdn_ssm_scan_kernel(const SsmParams p) {
  constexpr int THREADS = ssm_threads<DK, DV>, LANES = DV / 4, ROWS = THREADS / LANES;
  __shared__ float s_k[DK], s_q[DK];
  __shared__ __align__(16) float s_part[ROWS][DV];
  const int tid = threadIdx.x, col = 4 * (tid % LANES), r0 = tid / LANES;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.nv)), b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.nv));
  const int kh = h / (p.nv / p.nk);
  const int start = p.batch.start(b), end = p.batch.end(b);
  if (h == 0 && tid == 0) p.batch.report(b, p.status);
  if (!rows_held(start, end, p.batch.rows) || start == end) return;
  float* S = ssm_state<DK, DV>(p, b, h) + col;
  float4 s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = *reinterpret_cast<const float4*>(S + (i * ROWS + r0) * DV);
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f, a = p.a[h], skip = p.skip ? p.skip[h] : 0.f;
  for (int64_t row = start; row < end; ++row) {
    for (int i = tid; i < DK; i += THREADS) {
      s_k[i] = __bfloat162float(p.k[row * p.k_stride + kh * DK + i]);
      s_q[i] = __bfloat162float(p.q[row * p.q_stride + kh * DK + i]);
    }
    const float d = ssm_step_of(p, row, h, bias), decay = __expf(d * a);
    float v[4];
    load4(p.v + row * p.v_stride + h * DV + col, v);
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = i * ROWS + r0;
      const float kk = d * s_k[r], qq = s_q[r];
      s[i].x = fmaf(kk, v[0], decay * s[i].x);
      s[i].y = fmaf(kk, v[1], decay * s[i].y);
      s[i].z = fmaf(kk, v[2], decay * s[i].z);
      s[i].w = fmaf(kk, v[3], decay * s[i].w);
      o.x = fmaf(qq, s[i].x, o.x);
      o.y = fmaf(qq, s[i].y, o.y);
      o.z = fmaf(qq, s[i].z, o.z);
      o.w = fmaf(qq, s[i].w, o.w);
    }
    *reinterpret_cast<float4*>(&s_part[r0][col]) = o;
    __syncthreads();
    if (tid < LANES) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = skip * v[i];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float4 t = *reinterpret_cast<const float4*>(&s_part[j][col]);
        f[0] += t.x;
        f[1] += t.y;
        f[2] += t.z;
        f[3] += t.w;
      }
      store4(p.out + row * p.out_stride + h * DV + col, f);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) *reinterpret_cast<float4*>(S + (i * ROWS + r0) * DV) = s[i];
}

}  // namespace gdn
