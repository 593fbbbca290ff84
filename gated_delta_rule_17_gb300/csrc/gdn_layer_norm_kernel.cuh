// Layer norm and RMS norm of rows, with an optional gate, and the backward pass, for sm_103a.
//
// For a group of n values x with weights w, b and gate z (s(z) = z sigmoid(z)):
//
//     u = x (or x s(z), the gate first);   m = mean(u) (0 for the RMS norm);   r = 1 / sqrt(mean((u - m)^2) + eps)
//     h = (u - m) r;   y = h w + b;   out = y (or y s(z), the gate after)
//
// and backward, with dy = dout (or dout s(z), and dz = dout y s'(z)):
//
//     dw = sum dy h;  db = sum dy;  t = dy w;  du = r (t - mean(t) - h mean(t h))     (no mean(t) for the RMS norm)
//     dx = du (or du s(z), and dz = du x s'(z))
//
// Bound by HBM: 4 to 10 bytes a value in 16-bit types. A group is read once and stays in the registers
// of L lanes of a warp, or of a CTA; the variance is that of the differences from the mean, as they are there.
#pragma once
#include "gdn_row_common.cuh"

namespace gdn {

struct LayerNormParams {
  const void* x;
  const void* gate;
  const float* weight;  // [dim] or null
  const float* bias;    // [dim] or null
  void* out;            // backward: dx
  const void* dout;
  void* dgate;
  float* partials;  // backward: [ctas][2][dim] sums for the weight and the bias, or null
  int64_t x_stride, gate_stride, out_stride, dout_stride, dgate_stride;
  int64_t items;  // rows x groups
  int groups, dim;
  int rms, gate_first;
  float eps;
};

// Sum over the L lanes (a power of two up to 32) or, for larger L, over the CTA of L threads that hold a
// group; `buf` holds 128 floats then, and `turn` alternates between its halves, so that one barrier does.
template <int L, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* buf, int& turn) {
#pragma unroll
  for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (L > 32) {
    constexpr int WARPS = L / 32;
    float* at = buf + turn * 64;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) at[k * 32 + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) v[k] += at[k * 32 + i];
    }
  }
}

// Eight values of a row.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(w[i].x);
        f[4 * i + 1] = __uint_as_float(w[i].y);
        f[4 * i + 2] = __uint_as_float(w[i].z);
        f[4 * i + 3] = __uint_as_float(w[i].w);
      }
    } else {
      floats16<T>(w[0], f);
    }
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = pack16<T>(f);
  }
}
__device__ __forceinline__ void weights8(const float* w, int c, float other, float (&f)[8]) {
  if (w) {
    const float4 a = *reinterpret_cast<const float4*>(w + c), b = *reinterpret_cast<const float4*>(w + c + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = other;
  }
}

// Threads of a CTA: that of a group, or 128.
template <int L>
constexpr int norm_threads = L > 128 ? L : 128;

// Mean and 1 / deviation of the group's values u (zeros past its end, where `held` is false).
template <int L, int NV>
__device__ __forceinline__ void norm_stats(const LayerNormParams& p, const float (&u)[NV][8], const bool (&held)[NV], float* buf, int& turn,
                                           float& mean, float& r) {
  const float inv = 1.f / static_cast<float>(p.dim);
  mean = 0.f;
  if (!p.rms) {
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += u[v][i];
    group_sum<L>(s, buf, turn);
    mean = s[0] * inv;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (held[v])
#pragma unroll
      for (int i = 0; i < 8; ++i) q[0] = fmaf(u[v][i] - mean, u[v][i] - mean, q[0]);
  group_sum<L>(q, buf, turn);
  r = rsqrtf(q[0] * inv + p.eps);
}

// L lanes hold a group, NV words of eight values each.
template <typename T, int L, int NV, bool kGate>
__global__ void __launch_bounds__(norm_threads<L>) gdn_layer_norm_kernel(const LayerNormParams p) {
  constexpr int SLOTS = norm_threads<L> / L;
  __shared__ float buf[128];
  int turn = 0;
  const int lane = threadIdx.x % L;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * SLOTS + threadIdx.x / L;
  const bool real = item < p.items;
  const int64_t row = real ? item / p.groups : 0;
  const int64_t at = real ? (item - row * p.groups) * p.dim : 0;
  Eight<T> xw[NV], zw[NV];
  bool held[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * L + lane) * 8;
    held[v] = real && c < p.dim;
    xw[v].zero();
    zw[v].zero();
    if (held[v]) {
      xw[v].load(static_cast<const T*>(p.x) + row * p.x_stride + at + c);
      if (kGate) zw[v].load(static_cast<const T*>(p.gate) + row * p.gate_stride + at + c);
    }
  }
  float u[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    xw[v].floats(u[v]);
    if (kGate && p.gate_first) {
      float z[8];
      zw[v].floats(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] *= silu(z[i]);
    }
  }
  float mean, r;
  norm_stats<L, NV>(p, u, held, buf, turn, mean, r);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * L + lane) * 8;
    if (!held[v]) continue;
    float w[8], b[8];
    weights8(p.weight, c, 1.f, w);
    weights8(p.bias, c, 0.f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[v][i] = fmaf((u[v][i] - mean) * r, w[i], b[i]);
    if (kGate && !p.gate_first) {
      float z[8];
      zw[v].floats(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] *= silu(z[i]);
    }
    store8(static_cast<T*>(p.out) + row * p.out_stride + at + c, u[v]);
  }
}

// ---- backward ------------------------------------------------------------------------
// A fixed grid: a slot of L lanes walks every (grid x slots)-th group, the next one's words under way, and
// keeps the sums of its own columns.
template <typename T, int L, int NV, bool kGate>
__global__ void __launch_bounds__(norm_threads<L>) gdn_layer_norm_bwd_kernel(const LayerNormParams p) {
  constexpr int SLOTS = norm_threads<L> / L;
  __shared__ float buf[128];
  __shared__ float s_sum[SLOTS > 1 ? SLOTS * L * NV * 8 : 1];
  int turn = 0;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t step = static_cast<int64_t>(gridDim.x) * SLOTS;
  float dw[NV][8] = {}, db[NV][8] = {};
  Eight<T> xw[NV], gw[NV], zw[NV];
  auto fetch = [&](int64_t item) {
    const bool real = item < p.items;
    const int64_t row = real ? item / p.groups : 0, at = real ? (item - row * p.groups) * p.dim : 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      xw[v].zero();
      gw[v].zero();
      zw[v].zero();
      if (real && c < p.dim) {
        xw[v].load(static_cast<const T*>(p.x) + row * p.x_stride + at + c);
        gw[v].load(static_cast<const T*>(p.dout) + row * p.dout_stride + at + c);
        if (kGate) zw[v].load(static_cast<const T*>(p.gate) + row * p.gate_stride + at + c);
      }
    }
  };
  int64_t item = static_cast<int64_t>(blockIdx.x) * SLOTS + slot;
  fetch(item);
  // every slot of the CTA takes as many steps, for the shuffles and barriers among them
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * SLOTS; first < p.items; first += step, item += step) {
    const bool real = item < p.items;
    const int64_t row = real ? item / p.groups : 0, at = real ? (item - row * p.groups) * p.dim : 0;
    float u[NV][8], g[NV][8];
    Eight<T> xc[NV], zc[NV];
    bool held[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      held[v] = real && (v * L + lane) * 8 < p.dim;
      xw[v].floats(u[v]);
      gw[v].floats(g[v]);
      if constexpr (kGate) {
        xc[v] = xw[v];
        zc[v] = zw[v];
        if (p.gate_first) {
          float z[8];
          zc[v].floats(z);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[v][i] *= silu(z[i]);
        }
      }
    }
    fetch(item + step);
    float mean, r;
    norm_stats<L, NV>(p, u, held, buf, turn, mean, r);
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      if (!held[v]) continue;
      float w[8], b[8], z[8], dz[8];
      weights8(p.weight, c, 1.f, w);
      if (kGate && !p.gate_first) {
        weights8(p.bias, c, 0.f, b);
        zc[v].floats(z);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = (u[v][i] - mean) * r;
        if (kGate && !p.gate_first) {
          const float sg = sigmoid(z[i]), s = z[i] * sg;
          dz[i] = g[v][i] * fmaf(h, w[i], b[i]) * (sg + s * (1.f - sg));
          g[v][i] *= s;
        }
        dw[v][i] = fmaf(g[v][i], h, dw[v][i]);
        db[v][i] += g[v][i];
        u[v][i] = h;
        g[v][i] *= w[i];
        sums[0] += g[v][i];
        sums[1] = fmaf(g[v][i], h, sums[1]);
      }
      if (kGate && !p.gate_first) store8(static_cast<T*>(p.dgate) + row * p.dgate_stride + at + c, dz);
    }
    group_sum<L>(sums, buf, turn);
    const float inv = 1.f / static_cast<float>(p.dim), mt = p.rms ? 0.f : sums[0] * inv, mth = sums[1] * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      if (!held[v]) continue;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) dx[i] = r * (g[v][i] - mt - u[v][i] * mth);
      if (kGate && p.gate_first) {
        float x[8], z[8], dz[8];
        xc[v].floats(x);
        zc[v].floats(z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float sg = sigmoid(z[i]), s = z[i] * sg;
          dz[i] = dx[i] * x[i] * (sg + s * (1.f - sg));
          dx[i] *= s;
        }
        store8(static_cast<T*>(p.dgate) + row * p.dgate_stride + at + c, dz);
      }
      store8(static_cast<T*>(p.out) + row * p.out_stride + at + c, dx);
    }
  }
  if (!p.partials) return;
  // the CTA's sums, slot after slot
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (SLOTS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_sum[(slot * NV + v) * L * 8 + lane * 8 + i] = k ? db[v][i] : dw[v][i];
      __syncthreads();
      for (int c = threadIdx.x; c < p.dim; c += norm_threads<L>) {
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) acc += s_sum[i * NV * L * 8 + c];
        out[k * p.dim + c] = acc;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * L + lane) * 8;
        if (c >= p.dim) continue;
        store4(out + k * p.dim + c, reinterpret_cast<const float(&)[4]>(k ? db[v][0] : dw[v][0]));
        store4(out + k * p.dim + c + 4, reinterpret_cast<const float(&)[4]>(k ? db[v][4] : dw[v][4]));
      }
    }
  }
}

// The CTAs' sums, added up in their order.
__global__ void __launch_bounds__(1024) gdn_layer_norm_sum_kernel(const float* partials, int ctas, int dim, float* dweight, float* dbias) {
  tc::grid_dependency_wait();
  sum_columns(partials, ctas, 2 * dim, static_cast<int>(blockIdx.x) * 32, [&](int c, float v) {
    if (c < dim) {
      if (dweight) dweight[c] = v;
    } else if (dbias) {
      dbias[c - dim] = v;
    }
  });
}

}  // namespace gdn
