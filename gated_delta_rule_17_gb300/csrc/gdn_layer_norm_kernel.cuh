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
// of L lanes of a warp, or of a CTA; the variance is that of the differences from the mean, as they are there. What then
// counts are the loads under way: a lane takes several groups at once, and the backward's CTAs, which have to stay to
// keep the columns' sums, copy the rows to come into a ring in shared memory.
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
  int stages;  // backward of wide groups: rows of the ring
  unsigned* status;
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
      float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < WARPS; i += 4) {
        float g[4];
        load4(at + k * 32 + i, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += g[e];
      }
      v[k] = (f[0] + f[1]) + (f[2] + f[3]);
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
// The same as pairs; and pairs as values.
template <typename T>
__device__ __forceinline__ void pairs8(const Eight<T>& e, Pair (&p)[4]) {
  if constexpr (sizeof(T) == 4) {
    unpack16<T>(e.w[0], *reinterpret_cast<Pair(*)[2]>(&p[0]));
    unpack16<T>(e.w[1], *reinterpret_cast<Pair(*)[2]>(&p[2]));
  } else {
    unpack16<T>(e.w[0], p);
  }
}
__device__ __forceinline__ void values8(const Pair (&p)[4], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) parts_of(p[i], f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ Pair both(float x) { return pair_of(x, x); }
__device__ __forceinline__ float sum_of(Pair p) {
  float a, b;
  parts_of(p, a, b);
  return a + b;
}

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

// Groups that a lane takes at once.
template <int L, int NV>
constexpr int norm_rows = L <= 32 && NV == 1 ? 4 : 1;

// L lanes hold a group, NV words of eight values each; R groups at once, all loads first: 32768 x 32 gated groups of 128 in bf16
// take 122 us so, 6.6 TB/s (97% of the measured copy rate), 163 with one group at a time.
template <typename T, int L, int NV, bool kGate>
__global__ void __launch_bounds__(norm_threads<L>) gdn_layer_norm_kernel(const LayerNormParams p) {
  constexpr int SLOTS = norm_threads<L> / L, R = norm_rows<L, NV>;
  __shared__ __align__(16) float buf[128];
  int turn = 0;
  const int lane = threadIdx.x % L;
  const uint32_t first = blockIdx.x * (SLOTS * R) + threadIdx.x / L, groups = static_cast<uint32_t>(p.groups), items = static_cast<uint32_t>(p.items);
  tc::grid_dependency_wait();
  Eight<T> xw[R][NV], zw[kGate ? R : 1][NV];
  uint32_t row[R], at[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const uint32_t item = first + k * SLOTS;
    row[k] = item / groups;
    at[k] = (item - row[k] * groups) * p.dim;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      xw[k][v].zero();
      if (kGate) zw[k][v].zero();
      if (item < items && c < p.dim) {
        xw[k][v].load(static_cast<const T*>(p.x) + row[k] * p.x_stride + at[k] + c);
        if (kGate) zw[k][v].load(static_cast<const T*>(p.gate) + row[k] * p.gate_stride + at[k] + c);
      }
    }
  }
  const float inv = 1.f / static_cast<float>(p.dim);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float u[NV][8], mean = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xw[k][v].floats(u[v]);
      if (kGate && p.gate_first) {
        float z[8];
        zw[k][v].floats(z);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] *= silu(z[i]);
      }
    }
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
      if ((v * L + lane) * 8 < p.dim)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[0] = fmaf(u[v][i] - mean, u[v][i] - mean, q[0]);
    group_sum<L>(q, buf, turn);
    const float r = rsqrtf(q[0] * inv + p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      if (first + k * SLOTS >= items || c >= p.dim) continue;
      float w[8], b[8];
      weights8(p.weight, c, 1.f, w);
      weights8(p.bias, c, 0.f, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] = fmaf((u[v][i] - mean) * r, w[i], b[i]);
      if (kGate && !p.gate_first) {
        float z[8];
        zw[k][v].floats(z);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] *= silu(z[i]);
      }
      store8(static_cast<T*>(p.out) + row[k] * p.out_stride + at[k] + c, u[v]);
    }
  }
}

// ---- backward ------------------------------------------------------------------------
// A lane's columns: their weights (and biases, for a gate behind them), and the sums for both.
template <int NV, bool kGate>
struct NormColumns {
  Pair w[NV][4], b[kGate ? NV : 1][4], dw[NV][4], db[NV][4];
  __device__ __forceinline__ void start(const LayerNormParams& p, int lane, int lanes) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * lanes + lane) * 8;
      float f[8] = {}, g[8] = {};
      if (c < p.dim) {
        weights8(p.weight, c, 1.f, f);
        weights8(p.bias, c, 0.f, g);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[v][i] = pair_of(f[2 * i], f[2 * i + 1]);
        if (kGate) b[v][i] = pair_of(g[2 * i], g[2 * i + 1]);
        dw[v][i] = db[v][i] = 0;
      }
    }
  }
};

// One group's gradients, in the L lanes' words (zeros past its end); its columns' sums go to `cols`. `read` runs once every
// lane has its words (and its group's lanes have met, where the group is a CTA's). In pairs of fp32, and with the columns'
// weights in registers: what bounds it is the issue of instructions (430 a warp and row without either: 264 us for 32768 rows of
// 4096 in bf16).
template <typename T, int L, int NV, bool kGate, typename Read>
__device__ __forceinline__ void norm_backward(const LayerNormParams& p, const Eight<T> (&xw)[NV], const Eight<T> (&gw)[NV],
                                              const Eight<T> (&zw)[kGate ? NV : 1], int lane, bool real, int64_t row, int64_t at,
                                              NormColumns<NV, kGate>& cols, float* buf, int& turn, Read&& read) {
  const float inv = 1.f / static_cast<float>(p.dim);
  const bool after = kGate && !p.gate_first;
  Pair u[NV][4], g[NV][4];  // g: dL/dy, before the weight
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    pairs8<T>(xw[v], u[v]);
    pairs8<T>(gw[v], g[v]);
    if constexpr (kGate) {
      float z[8];
      zw[v].floats(z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair s = pair_of(silu(z[2 * i]), silu(z[2 * i + 1]));
        if (after) g[v][i] = mul2(g[v][i], s);
        else u[v][i] = mul2(u[v][i], s);
      }
    }
  }
  float sums[2], mt = 0.f;
  if (!p.rms) {
    Pair a = 0, t = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a = add2(a, u[v][i]);
        t = fma2(g[v][i], cols.w[v][i], t);
      }
    sums[0] = sum_of(a);
    sums[1] = sum_of(t);
    group_sum<L>(sums, buf, turn);
    mt = sums[1] * inv;
    const Pair mean = both(-sums[0] * inv);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if ((v * L + lane) * 8 < p.dim)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[v][i] = add2(u[v][i], mean);
  }
  Pair q = 0, c = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q = fma2(u[v][i], u[v][i], q);
      c = fma2(mul2(g[v][i], cols.w[v][i]), u[v][i], c);
    }
  sums[0] = sum_of(q);
  sums[1] = sum_of(c);
  group_sum<L>(sums, buf, turn);
  read();
  const float r = rsqrtf(sums[0] * inv + p.eps);
  const Pair r2 = both(r), by_h = both(-sums[1] * inv * r * r), by_1 = both(-mt * r);  // dx = r t - r mt - r mth h, mth = sum t u r / n
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at_c = (v * L + lane) * 8;
    if (!real || at_c >= p.dim) continue;
    Pair d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[v][i] = mul2(u[v][i], r2);  // h
      cols.dw[v][i] = fma2(g[v][i], u[v][i], cols.dw[v][i]);
      cols.db[v][i] = add2(cols.db[v][i], g[v][i]);
      d[i] = fma2(u[v][i], by_h, fma2(mul2(g[v][i], cols.w[v][i]), r2, by_1));
    }
    float dx[8];
    values8(d, dx);
    if constexpr (kGate) {
      float z[8], o[8], y[8], dz[8];
      zw[v].floats(z);
      if (after) {
        gw[v].floats(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) parts_of(fma2(u[v][i], cols.w[v][i], cols.b[v][i]), y[2 * i], y[2 * i + 1]);
      } else {
        xw[v].floats(o);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sg = sigmoid(z[i]), s = z[i] * sg, slope = fmaf(s, 1.f - sg, sg);
        dz[i] = o[i] * slope * (after ? y[i] : dx[i]);
        if (!after) dx[i] *= s;
      }
      store8(static_cast<T*>(p.dgate) + row * p.dgate_stride + at + at_c, dz);
    }
    store8(static_cast<T*>(p.out) + row * p.out_stride + at + at_c, dx);
  }
}

// Groups of up to 256, as they lie in a warp: a fixed grid; a slot of L lanes walks every (grid x slots)-th group, the next one's words under way.
constexpr int kNormSmallCtas = 6;  // an SM

template <typename T, int L, bool kGate>
__global__ void __launch_bounds__(128, kGate ? 4 : kNormSmallCtas) gdn_layer_norm_bwd_kernel(const LayerNormParams p) {
  constexpr int SLOTS = 128 / L;
  __shared__ float s_sum[SLOTS * L * 8];
  int turn = 0;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L, c = lane * 8;
  const uint32_t step = gridDim.x * SLOTS, groups = static_cast<uint32_t>(p.groups), items = static_cast<uint32_t>(p.items);
  tc::grid_dependency_wait();
  NormColumns<1, kGate> cols;
  cols.start(p, lane, L);
  Eight<T> xw[1], gw[1], zw[1];
  uint32_t item = blockIdx.x * SLOTS + slot, row = item / groups, at = (item - row * groups) * p.dim;
  auto fetch = [&] {
    xw[0].zero();
    gw[0].zero();
    zw[0].zero();
    if (item < items && c < p.dim) {
      xw[0].load(static_cast<const T*>(p.x) + row * p.x_stride + at + c);
      gw[0].load(static_cast<const T*>(p.dout) + row * p.dout_stride + at + c);
      if (kGate) zw[0].load(static_cast<const T*>(p.gate) + row * p.gate_stride + at + c);
    }
  };
  fetch();
  // every slot of the CTA takes as many steps, for the shuffles among them
  for (uint32_t first = blockIdx.x * SLOTS; first < items; first += step) {
    const Eight<T> xc[1] = {xw[0]}, gc[1] = {gw[0]}, zc[1] = {zw[0]};
    const uint32_t now_row = row, now_at = at;
    const bool real = item < items;
    item += step;
    row = item / groups;
    at = (item - row * groups) * p.dim;
    fetch();
    norm_backward<T, L, 1, kGate>(p, xc, gc, zc, lane, real, now_row, now_at, cols, nullptr, turn, [] {});
  }
  if (!p.partials) return;
  // the CTA's sums, slot after slot
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
    float f[8];
    values8(k ? cols.db[0] : cols.dw[0], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[slot * L * 8 + c + i] = f[i];
    __syncthreads();
    for (int i = threadIdx.x; i < p.dim; i += 128) {
      float acc = 0.f;
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) acc += s_sum[j * L * 8 + i];
      out[k * p.dim + i] = acc;
    }
  }
}

// Wider groups: a CTA of L threads has a group, and copies those to come into a ring of `stages` rows. 32768 rows of 4096 in bf16
// with 256 threads and two words each: 145 us, 5.54 TB/s (82% of the measured copy rate); it issues in 54% of the slots and waits for
// shared memory and the group's sums between.
// CTAs of an SM.
template <int L, bool kGate>
constexpr int norm_wide_ctas = L == 128 ? (kGate ? 4 : 6) : L == 256 ? 2 : 1;

template <typename T, int L, int NV, bool kGate>
__global__ void __launch_bounds__(L, norm_wide_ctas<L, kGate>) gdn_layer_norm_bwd_wide_kernel(const LayerNormParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t s_full[8];
  __shared__ __align__(16) float buf[128];
  __shared__ uint32_t s_abort;
  constexpr int ARRAYS = kGate ? 3 : 2;
  const int lane = threadIdx.x;
  const uint32_t groups = static_cast<uint32_t>(p.groups), items = static_cast<uint32_t>(p.items), step = gridDim.x;
  const uint32_t bytes = p.dim * static_cast<uint32_t>(sizeof(T)), bars = tc::smem_u32(s_full), base = tc::smem_u32(ring);
  int turn = 0;
  tc::grid_dependency_wait();
  auto copy = [&](uint32_t item, int stage) {
    const uint32_t row = item / groups, at = (item - row * groups) * p.dim, to = base + stage * ARRAYS * bytes, bar = bars + 8 * stage;
    tc::mbar_arrive_expect_tx(bar, ARRAYS * bytes);
    tc::bulk_load(to, static_cast<const T*>(p.x) + row * p.x_stride + at, bytes, bar);
    tc::bulk_load(to + bytes, static_cast<const T*>(p.dout) + row * p.dout_stride + at, bytes, bar);
    if (kGate) tc::bulk_load(to + 2 * bytes, static_cast<const T*>(p.gate) + row * p.gate_stride + at, bytes, bar);
  };
  if (lane == 0) {
    s_abort = 0;
    for (int i = 0; i < p.stages; ++i) tc::mbar_init(bars + 8 * i, 1);
    tc::mbar_fence_init();
    for (int i = 0; i < p.stages; ++i)
      if (blockIdx.x + static_cast<uint64_t>(i) * step < items) copy(blockIdx.x + i * step, i);
  }
  __syncthreads();
  NormColumns<NV, kGate> cols;
  cols.start(p, lane, L);
  int stage = 0;
  uint32_t phase = 0;
  for (uint32_t item = blockIdx.x; item < items; item += step) {
    const uint32_t row = item / groups, at = (item - row * groups) * p.dim;
    bool there = tc::mbar_try_wait(bars + 8 * stage, phase);
    for (int k = 0; k < (1 << 18) && !there && !*static_cast<volatile uint32_t*>(&s_abort); ++k) there = tc::mbar_try_wait_hint(bars + 8 * stage, phase, 10000u);
    if (!there) {  // walks on with what there is, so that the barriers fill
      s_abort = 1;
      atomicOr(p.status, kStatusTimeout);
    }
    Eight<T> xw[NV], gw[NV], zw[kGate ? NV : 1];
    const T* from = reinterpret_cast<const T*>(ring + stage * ARRAYS * bytes);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * L + lane) * 8;
      xw[v].zero();
      gw[v].zero();
      if (kGate) zw[v].zero();
      if (c < p.dim) {
        xw[v].load(from + c);
        gw[v].load(from + p.dim + c);
        if (kGate) zw[v].load(from + 2 * p.dim + c);
      }
    }
    norm_backward<T, L, NV, kGate>(p, xw, gw, zw, lane, true, row, at, cols, buf, turn, [&] {
      const uint64_t next = item + static_cast<uint64_t>(p.stages) * step;
      if (lane == 0 && next < items) copy(static_cast<uint32_t>(next), stage);
    });
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  __syncthreads();
  if (s_abort) {  // copies in flight land before the ring is given up
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (!p.partials) return;
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * L + lane) * 8;
    if (c >= p.dim) continue;
    float f[8];
    values8(cols.dw[v], f);
    store8(out + c, f);
    values8(cols.db[v], f);
    store8(out + p.dim + c, f);
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
