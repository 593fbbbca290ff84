// The short causal convolution of every channel with its silu, its backward, and the rows that a
// sequence carries to its next call, for sm_103a.
//
//     y[t] = b + sum_j w[j] x[t - (W - 1) + j],   out = silu(y)          (every channel by itself)
//
// with the W - 1 inputs before a sequence's first from its state (or zeros). Backward, given dout:
//
//     dy = dout silu'(y);   dx[t] = sum_j w[j] dy[t + (W - 1) - j];   dw[j] = sum_t dy[t] x[t - (W - 1) + j];   db = sum_t dy[t]
//
// Bound by HBM: 4 bytes a value in 16-bit types (6 backward) against 2 W + 10 operations, two of
// them on the special function unit. A thread owns 16 bytes of a row and walks a strip of rows with
// the last W - 1 inputs and the weights in registers, so that an input is loaded once (and the W - 1
// rows before a strip again, from L2). 59010 ragged rows of 8192 channels in bf16: 300 us, 6.45 TB/s (95%
// of the measured copy rate); 448 before strips, ring and weights were as they are.
#pragma once
#include "gdn_row_common.cuh"

namespace gdn {

constexpr int kConvThreads = 128;
constexpr int kConvCtasPerSm = 4;
// A thread's words of the rows to come lie in a ring in shared memory, kConvAhead steps of conv_step rows (cp.async): in registers there
// is no room for as many as HBM's latency asks for (25% occupancy and a step ahead: 69% of the measured rate forward, 70% backward).
// A step is a multiple of W - 1 rows, after which the window of inputs is in the registers it was in.
template <int W>
constexpr int conv_step = W == 4 ? 6 : 4;
constexpr int kConvAhead = 3;

template <int BYTES>
__device__ __forceinline__ void conv_fetch(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void conv_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct ConvParams {
  const void* x;
  const float* weight;  // [D][W]
  const float* bias;    // [D] or null
  void* state;          // [B][W - 1][D], or pointers to [W - 1][D]; null: zeros before every sequence
  void* out;
  int64_t x_stride, out_stride;
  Rows batch;
  int D, strip, strips;
  int state_is_table;
  int state_here;  // every sequence lies in one strip, whose thread also writes its state
  int silu;
  // backward
  const void* dout;
  void* dx;
  int64_t dout_stride, dx_stride;
  const void* dlast;  // [B][W - 1][D]: dL/d(the state after the call), or null
  void* dfirst;       // [B][W - 1][D]: dL/d(the state before it), or null
  float* dweight;
  float* dbias;
  float* partials;  // [strips][W + 1][D]
  unsigned* status;
};

template <typename T>
__device__ __forceinline__ T* conv_state(void* state, int table, int s, int64_t size) {
  if (!state) return nullptr;
  return table ? static_cast<T* const*>(state)[s] : static_cast<T*>(state) + s * size;
}

// The weights of a thread's 2 P channels, tap by tap, in pairs (c0 is a multiple of 4: their W x 2 P values are whole words).
template <int W, int P>
__device__ __forceinline__ void conv_weights(const ConvParams& p, int c0, Pair (&w)[W][P], Pair (&b)[P]) {
  float f[2 * P * W], g[2 * P];
#pragma unroll
  for (int i = 0; i < 2 * P * W; i += 4) load4(p.weight + static_cast<int64_t>(c0) * W + i, *reinterpret_cast<float(*)[4]>(f + i));
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) g[i] = 0.f;
  if (p.bias)
#pragma unroll
    for (int i = 0; i < 2 * P; i += 4) load4(p.bias + c0 + i, *reinterpret_cast<float(*)[4]>(g + i));
#pragma unroll
  for (int i = 0; i < P; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = pair_of(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
    b[i] = pair_of(g[2 * i], g[2 * i + 1]);
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kConvThreads, kConvCtasPerSm) gdn_conv_kernel(const ConvParams p) {
  constexpr int N = Word16<T>::N, P = Word16<T>::PAIRS, U = conv_step<W>, A = kConvAhead;
  __shared__ uint4 ring[A * U][kConvThreads];
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  tc::grid_dependency_wait();
  for (int64_t s = item; s < p.batch.B; s += static_cast<int64_t>(gridDim.x) * kConvThreads) p.batch.report(static_cast<int>(s), p.status);
  const int words = p.D / N;
  const int strip = static_cast<int>(item / words);
  if (strip >= p.strips) return;
  const int c0 = static_cast<int>(item - static_cast<int64_t>(strip) * words) * N;
  const T* x = static_cast<const T*>(p.x) + c0;
  T* out = static_cast<T*>(p.out) + c0;
  int row = strip * p.strip;
  const int stop = min(row + p.strip, p.batch.rows);
  Pair w[W][P], b[P];
  conv_weights<W, P>(p, c0, w, b);
  for (int s = p.batch.find(row); row < stop && s < p.batch.B; ++s) {
    const int start = p.batch.start(s), end = p.batch.end(s);
    if (end <= row || start >= stop || !rows_held(start, end, p.batch.rows)) continue;
    row = max(row, start);  // behind rows of refused sequences
    T* state = conv_state<T>(p.state, p.state_is_table, s, static_cast<int64_t>(W - 1) * p.D);
    if (state) state += c0;
    uint4 last[W - 1];  // the inputs before
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const int t = row - (W - 1) + i;
      last[i] = make_uint4(0, 0, 0, 0);
      if (t >= start) last[i] = *reinterpret_cast<const uint4*>(x + t * p.x_stride);
      else if (state) last[i] = *reinterpret_cast<const uint4*>(state + static_cast<int64_t>(t - start + W - 1) * p.D);
    }
    const int to = min(end, stop);
    Pair before[W - 1][P];
    // one row: `word` in, out to `at`
    auto step = [&](const uint4 word, T* at) {
      Pair now[P];
      unpack16<T>(word, now);
      float y[N];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        Pair acc = fma2(now[i], w[W - 1][i], b[i]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) acc = fma2(before[j][i], w[j][i], acc);
        parts_of(acc, y[2 * i], y[2 * i + 1]);
      }
      if (p.silu) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = silu(y[i]);
      }
      *reinterpret_cast<uint4*>(at) = pack16<T>(y);
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) before[j][i] = before[j + 1][i];
#pragma unroll
      for (int i = 0; i < P; ++i) before[W - 2][i] = now[i];
    };
#pragma unroll
    for (int i = 0; i < W - 1; ++i) unpack16<T>(last[i], before[i]);
    const T* from = x + row * p.x_stride;
    T* at = out + row * p.out_stride;
    uint4* mine = &ring[0][threadIdx.x];
    const uint32_t slots = tc::smem_u32(mine);
    auto fetch = [&](int k, int left) {  // step k from here, of `left` rows
      if (left > 0)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < left) conv_fetch<16>(slots + (k % A * U + u) * (kConvThreads * 16), from + (k * U + u) * p.x_stride);
      tc::cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < A - 1; ++k) fetch(k, to - row - k * U);
    for (int k = 0; row < to; row += U, ++k) {
      fetch(k + A - 1, to - row - (A - 1) * U);
      conv_wait<A - 1>();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (row + u < to) step(mine[(k % A * U + u) * kConvThreads], at + (k * U + u) * p.out_stride);
    }
    row = to;
    if (p.state_here && state) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        float f[N];
#pragma unroll
        for (int i = 0; i < P; ++i) parts_of(before[j][i], f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4*>(state + static_cast<int64_t>(j) * p.D) = pack16<T>(f);
      }
    }
  }
}

// The state of every sequence after the call: the last W - 1 of its old state's rows and its inputs.
// By itself, after the convolution, because the strip at a sequence's start reads what the one at its
// end would overwrite.
template <typename T, int W>
__global__ void __launch_bounds__(kConvThreads) gdn_conv_state_kernel(const ConvParams p) {
  constexpr int N = Word16<T>::N;
  tc::grid_dependency_wait();
  const int words = p.D / N;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int s = static_cast<int>(item / words);
  if (s >= p.batch.B) return;
  const int c0 = static_cast<int>(item - static_cast<int64_t>(s) * words) * N;
  const int start = p.batch.start(s), end = p.batch.end(s);
  if (!rows_held(start, end, p.batch.rows) || start == end) return;
  const T* x = static_cast<const T*>(p.x) + c0;
  T* state = conv_state<T>(p.state, p.state_is_table, s, static_cast<int64_t>(W - 1) * p.D) + c0;
  uint4 v[W - 1];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int t = end - (W - 1) + i;
    v[i] = t >= start ? *reinterpret_cast<const uint4*>(x + t * p.x_stride)
                      : *reinterpret_cast<const uint4*>(state + static_cast<int64_t>(t - start + W - 1) * p.D);
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) *reinterpret_cast<uint4*>(state + static_cast<int64_t>(i) * p.D) = v[i];
}

// ---- backward ------------------------------------------------------------------------
// dy of one row of four channels: y from the inputs before[0..W-2] and now.
template <int W>
__device__ __forceinline__ void conv_dy(const Pair (&w)[W][2], const Pair (&b)[2], const Pair (&before)[W - 1][2], const Pair (&now)[2],
                                        const float (&g)[4], int with_silu, Pair (&dy)[2]) {
  const Pair one = pair_of(1.f, 1.f), minus = pair_of(-1.f, -1.f), to_log2 = pair_of(-1.4426950408889634f, -1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    dy[i] = pair_of(g[2 * i], g[2 * i + 1]);
    if (!with_silu) continue;
    Pair y = fma2(now[i], w[W - 1][i], b[i]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) y = fma2(before[j][i], w[j][i], y);
    // s = 1 / (1 + e^-y); silu' = s (1 + y (1 - s))
    float e[2], s[2];
    parts_of(mul2(y, to_log2), e[0], e[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e[k]));
    parts_of(add2(pair_of(e[0], e[1]), one), s[0], s[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[k]));
    const Pair sg = pair_of(s[0], s[1]);
    dy[i] = mul2(dy[i], mul2(sg, fma2(y, fma2(sg, minus, one), one)));
  }
}

// A thread owns four channels and a strip of rows; it walks W - 1 rows past the strip's end, whose dy
// the last gradients need, and keeps the weight gradients of its own rows. (Eight channels would need twice its 128 registers.)
// 32768 rows of 8192 in bf16: 282 us, 5.71 TB/s, 84% of the measured copy rate. It issues in 55% of the slots, its fp32 pipe is at
// half, with 14 warps an SM: what is left is the arithmetic. Addresses by products of row and stride cost another 14 us.
template <typename T, int W>
__global__ void __launch_bounds__(kConvThreads, sizeof(T) == 4 ? 3 : 4) gdn_conv_bwd_kernel(const ConvParams p) {
  using Word = typename Four<T>::Word;
  constexpr int U = conv_step<W>, A = sizeof(T) == 4 ? 2 : kConvAhead;
  __shared__ Word ring[A * U][2][kConvThreads];
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  tc::grid_dependency_wait();
  for (int64_t s = item; s < p.batch.B; s += static_cast<int64_t>(gridDim.x) * kConvThreads) p.batch.report(static_cast<int>(s), p.status);
  const int words = p.D / 4;
  const int strip = static_cast<int>(item / words);
  if (strip >= p.strips) return;
  const int c0 = static_cast<int>(item - static_cast<int64_t>(strip) * words) * 4;
  const T* x = static_cast<const T*>(p.x) + c0;
  const T* dout = static_cast<const T*>(p.dout) + c0;
  T* dx = static_cast<T*>(p.dx) + c0;
  int row = strip * p.strip;
  const int stop = min(row + p.strip, p.batch.rows);
  Pair w[W][2], b[2];
  conv_weights<W, 2>(p, c0, w, b);
  const Pair zero = pair_of(0.f, 0.f);
  Pair dw[W][2], db[2] = {zero, zero};
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j][0] = dw[j][1] = zero;
  for (int s = p.batch.find(row); row < stop && s < p.batch.B; ++s) {
    const int start = p.batch.start(s), end = p.batch.end(s);
    if (end <= row || start >= stop || !rows_held(start, end, p.batch.rows)) continue;
    row = max(row, start);  // behind rows of refused sequences
    const int64_t size = static_cast<int64_t>(W - 1) * p.D;
    const T* state = conv_state<const T>(p.state, 0, s, size);
    const T* dlast = p.dlast ? static_cast<const T*>(p.dlast) + s * size + c0 : nullptr;
    const int first = row, own = min(end, stop), to = min(end, stop + W - 1);
    Pair before[W - 1][2], past[W - 1][2];  // inputs, and dy, of the rows before `row`
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const int t = row - (W - 1) + i;
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (t >= start) load4(x + t * p.x_stride, f);
      else if (state) load4(state + static_cast<int64_t>(t - start + W - 1) * p.D + c0, f);
      before[i][0] = pair_of(f[0], f[1]);
      before[i][1] = pair_of(f[2], f[3]);
      past[i][0] = past[i][1] = zero;
    }
    // the gradient of the row W - 1 before that of dy: dy[at + (W - 1) - j] takes w[j]
    auto gradient = [&](const Pair (&dy)[2], float (&f)[4]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Pair acc = mul2(dy[i], w[0][i]);
#pragma unroll
        for (int j = 1; j < W; ++j) acc = fma2(past[W - 1 - j][i], w[j][i], acc);
        parts_of(acc, f[2 * i], f[2 * i + 1]);
      }
    };
    auto put = [&](int t, const Pair (&dy)[2]) {
      const int at = t - (W - 1);
      if (at < first || at >= own) return;
      float f[4];
      gradient(dy, f);
      if (dlast && at >= end - (W - 1)) {
        float e[4];
        load4(dlast + static_cast<int64_t>(at - (end - (W - 1))) * p.D, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += e[i];
      }
      store4(dx + at * p.dx_stride, f);
    };
    auto push = [&](const Pair (&dy)[2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) past[j][i] = past[j + 1][i];
        past[W - 2][i] = dy[i];
      }
    };
    // one row: its words in; `own_row` whether it is of the strip itself, `at` where the gradient of the row W - 1 before goes
    auto step = [&](const Word& xw, const Word& gw, bool own_row, auto&& give) {
      float f[4], g[4];
      unpack4<T>(xw, f);
      unpack4<T>(gw, g);
      const Pair now[2] = {pair_of(f[0], f[1]), pair_of(f[2], f[3])};
      Pair dy[2];
      conv_dy<W>(w, b, before, now, g, p.silu, dy);
      if (own_row) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][i] = fma2(dy[i], before[j][i], dw[j][i]);
          dw[W - 1][i] = fma2(dy[i], now[i], dw[W - 1][i]);
          db[i] = add2(db[i], dy[i]);
        }
      }
      give(dy);
      push(dy);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) before[j][i] = before[j + 1][i];
        before[W - 2][i] = now[i];
      }
    };
    const T *fx = x + row * p.x_stride, *fg = dout + row * p.dout_stride;  // of the row that is fetched next
    T* to_dx = dx + (row - (W - 1)) * p.dx_stride;
    Word* mine = &ring[0][0][threadIdx.x];
    constexpr int BYTES = sizeof(Word), ROW = 2 * kConvThreads;
    const uint32_t slots = tc::smem_u32(mine), after = slots + A * U * ROW * BYTES;
    uint32_t slot = slots;
    auto fetch = [&](int left) {  // a step, of `left` rows
      auto one = [&](int u) {
        conv_fetch<BYTES>(slot + u * (ROW * BYTES), fx);
        conv_fetch<BYTES>(slot + u * (ROW * BYTES) + kConvThreads * BYTES, fg);
        fx += p.x_stride;
        fg += p.dout_stride;
      };
      if (left >= U) {
#pragma unroll
        for (int u = 0; u < U; ++u) one(u);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < left) one(u);
      }
      slot = slot + U * ROW * BYTES == after ? slots : slot + U * ROW * BYTES;
      tc::cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < A - 1; ++k) fetch(to - row - k * U);
    for (const Word* now = mine; row < to; row += U) {
      fetch(to - row - (A - 1) * U);
      conv_wait<A - 1>();
      if (row >= first + W - 1 && row + U <= own) {  // inside the strip: no ends to look for
#pragma unroll
        for (int u = 0; u < U; ++u)
          step(now[u * ROW], now[u * ROW + kConvThreads], true, [&](const Pair (&dy)[2]) {
            float f[4];
            gradient(dy, f);
            store4(to_dx, f);
            to_dx += p.dx_stride;
          });
      } else {
#pragma unroll 1
        for (int u = 0; u < U && row + u < to; ++u)
          step(now[u * ROW], now[u * ROW + kConvThreads], row + u < own, [&](const Pair (&dy)[2]) { put(row + u, dy); });
        to_dx += U * p.dx_stride;
      }
      now = now + U * ROW == mine + A * U * ROW ? mine : now + U * ROW;
    }
    row = to;
    if (to == end) {  // nothing comes after the sequence's end
      const Pair none[2] = {zero, zero};
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        put(to + i, none);
        push(none);
      }
    }
    row = own;
  }
  if (p.partials) {
    float* out = p.partials + static_cast<int64_t>(strip) * (W + 1) * p.D + c0;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      const Pair* d = j < W ? dw[j] : db;
      float f[4];
      parts_of(d[0], f[0], f[1]);
      parts_of(d[1], f[2], f[3]);
      store4(out + static_cast<int64_t>(j) * p.D, f);
    }
  }
}

constexpr int kConvSumThreads = 1024;

// What the strips leave over: the first sum_ctas CTAs add up the weight gradients, the others work out
// the gradient of the carried-in states, from the first W - 1 rows of every sequence:
//     dfirst[i] = sum_{j <= i} w[j] dy[i - j], and dlast[i - length] where the sequence is that short
template <typename T, int W>
__global__ void __launch_bounds__(kConvSumThreads) gdn_conv_bwd_ends_kernel(const ConvParams p, int sum_ctas) {
  tc::grid_dependency_wait();
  if (static_cast<int>(blockIdx.x) < sum_ctas) {
    sum_columns(p.partials, p.strips, (W + 1) * p.D, static_cast<int>(blockIdx.x) * 32, [&](int c, float v) {
      const int j = c / p.D, d = c - j * p.D;
      if (j < W) {
        if (p.dweight) p.dweight[static_cast<int64_t>(d) * W + j] = v;
      } else if (p.dbias) {
        p.dbias[d] = v;
      }
    });
    return;
  }
  const int words = p.D / 4;
  const int64_t item = static_cast<int64_t>(blockIdx.x - sum_ctas) * kConvSumThreads + threadIdx.x;
  const int s = static_cast<int>(item / words);
  if (s >= p.batch.B) return;
  const int c0 = static_cast<int>(item - static_cast<int64_t>(s) * words) * 4;
  const int start = p.batch.start(s), end = p.batch.end(s);
  if (!rows_held(start, end, p.batch.rows)) return;
  const int64_t size = static_cast<int64_t>(W - 1) * p.D;
  const T* state = p.state ? static_cast<const T*>(p.state) + s * size + c0 : nullptr;
  const T* dlast = p.dlast ? static_cast<const T*>(p.dlast) + s * size + c0 : nullptr;
  Pair w[W][2], b[2];
  conv_weights<W, 2>(p, c0, w, b);
  const Pair zero = pair_of(0.f, 0.f);
  Pair before[W - 1][2], dy[W - 1][2];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (state) load4(state + static_cast<int64_t>(i) * p.D, f);
    before[i][0] = pair_of(f[0], f[1]);
    before[i][1] = pair_of(f[2], f[3]);
  }
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    dy[t][0] = dy[t][1] = zero;
    if (start + t < end) {
      float f[4], g[4];
      load4(static_cast<const T*>(p.x) + (start + t) * p.x_stride + c0, f);
      load4(static_cast<const T*>(p.dout) + (start + t) * p.dout_stride + c0, g);
      const Pair now[2] = {pair_of(f[0], f[1]), pair_of(f[2], f[3])};
      conv_dy<W>(w, b, before, now, g, p.silu, dy[t]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) before[j][i] = before[j + 1][i];
        before[W - 2][i] = now[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    Pair acc[2] = {zero, zero};
#pragma unroll
    for (int j = 0; j <= i; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) acc[e] = fma2(dy[i - j][e], w[j][e], acc[e]);
    float f[4];
    parts_of(acc[0], f[0], f[1]);
    parts_of(acc[1], f[2], f[3]);
    if (dlast && i >= end - start) {
      float e[4];
      load4(dlast + static_cast<int64_t>(i - (end - start)) * p.D, e);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] += e[k];
    }
    store4(static_cast<T*>(p.dfirst) + s * size + static_cast<int64_t>(i) * p.D + c0, f);
  }
}

}  // namespace gdn
