// Shared by the kernels that work on rows of activations (norms, rotation, convolution): words of
// 4 values or 16 bytes of them as fp32 values, paired arithmetic, silu, the sequence that a packed
// row belongs to, and the sum of per-CTA partial columns.
#pragma once
#include "gdn_common.cuh"

namespace gdn {

// ---- four consecutive values of a row -----------------------------------------------
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const __half* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(__half* p, const float (&f)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]));
}

// Four values as they lie in memory (held packed while their load is under way).
template <typename T>
struct Four {
  using Word = uint2;
};
template <>
struct Four<float> {
  using Word = uint4;
};
template <typename T>
__device__ __forceinline__ void unpack4(const typename Four<T>::Word& w, float (&f)[4]) {
  load4(reinterpret_cast<const T*>(&w), f);
}

// Two fp32 values in one register pair, and the paired arithmetic of sm_100 and up.
using Pair = uint64_t;
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void parts_of(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 16 bytes of a row: 8 values of 16 bits or 4 of fp32, as pairs for the paired arithmetic.
template <typename T>
struct Word16 {
  static constexpr int N = 16 / static_cast<int>(sizeof(T)), PAIRS = N / 2;
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 w, Pair (&p)[Word16<T>::PAIRS]);
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 w, Pair (&p)[4]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair_of(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ void unpack16<__half>(const uint4 w, Pair (&p)[4]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
    p[i] = pair_of(f.x, f.y);
  }
}
template <>
__device__ __forceinline__ void unpack16<float>(const uint4 w, Pair (&p)[2]) {
  p[0] = pair_of(__uint_as_float(w.x), __uint_as_float(w.y));
  p[1] = pair_of(__uint_as_float(w.z), __uint_as_float(w.w));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return pack_half2(a, b);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[Word16<T>::N]) {
  if constexpr (sizeof(T) == 4) return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}
template <typename T>
__device__ __forceinline__ void floats16(const uint4 w, float (&f)[Word16<T>::N]) {
  Pair p[Word16<T>::PAIRS];
  unpack16<T>(w, p);
#pragma unroll
  for (int i = 0; i < Word16<T>::PAIRS; ++i) parts_of(p[i], f[2 * i], f[2 * i + 1]);
}

// 32 bytes to global memory: as one sector, or in two halves where dst is only 16-byte aligned.
__device__ __forceinline__ void store32(void* dst, const uint32_t* r, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(dst)), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// 1 / (1 + e^-y), y of it, in two operations of the special function unit: the plain exponential and division cost
// twice the instructions for results in the subnormal range. Where e^-y passes fp32's range they give 0.
__device__ __forceinline__ float sigmoid(float y) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float silu(float y) { return y * sigmoid(y); }

// The packed rows of a batch: sequence s owns rows [start(s), end(s)), from cu_seqlens, or T rows each.
struct Rows {
  const int32_t* cu;
  int B, T, rows;
  __device__ __forceinline__ int start(int s) const { return cu ? cu[s] : s * T; }
  __device__ __forceinline__ int end(int s) const { return cu ? cu[s + 1] : (s + 1) * T; }
  // The last sequence that starts at or before `row` (0 where none does).
  __device__ __forceinline__ int find(int row) const {
    if (!cu) return row / T;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
  // Offsets that do not rise from 0, or pass the rows: found by one thread of the grid for each sequence.
  __device__ __forceinline__ void report(int s, unsigned* status) const {
    if (!cu || s >= B) return;
    const int a = cu[s], b = cu[s + 1];
    if (b < a || b > rows || (s == 0 && a != 0)) atomicOr(status, kStatusBadSeqlens);
  }
};

// Whether a sequence's rows lie inside the buffers.
__device__ __forceinline__ bool rows_held(int start, int end, int rows) { return start >= 0 && start <= end && end <= rows; }

// Adds up columns of partials [parts][cols] in fixed order: 32 columns and 32 runs of parts a CTA.
// Column c goes to out(c).
template <typename Out>
__device__ __forceinline__ void sum_columns(const float* partials, int parts, int cols, int c0, Out&& out) {
  __shared__ float s_sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = c0 + lane;
  float acc = 0.f;
  if (col < cols)
    for (int i = warp; i < parts; i += 32) acc += partials[static_cast<int64_t>(i) * cols + col];
  s_sum[warp][lane] = acc;
  __syncthreads();
  acc = s_sum[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0 && c0 + warp < cols) out(c0 + warp, acc);
}

}  // namespace gdn
