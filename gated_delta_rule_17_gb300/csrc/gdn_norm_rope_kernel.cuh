// RMS norm and rotation of query and key heads, its backward, and the append of
// keys and values to a paged cache, for sm_103a.
//
// For a head row x of d values, with r = 1 / sqrt(mean(x^2) + eps) and weights w,
//
//     z = x r w;   y = R z      (R turns the value pairs of the first `rot` values)
//
// and backward, given dy:
//
//     dz = R^T dy;  dw = sum dz x r;  t = dz w;  dx = r (t - x r^2 mean(t x))
//
// All of it is bound by HBM: ~10 (20) flops a value against 4 (6) bytes in 16-bit
// types. So each head row is read once and stays in registers: d / 8 lanes hold it,
// eight values each, and the two values of a pair sit in the same lane, so the
// rotation needs no exchange; only the row sums go over the lanes. A lane's eight
// values are two runs of four: values 4l and 4l + rot/2 for pairs half a rotation
// apart, 8l and 8l + 4 for neighbouring pairs and for values past `rot`. A warp takes up to
// kNormUnroll x (32 lanes / lanes a row) heads of one token, all loads first, with the
// products of weight and cosine or sine in registers for all of them. At 4 x 8192 tokens
// of 32 + 8 heads of 128, bf16: forward 106 us (6.5 TB/s, 95% of the measured copy
// rate), backward 173 us (5.9 TB/s, 87%); the append of 8 prompts of 100 to 16000 tokens,
// 8 kv heads: 92 us (6.6 TB/s, 97%).
#pragma once
#include "gdn_row_common.cuh"

namespace gdn {

constexpr unsigned kStatusBadPosition = 8u;  // a rotation position outside the table
constexpr unsigned kStatusBadPage = 16u;     // a page number or token index outside the cache or table

constexpr int kNormThreads = 128;
// Registers for 40 warps an SM keep enough loads under way (fp32 words take twice the room: 20).
template <typename T>
constexpr int kNormCtasPerSm = sizeof(T) == 4 ? 5 : 10;
constexpr int kAppendCtasPerSm = 9;
// Head rows a lane group of a warp: four, or two or one for tokens of so few heads that the rest would
// idle (append of 94 sequences of 258 to 516 tokens with one kv head: 40 us with four, 19 with one).
constexpr int kNormUnroll = 4;
constexpr int kNormBwdThreads = 128;
constexpr int kNormBwdCtasPerSm = 6;

struct RopeParams {
  const float* cos;
  const float* sin;
  int64_t stride;
  int positions;
  int rot;  // 0: no rotation
};

// A lane's part of a head row: its two runs of four values and its four pairs' angles.
template <int D, bool kNext>
struct HeadLane {
  int a, b;  // first value of each run
  int pair;  // index of the first of its four pairs
  bool turned;
  __device__ __forceinline__ HeadLane(int l, int rot) {
    turned = 8 * l < rot;
    pair = 4 * l;
    a = (!kNext && turned) ? 4 * l : 8 * l;
    b = (!kNext && turned) ? 4 * l + rot / 2 : 8 * l + 4;
  }
  // The angles of the lane's pairs at position `pos` (cos 1, sin 0 where not turned).
  __device__ __forceinline__ void angles(const RopeParams& r, int64_t pos, float (&c)[4], float (&s)[4]) const {
    if (turned) {
      load4(r.cos + pos * r.stride + pair, c);
      load4(r.sin + pos * r.stride + pair, s);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
  }
  // Regroups the two runs as pairs (u, v), and back.
  __device__ __forceinline__ static void to_pairs(const float (&xa)[4], const float (&xb)[4], float (&u)[4],
                                                  float (&v)[4]) {
    if (kNext) {
      u[0] = xa[0]; v[0] = xa[1]; u[1] = xa[2]; v[1] = xa[3];
      u[2] = xb[0]; v[2] = xb[1]; u[3] = xb[2]; v[3] = xb[3];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = xa[i];
        v[i] = xb[i];
      }
    }
  }
  __device__ __forceinline__ static void from_pairs(const float (&u)[4], const float (&v)[4], float (&xa)[4],
                                                    float (&xb)[4]) {
    if (kNext) {
      xa[0] = u[0]; xa[1] = v[0]; xa[2] = u[1]; xa[3] = v[1];
      xb[0] = u[2]; xb[1] = v[2]; xb[2] = u[3]; xb[3] = v[3];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xa[i] = u[i];
        xb[i] = v[i];
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, float (&u)[4], float (&v)[4]) const {
    float xa[4], xb[4];
    load4(row + a, xa);
    load4(row + b, xb);
    to_pairs(xa, xb, u, v);
  }
  // The same in two steps: the words, and the pairs in them.
  template <typename T>
  __device__ __forceinline__ void fetch(const T* row, bool real, typename Four<T>::Word (&w)[2]) const {
    w[0] = w[1] = typename Four<T>::Word{};
    if (real) {
      w[0] = *reinterpret_cast<const typename Four<T>::Word*>(row + a);
      w[1] = *reinterpret_cast<const typename Four<T>::Word*>(row + b);
    }
  }
  template <typename T>
  __device__ __forceinline__ void pairs(const typename Four<T>::Word (&w)[2], float (&u)[4], float (&v)[4]) const {
    float xa[4], xb[4];
    unpack4<T>(w[0], xa);
    unpack4<T>(w[1], xb);
    to_pairs(xa, xb, u, v);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, const float (&u)[4], const float (&v)[4]) const {
    float xa[4], xb[4];
    from_pairs(u, v, xa, xb);
    store4(row + a, xa);
    store4(row + b, xb);
  }
  __device__ __forceinline__ void weights(const float* w, float (&u)[4], float (&v)[4]) const {
    if (w) {
      load(w, u, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = v[i] = 1.f;
    }
  }
};

// 16 bytes to shared memory, or zeros; and through L1, for what several warps read.
__device__ __forceinline__ void cp_async_16(uint32_t dst_saddr, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_saddr), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_16_ca(uint32_t dst_saddr, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst_saddr), "l"(src) : "memory");
}

// Sum over the LPH lanes that hold one head row.
template <int LPH>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The words of up to U x SLOTS heads of one token row (head h at h * src_head): the first
// loads of a warp, before it looks up where and how far to turn them.
template <typename T, int D, bool kNext, int U>
__device__ __forceinline__ void fetch_heads(const T* src, int64_t src_head, int h0, int heads, int rot,
                                            typename Four<T>::Word (&x)[U][2]) {
  constexpr int LPH = D / 8, SLOTS = 32 / LPH;
  const int lane = threadIdx.x & 31, slot = lane / LPH;
  const HeadLane<D, kNext> hl(lane % LPH, rot);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * SLOTS + slot;
    hl.fetch(src + h * src_head, h < heads, x[i]);
  }
}

// Norms (where `normed`) and rotates them, and writes them to `dst` (head h at h * dst_head).
template <typename T, int D, bool kNext, int U>
__device__ __forceinline__ void norm_rope_heads(const typename Four<T>::Word (&x)[U][2], T* dst, int64_t dst_head,
                                                int h0, int heads, const float* weight, bool normed, float eps,
                                                const RopeParams& rope, int64_t pos) {
  constexpr int LPH = D / 8, SLOTS = 32 / LPH;
  const int lane = threadIdx.x & 31, l = lane % LPH, slot = lane / LPH;
  const HeadLane<D, kNext> hl(l, rope.rot);
  float c[4], s[4], wu[4], wv[4];
  hl.angles(rope, pos, c, s);
  hl.weights(weight, wu, wv);
  float uc[4], us[4], vc[4], vs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uc[j] = wu[j] * c[j];
    us[j] = wu[j] * s[j];
    vc[j] = wv[j] * c[j];
    vs[j] = wv[j] * s[j];
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * SLOTS + slot;
    float u[4], v[4], r = 1.f;
    hl.template pairs<T>(x[i], u, v);
    if (normed) {  // the same for the whole warp
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) q = fmaf(u[j], u[j], fmaf(v[j], v[j], q));
      r = rsqrtf(row_sum<LPH>(q) * (1.f / D) + eps);
    }
    float yu[4], yv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      yu[j] = r * (u[j] * uc[j] - v[j] * vs[j]);
      yv[j] = r * (v[j] * vc[j] + u[j] * us[j]);
    }
    if (h < heads) hl.store(dst + h * dst_head, yu, yv);
  }
}

struct NormRopeParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* q_grad;  // backward
  const void* k_grad;
  const int32_t* positions;
  RopeParams rope;
  const float* q_weight;
  const float* k_weight;
  float* partials;  // backward: [grid][D] sums of the weight gradients, or null
  int q_ctas;       // backward: CTAs for q, and the runs that a token's heads are cut into
  int q_parts, k_parts, q_per, k_per;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride, q_grad_stride, k_grad_stride;
  int rows, nq, nkv;
  int q_chunks, chunks;  // warp items of a token: q_chunks for q's heads, the rest for k's
  float eps;
  unsigned* status;
};

// Whether the table holds a row's position; reports it where not.
__device__ __forceinline__ bool position_held(int64_t pos, const RopeParams& rope, unsigned* status) {
  if (rope.rot == 0 || (pos >= 0 && pos < rope.positions)) return true;
  if ((threadIdx.x & 31) == 0) atomicOr(status, kStatusBadPosition);
  return false;
}

template <typename T, int D, bool kNext, int U>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm<T>) gdn_head_norm_rope_kernel(const NormRopeParams p) {
  constexpr int PER = U * (32 / (D / 8));  // heads of an item
  const unsigned item = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  const unsigned row = item / static_cast<unsigned>(p.chunks);
  if (row >= static_cast<unsigned>(p.rows)) return;
  const int ch = static_cast<int>(item - row * p.chunks);
  const bool is_q = ch < p.q_chunks;
  const int h0 = (is_q ? ch : ch - p.q_chunks) * PER, heads = is_q ? p.nq : p.nkv;
  const int pos = p.rope.rot ? p.positions[row] : 0;
  typename Four<T>::Word x[U][2];
  fetch_heads<T, D, kNext, U>(is_q ? static_cast<const T*>(p.q) + row * p.q_stride : static_cast<const T*>(p.k) + row * p.k_stride,
                           D, h0, heads, p.rope.rot, x);
  if (!position_held(pos, p.rope, p.status)) return;
  norm_rope_heads<T, D, kNext, U>(x, is_q ? static_cast<T*>(p.q_out) + row * p.q_out_stride : static_cast<T*>(p.k_out) + row * p.k_out_stride,
                               D, h0, heads, is_q ? p.q_weight : p.k_weight, true, p.eps, p.rope, pos);
}

// ---- backward ------------------------------------------------------------------------
// A fixed grid, the first q_ctas CTAs for q and the rest for k, so that the weight gradient's sums
// stay in registers. A warp walks its share of (token, run of heads) items, U x SLOTS heads a step,
// and copies x, dy and the angles of the next STAGES - 1 steps into its own ring in shared memory
// (cp.async): with the words in registers instead, the loads under way were too few (294 us for 4 x
// 8192 tokens of 32 + 8 heads) or spilled. What bounds it then is the issue of instructions (two
// thirds of all slots at one head a lane group and step, 216 us), so a step has two heads and the
// arithmetic goes in pairs of fp32. Each CTA adds its warps' sums in a fixed order and writes one
// row of partials.
template <typename T, int D>
struct NormBwdPlan {
  static constexpr int WARPS = kNormBwdThreads / 32, SLOTS = 256 / D, U = sizeof(T) == 4 ? 1 : 2;
  static constexpr int ROW = D * static_cast<int>(sizeof(T));
  static constexpr int HEADS = U * SLOTS * ROW;  // bytes of a step's x or dy
  static constexpr int STEP = 2 * HEADS + 4 * D;  // and its cosines and sines
  static constexpr int STAGES = 3;
  static constexpr int BYTES = WARPS * STAGES * STEP;
};

__device__ __forceinline__ void to_pairs2(const float (&x)[4], Pair (&p)[2]) {
  p[0] = pair_of(x[0], x[1]);
  p[1] = pair_of(x[2], x[3]);
}
__device__ __forceinline__ void from_pairs2(const Pair (&p)[2], float (&x)[4]) {
  parts_of(p[0], x[0], x[1]);
  parts_of(p[1], x[2], x[3]);
}

template <typename T, int D, bool kNext>
__global__ void __launch_bounds__(kNormBwdThreads, kNormBwdCtasPerSm)
gdn_head_norm_rope_bwd_kernel(const NormRopeParams p) {
  using Plan = NormBwdPlan<T, D>;
  constexpr int LPH = D / 8, SLOTS = Plan::SLOTS, U = Plan::U, WARPS = Plan::WARPS, STAGES = Plan::STAGES, ROW = Plan::ROW;
  __shared__ __align__(16) uint8_t s_ring[Plan::BYTES];
  __shared__ __align__(16) float s_sum[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPH, slot = lane / LPH;
  uint8_t* ring = s_ring + warp * STAGES * Plan::STEP;
  const bool is_q = static_cast<int>(blockIdx.x) < p.q_ctas;
  const T* x = static_cast<const T*>(is_q ? p.q : p.k);
  const T* dy = static_cast<const T*>(is_q ? p.q_grad : p.k_grad);
  T* dx = static_cast<T*>(is_q ? p.q_out : p.k_out);
  const int64_t xs = is_q ? p.q_stride : p.k_stride, gs = is_q ? p.q_grad_stride : p.k_grad_stride,
                ds = is_q ? p.q_out_stride : p.k_out_stride;
  const int heads = is_q ? p.nq : p.nkv;
  const unsigned parts = is_q ? p.q_parts : p.k_parts, per = is_q ? p.q_per : p.k_per;
  const unsigned items = static_cast<unsigned>(p.rows) * parts;
  const unsigned stride = (is_q ? p.q_ctas : gridDim.x - p.q_ctas) * WARPS;
  const HeadLane<D, kNext> hl(l, p.rope.rot);
  Pair wu[2], wv[2], du[2] = {0, 0}, dv[2] = {0, 0};
  {
    float a[4], b[4];
    hl.weights(is_q ? p.q_weight : p.k_weight, a, b);
    to_pairs2(a, wu);
    to_pairs2(b, wv);
  }

  // Two walks over the steps: one fetches, one computes and writes.
  unsigned f_item = (is_q ? blockIdx.x : blockIdx.x - p.q_ctas) * WARPS + warp, c_item = f_item;
  int f_left = 0, c_left = 0;  // heads that the item still has
  // the position of the item to fetch next, loaded an item ahead: its latency would else stand
  // before every item's angles
  auto position = [&](unsigned item) { return p.rope.rot && item < items ? p.positions[parts == 1 ? item : item / parts] : 0; };
  int pos = position(f_item);
  const uint8_t *f_x = nullptr, *f_g = nullptr;
  const float* f_angle = nullptr;
  T* c_dx = nullptr;
  bool f_ok = false;
  const int pieces = p.rope.rot >> 3;  // 16-byte pieces of the cosines, and of the sines
  const bool sine = lane >= pieces;
  const int piece = 4 * (sine ? lane - pieces : lane);
  auto item_heads = [&](unsigned item, unsigned* row, int* h) {
    *row = parts == 1 ? item : item / parts;
    *h = static_cast<int>((item - *row * parts) * per);
    return *h + static_cast<int>(per) < heads ? static_cast<int>(per) : heads - *h;
  };
  auto f_enter = [&] {
    if (f_item >= items) return;
    unsigned row;
    int h;
    f_left = item_heads(f_item, &row, &h);
    if (p.rope.rot) {
      f_ok = position_held(pos, p.rope, p.status);
      f_angle = (sine ? p.rope.sin : p.rope.cos) + static_cast<int64_t>(pos) * p.rope.stride + piece;
      pos = position(f_item + stride);
    } else {
      f_ok = true;
    }
    f_x = reinterpret_cast<const uint8_t*>(x + row * xs + static_cast<int64_t>(h) * D);
    f_g = reinterpret_cast<const uint8_t*>(dy + row * gs + static_cast<int64_t>(h) * D);
  };
  auto c_enter = [&] {
    if (c_item >= items) return;
    unsigned row;
    int h;
    c_left = item_heads(c_item, &row, &h);
    c_dx = dx + row * ds + static_cast<int64_t>(h + slot) * D;
  };
  unsigned held = 0;  // a bit a fetched step, the newest last: its position is in the table
  auto fetch = [&](int stage) {
    held <<= 1;
    if (f_item < items) {
      const uint32_t dst = tc::smem_u32(ring) + stage * Plan::STEP;
      held |= f_ok ? 1u : 0u;
#pragma unroll
      for (int b = 0; b < Plan::HEADS; b += 512) {
        const int at = b + 16 * lane;
        const bool real = f_ok && at / ROW < f_left;
        cp_async_16(dst + at, f_x + (real ? at : 0), real);
        cp_async_16(dst + Plan::HEADS + at, f_g + (real ? at : 0), real);
      }
      // (nothing of the table for a position outside it: it may have no rows; what the step then works out is dropped)
      if (f_ok && lane < 2 * pieces) cp_async_16_ca(dst + 2 * Plan::HEADS + (sine ? 2 * D : 0) + 4 * piece, f_angle);
      f_x += Plan::HEADS;
      f_g += Plan::HEADS;
      f_left -= U * SLOTS;
      if (f_left <= 0) {
        f_item += stride;
        f_enter();
      }
    }
    tc::cp_async_commit();
  };
  f_enter();
  c_enter();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  for (int stage = 0; c_item < items; stage = stage + 1 < STAGES ? stage + 1 : 0) {
    fetch(stage == 0 ? STAGES - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    __syncwarp();
    const uint8_t* src = ring + stage * Plan::STEP;
    Pair c[2], s[2], ns[2];
    {
      const float* angles = reinterpret_cast<const float*>(src + 2 * Plan::HEADS);
      float a[4], b[4];
      hl.angles(RopeParams{angles, angles + D / 2, 0, 1, p.rope.rot}, 0, a, b);
      to_pairs2(a, c);
      to_pairs2(b, s);
#pragma unroll
      for (int j = 0; j < 2; ++j) ns[j] = s[j] ^ 0x8000000080000000ull;
    }
    const bool ok = (held >> (STAGES - 1)) & 1;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      Pair u[2], v[2], gu[2], gv[2], zu[2], zv[2], tu[2], tv[2];
      {
        float a[4], b[4];
        hl.load(reinterpret_cast<const T*>(src) + (i * SLOTS + slot) * D, a, b);
        to_pairs2(a, u);
        to_pairs2(b, v);
        hl.load(reinterpret_cast<const T*>(src + Plan::HEADS) + (i * SLOTS + slot) * D, a, b);
        to_pairs2(a, gu);
        to_pairs2(b, gv);
      }
      Pair q2 = 0, m2 = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        zu[j] = fma2(gu[j], c[j], mul2(gv[j], s[j]));
        zv[j] = fma2(gv[j], c[j], mul2(gu[j], ns[j]));
        tu[j] = mul2(zu[j], wu[j]);
        tv[j] = mul2(zv[j], wv[j]);
        q2 = fma2(u[j], u[j], fma2(v[j], v[j], q2));
        m2 = fma2(tu[j], u[j], fma2(tv[j], v[j], m2));
      }
      float qa, qb, ma, mb;
      parts_of(q2, qa, qb);
      parts_of(m2, ma, mb);
      // dx = r (t - (x r) (r mean(t x))): the powers of r stay with what they scale, since r^3 by itself leaves
      // fp32 for rows far from 1 (of 1e13 and more, below 1e-13 without eps) whose gradient does not
      const float r = rsqrtf(row_sum<LPH>(qa + qb) * (1.f / D) + p.eps);
      const float f = -r * (row_sum<LPH>(ma + mb) * (1.f / D));
      if (ok && i * SLOTS + slot < c_left) {
        const Pair rr = pair_of(r, r), ff = pair_of(f, f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Pair xu = mul2(u[j], rr), xv = mul2(v[j], rr);
          du[j] = fma2(zu[j], xu, du[j]);
          dv[j] = fma2(zv[j], xv, dv[j]);
          tu[j] = mul2(fma2(xu, ff, tu[j]), rr);
          tv[j] = mul2(fma2(xv, ff, tv[j]), rr);
        }
        float a[4], b[4];
        from_pairs2(tu, a);
        from_pairs2(tv, b);
        hl.store(c_dx + i * SLOTS * D, a, b);
      }
    }
    __syncwarp();  // the stage is read before the next step's fetch overwrites it
    c_dx += U * SLOTS * D;
    c_left -= U * SLOTS;
    if (c_left <= 0) {
      c_item += stride;
      c_enter();
    }
  }
  float su[4], sv[4];
  from_pairs2(du, su);
  from_pairs2(dv, sv);
  if (!p.partials) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // over the head rows that a warp holds side by side
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      su[j] += __shfl_xor_sync(0xffffffffu, su[j], o);
      sv[j] += __shfl_xor_sync(0xffffffffu, sv[j], o);
    }
  }
  if (lane < LPH) hl.store(&s_sum[warp][0], su, sv);
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kNormBwdThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) t += s_sum[w][i];
    p.partials[static_cast<int64_t>(blockIdx.x) * D + i] = t;
  }
}

// dw[i] = sum over the partials of q's CTAs (blockIdx.y 0) or k's (1), in a fixed order: 32 values a
// CTA, a warp every 32nd partial.
__global__ void __launch_bounds__(1024) gdn_norm_weight_sum_kernel(const float* partials, int d, int q_ctas, int ctas,
                                                                  float* dq_weight, float* dk_weight) {
  __shared__ float s_part[32][33];
  tc::grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  float* dst = blockIdx.y == 0 ? dq_weight : dk_weight;
  if (!dst) return;
  const int first = blockIdx.y == 0 ? 0 : q_ctas, end = blockIdx.y == 0 ? q_ctas : ctas;
  float t = 0.f;
#pragma unroll 8
  for (int j = first + warp; j < end; j += 32) t += partials[static_cast<int64_t>(j) * d + i];
  s_part[warp][lane] = t;
  __syncthreads();
  t = s_part[lane][warp];  // warp w adds value w's 32 sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) dst[blockIdx.x * 32 + warp] = t;
}

// ---- paged cache -----------------------------------------------------------------------
struct PagedParams {
  void* k;
  void* v;
  int64_t k_page, k_token, k_head;
  int64_t v_page, v_token, v_head;
  int num_pages, page_size;
  const int32_t* block_table;
  int64_t table_stride;
  int max_pages;
  int B, rows;
  const int32_t* ctx_lens;
  const int32_t* cu_rows;
};

// The sequence that owns a row: the last b with cu[b] <= row, by a 32-way search of the whole
// warp (two steps for 1024 sequences). Any cu gives some b in [0, B).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && cu[lo + (at < n ? at : 0)] <= row);
    const int w = m ? 31 - __clz(m) : 0;
    lo += w * step;
    n = n - w * step < step ? n - w * step : step;
  }
  return lo;
}

struct AppendParams {
  const void* k;
  const void* v;
  PagedParams cache;
  const int32_t* positions;
  RopeParams rope;
  const float* k_weight;
  int64_t k_stride, v_stride;
  int nkv, chunks;  // warp items of a token
  int norm;
  float eps;
  unsigned* status;
};

template <typename T, int D, bool kNext, int U>
__global__ void __launch_bounds__(kNormThreads, kAppendCtasPerSm) gdn_paged_append_kernel(const AppendParams p) {
  constexpr int LPH = D / 8, SLOTS = 32 / LPH, PER = U * SLOTS;
  const unsigned item = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  const unsigned row = item / static_cast<unsigned>(p.chunks);
  const PagedParams& c = p.cache;
  if (row >= static_cast<unsigned>(c.rows)) return;
  const int h0 = static_cast<int>(item - row * p.chunks) * PER;
  const int lane = threadIdx.x & 31, slot = lane / LPH, at8 = 8 * (lane % LPH);
  // the heads first, keys and values: their loads overlap the look-up of the token's place
  typename Four<T>::Word x[U][2];
  fetch_heads<T, D, kNext, U>(static_cast<const T*>(p.k) + row * p.k_stride, D, h0, p.nkv, p.rope.rot, x);
  uint4 v[U];
  {
    const T* src = static_cast<const T*>(p.v) + row * p.v_stride + at8;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * SLOTS + slot;
      v[i] = h < p.nkv ? *reinterpret_cast<const uint4*>(src + h * D) : make_uint4(0, 0, 0, 0);
    }
  }
  const int b = c.cu_rows ? find_sequence(c.cu_rows, c.B, static_cast<int>(row)) : static_cast<int>(row);
  const int first = c.cu_rows ? c.cu_rows[b] : static_cast<int>(row);
  const int end = c.cu_rows ? c.cu_rows[b + 1] : static_cast<int>(row) + 1;
  const int ctx = c.ctx_lens[b];
  if (first < 0 || first > static_cast<int>(row) || end <= static_cast<int>(row) || end > c.rows || ctx < 0) {
    if (lane == 0) atomicOr(p.status, kStatusBadSeqlens);
    return;
  }
  const int64_t token = static_cast<int64_t>(ctx) + (static_cast<int>(row) - first);
  // (below max_pages * page_size < 2^31 where it counts; the division is 32-bit then)
  const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_size;
  const unsigned at = token < room ? static_cast<unsigned>(token) / static_cast<unsigned>(c.page_size) : 0u;
  const int page = token < room ? c.block_table[b * c.table_stride + at] : -1;
  if (page < 0 || page >= c.num_pages) {
    if (lane == 0) atomicOr(p.status, kStatusBadPage);
    return;
  }
  const int64_t place = token - static_cast<int64_t>(at) * c.page_size;
  const int64_t pos = p.positions && p.rope.rot ? p.positions[row] : token;
  if (!position_held(pos, p.rope, p.status)) return;  // the token is left out whole
  T* dst = static_cast<T*>(c.v) + page * c.v_page + place * c.v_token + at8;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * SLOTS + slot;
    if (h < p.nkv) *reinterpret_cast<uint4*>(dst + h * c.v_head) = v[i];
  }
  norm_rope_heads<T, D, kNext, U>(x, static_cast<T*>(c.k) + page * c.k_page + place * c.k_token, c.k_head, h0, p.nkv,
                               p.k_weight, p.norm != 0, p.eps, p.rope, pos);
}

}  // namespace gdn
