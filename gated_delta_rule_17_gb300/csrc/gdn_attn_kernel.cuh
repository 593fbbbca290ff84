// Attention of decode tokens and small drafted trees over a paged cache, for sm_103a.
//
// For few query rows a kv head (R = rows x heads of a group) the operator does R flops a
// byte of the cache, far below the 289 flops a byte at which the card's tensor rate meets
// its bandwidth, so it is bound by reading K and V once. Every warp is on its own: it
// streams 16-token slabs of K and V through its private ring in shared memory (16-byte
// cp.async from the tokens' places in the pages, any page size), and has 16 query rows against
// them with register tensor products: scores S = Q K^T, running maximum and sum, O += P V.
// No barrier is needed in the loop; the warps' (m, l, O) are added up at a unit's end.
// One token each of 64 sequences of 100 to 16000 tokens, 32 heads on 8 kv heads of 128: 326 to
// 335 us with the join, 6.3 to 6.5 TB/s, 93 to 95% of the measured copy rate; the loads' latency at the units' ends and the
// join are the rest.
#pragma once
#include "gdn_attn_common.cuh"

namespace gdn {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnRows = 16;                      // query rows of a unit
constexpr int kAttnSlab = 16;                      // tokens of a warp's step
constexpr int kAttnTile = kAttnWarps * kAttnSlab;  // tokens of a CTA's step

template <int D>
struct AttnPlan {
  static constexpr int MT = kAttnRows;
  static constexpr int ROW = D * 2;                        // bytes of a key or value
  static constexpr int SLAB = kAttnSlab * ROW;             // bytes of a slab of K or V
  static constexpr int STAGES = 3 * 128 / D;
  static constexpr int RING = STAGES * 2 * SLAB;           // bytes of a warp's ring
  static constexpr int JOIN = kAttnWarps * MT * (D + 2) * 4;  // the warps' O, m and l at a unit's end
  static constexpr int BYTES = kAttnWarps * RING > JOIN ? kAttnWarps * RING : JOIN;
  static constexpr int DYN_SMEM = BYTES + 128;
};

__device__ __forceinline__ void ldmatrix4(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// d += a (16 x 16) b (16 x 8)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte piece c of row r: pieces are exchanged within a row by the row's number,
// so that eight rows' pieces c lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t attn_sw(int r, int c) {
  return static_cast<uint32_t>(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// The place of a token: its page (-1 for none) and place in it.
struct TokenPlace {
  int page, place;
};
__device__ __forceinline__ TokenPlace token_place(const AttnParams& p, const int32_t* table, int t, int len) {
  TokenPlace r{-1, 0};
  if (t < len) {
    const int at = t / p.cache.page_size;
    r.place = t - at * p.cache.page_size;
    r.page = table[at];
    if (r.page < 0 || r.page >= p.cache.num_pages) {
      r.page = -1;
      atomicOr(p.status, kStatusBadPage);
    }
  }
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 2) gdn_attn_kernel(const AttnParams p) {
  using Plan = AttnPlan<D>;
  constexpr int MT = Plan::MT, KS = D / 16, NT = D / 8, CH = D / 8, STAGES = Plan::STAGES;
  extern __shared__ uint8_t dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 127) & ~static_cast<uintptr_t>(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, tc = lane & 3;  // fragment row and column pair
  const uint32_t ring = tc::smem_u32(smem) + warp * Plan::RING;
  const PagedParams& c = p.cache;
  const int run = blockIdx.x;

  __shared__ AttnWalk<MT, kAttnTile> s_walk;
  tc::grid_dependency_wait();
  if (warp == 0) {
    AttnWalk<MT, kAttnTile> found;
    found.begin(p, attn_start<MT, kAttnTile>(p, run));
    if (lane == 0) s_walk = found;
  }
  __syncthreads();
  tc::allow_dependent_launch();  // the join waits for this grid's end before it reads anything
  if (threadIdx.x == 0 && !p.whole) p.cut[run] = make_int4(0, 0, 0, -1);
  AttnWalk<MT, kAttnTile> w = s_walk;
  for (; w.any; w.next(p)) {
    const AttnSeq& s = w.s;
    const int b = w.b, kvh = w.kvh, qt = w.qt, t0 = w.t0, t1 = w.t1;
    const int R = s.n * p.group;
    const int32_t* table = c.block_table + b * c.table_stride;

    // Q fragments: rows gr and gr + 8
    uint32_t qf[KS][4];
    int node[2];  // the new token of either row, -1 for none
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = qt * MT + hf * 8 + gr;
      const int i = r < R ? r / p.group : 0, g = r < R ? r - i * p.group : 0;
      node[hf] = r < R ? i : -1;
      const T* src = static_cast<const T*>(p.q) + (static_cast<int64_t>(s.first) + i) * p.q_stride +
                     static_cast<int64_t>(kvh * p.group + g) * D + 2 * tc;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks][hf] = r < R ? *reinterpret_cast<const uint32_t*>(src + 16 * ks) : 0u;
        qf[ks][2 + hf] = r < R ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8) : 0u;
      }
    }
    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][j] = 0.f;

    const T* kbase = static_cast<const T*>(c.k) + kvh * c.k_head;
    const T* vbase = static_cast<const T*>(c.v) + kvh * c.v_head;
    // the copies of slab `t` of this warp: lane i & 15 knows token i's place
    auto find = [&](int t) { return token_place(p, table, t * kAttnTile + warp * kAttnSlab + (lane & 15), t < t1 ? s.len : 0); };
    auto issue = [&](int t, const TokenPlace& place) {
      const uint32_t dst = ring + (t % STAGES) * (2 * Plan::SLAB);
      constexpr int ROWS = 32 / CH;  // tokens of one copy instruction
#pragma unroll
      for (int i = 0; i < kAttnSlab / ROWS; ++i) {
        const int r = i * ROWS + lane / CH, ch = lane % CH;
        const int page = __shfl_sync(0xffffffffu, place.page, r), at = __shfl_sync(0xffffffffu, place.place, r);
        const bool real = page >= 0;
        const int64_t pg = real ? page : 0;
        cp_async_16(dst + attn_sw<D>(r, ch), kbase + pg * c.k_page + at * c.k_token + 8 * ch, real);
        cp_async_16(dst + Plan::SLAB + attn_sw<D>(r, ch), vbase + pg * c.v_page + at * c.v_token + 8 * ch, real);
      }
    };
    TokenPlace next = find(t0);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      const TokenPlace place = next;
      next = find(t0 + i + 1);
      if (t0 + i < t1) issue(t0 + i, place);
      tc::cp_async_commit();
    }
    for (int t = t0; t < t1; ++t) {
      const TokenPlace place = next;
      next = find(t + STAGES);
      __syncwarp();  // all lanes have read the slab that is overwritten now
      if (t + STAGES - 1 < t1) issue(t + STAGES - 1, place);
      tc::cp_async_commit();
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t ks_addr = ring + (t % STAGES) * (2 * Plan::SLAB), vs_addr = ks_addr + Plan::SLAB;
      const int tok = t * kAttnTile + warp * kAttnSlab;
      if (tok >= s.len) continue;  // the whole warp: nothing of its slab is there

      float sc[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t kf[4];
        ldmatrix4(ks_addr + attn_sw<D>((lane >> 4) * 8 + (lane & 7), 2 * ks + ((lane >> 3) & 1)), kf);
        mma16816<T>(sc[0], qf[ks], kf[0], kf[1]);
        mma16816<T>(sc[1], qf[ks], kf[2], kf[3]);
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[nt][j] *= p.scale_log2;  // before the mask: the scale may be negative
      // tokens that a row does not see; before the new tokens every row sees all
      if (tok + kAttnSlab > s.ctx) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = tok + nt * 8 + 2 * tc + (j & 1), i = node[j >> 1], x = at - s.ctx;
            bool sees = at < s.len;
            if (sees && x >= 0) {
              if (!p.mask)
                sees = x <= i;
              else
                sees = i >= 0 && (x >> 6) < p.mask_words &&
                       ((p.mask[(static_cast<int64_t>(s.first) + i) * p.mask_words + (x >> 6)] >> (x & 63)) & 1);
            }
            if (!sees) sc[nt][j] = -INFINITY;
          }
      }
      uint32_t pf[4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float x0 = sc[0][2 * hf], x1 = sc[0][2 * hf + 1], x2 = sc[1][2 * hf], x3 = sc[1][2 * hf + 1];
        float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[hf], mx), base = mn == -INFINITY ? 0.f : mn;
        if (__any_sync(0xffffffffu, mn > m[hf])) {
          const float f = exp2_approx(m[hf] - base);
          l[hf] *= f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][2 * hf] *= f;
            o[nt][2 * hf + 1] *= f;
          }
          m[hf] = mn;
        }
        const float one = base - kWeightLog2<T>;
        x0 = exp2_approx(x0 - one);
        x1 = exp2_approx(x1 - one);
        x2 = exp2_approx(x2 - one);
        x3 = exp2_approx(x3 - one);
        l[hf] += (x0 + x1) + (x2 + x3);  // this thread's tokens; over the row at the end
        pf[hf] = pack2<T>(x0, x1);
        pf[2 + hf] = pack2<T>(x2, x3);
      }
#pragma unroll
      for (int cp = 0; cp < NT / 2; ++cp) {
        uint32_t vf[4];
        ldmatrix4_trans(vs_addr + attn_sw<D>(((lane >> 3) & 1) * 8 + (lane & 7), 2 * cp + (lane >> 4)), vf);
        mma16816<T>(o[2 * cp], pf, vf[0], vf[1]);
        mma16816<T>(o[2 * cp + 1], pf, vf[2], vf[3]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // add up the warps' parts
    float* jo = reinterpret_cast<float*>(smem);       // [warp][MT][D]
    float* jml = jo + kAttnWarps * MT * D;            // [warp][MT][2]
    __syncthreads();                                  // the rings are done with
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = hf * 8 + gr;
      float ll = l[hf];
      ll += __shfl_xor_sync(0xffffffffu, ll, 1);
      ll += __shfl_xor_sync(0xffffffffu, ll, 2);
      if (tc == 0) {
        jml[(warp * MT + r) * 2] = m[hf];
        jml[(warp * MT + r) * 2 + 1] = ll;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float2*>(jo + (warp * MT + r) * D + nt * 8 + 2 * tc) = make_float2(o[nt][2 * hf], o[nt][2 * hf + 1]);
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == s.tiles;
    const int slot = t0 == 0 ? 1 : 0;
    constexpr int LPR = D / 4;  // threads of a row
    for (int r = threadIdx.x / LPR; r < MT; r += kAttnThreads / LPR) {
      const int row = qt * MT + r;
      if (row >= R) continue;
      const int d4 = (threadIdx.x % LPR) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) mm = fmaxf(mm, jml[(w * MT + r) * 2]);
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f, a[4] = {};
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        const float f = exp2_approx(jml[(w * MT + r) * 2] - base);
        const float4 v = *reinterpret_cast<const float4*>(jo + (w * MT + r) * D + d4);
        ll = fmaf(f, jml[(w * MT + r) * 2 + 1], ll);
        a[0] = fmaf(f, v.x, a[0]);
        a[1] = fmaf(f, v.y, a[1]);
        a[2] = fmaf(f, v.z, a[2]);
        a[3] = fmaf(f, v.w, a[3]);
      }
      if (whole) {
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
        const int i = row / p.group, g = row - i * p.group;
        T* dst = static_cast<T*>(p.out) + (static_cast<int64_t>(s.first) + i) * p.out_stride +
                 static_cast<int64_t>(kvh * p.group + g) * D + d4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(a[0] * inv, a[1] * inv), pack2<T>(a[2] * inv, a[3] * inv));
      } else {
        const int64_t at = (static_cast<int64_t>(run) * 2 + slot) * MT + r;
        *reinterpret_cast<float4*>(p.part_o + (at - r) * D + attn_piece_at<MT>(r, d4)) = make_float4(a[0], a[1], a[2], a[3]);
        if (d4 == 0) {
          p.part_ml[at * 2] = mm;
          p.part_ml[at * 2 + 1] = ll;
        }
      }
    }
    __syncthreads();  // the join buffer is done with
    if (t0 == 0 && t1 < s.tiles && threadIdx.x == 0) p.cut[run] = w.cut(p);
  }
}

// Joins the pieces of the units that were cut. Every CTA reads the list of them and takes its share of
// their parts of 8 rows by 16 columns, a value of a row and four columns a lane: a grid of rows by runs
// had thousands of CTAs that only found nothing to do, and one warp for the fifty pieces of a row (one
// long sequence alone). Where there are more parts than warps a warp takes whole parts; where there are
// few, 2, 4 or 8 warps share one, each every W-th group of kJoinPieces pieces, whose loads are under
// way together. Measured: trees of 64 over 32768 in 8 sequences, 28 MB of pieces, 6 us and 1 us for
// the list; with 8 pieces at a time, or 2 or 4 CTAs an SM, 1 to 4 us more.
constexpr int kJoinWarps = 8;
constexpr int kJoinCtasPerSm = 3;
constexpr int kJoinPieces = 4;
constexpr int kJoinRuns = 512;  // runs whose units a CTA can list

template <typename T, int D, int MT>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinCtasPerSm) gdn_attn_join_kernel(const AttnParams p) {
  constexpr int U = kJoinPieces, CT = D / 16;
  __shared__ int4 s_cut[kJoinRuns];
  __shared__ int s_end[kJoinRuns];  // groups of 8 rows up to and with a run's unit
  __shared__ int s_sum[kJoinWarps];
  __shared__ float2 s_ml[kJoinWarps][32];
  __shared__ float4 s_o[kJoinWarps][32];
  tc::allow_dependent_launch();
  tc::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int total = 0;
  for (int c0 = 0; c0 < p.runs; c0 += 32 * kJoinWarps) {
    const int run = c0 + threadIdx.x;
    int groups = 0;
    if (run < p.runs) {
      const int4 cut = p.cut[run];
      s_cut[run] = cut;
      if (cut.w >= 0) groups = ((cut.w >> 16) + 7) / 8;
    }
    int upto = groups;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += y;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const int x = s_sum[w];
      if (w < warp) upto += x;
      all += x;
    }
    if (run < p.runs) s_end[run] = total + upto;
    total += all;
    __syncthreads();
  }
  const int parts = total * CT, ctas = gridDim.x;
  const int W = parts <= ctas ? 8 : parts <= 2 * ctas ? 4 : parts <= 4 * ctas ? 2 : 1;  // warps of a part
  const int sub = warp & (W - 1);
  // with W > 1 every part has its warps, and all warps take part in the one step
  for (int part = (blockIdx.x * kJoinWarps + warp) / W; part < parts || W > 1; part += ctas * kJoinWarps) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 cut = make_int4(0, 0, 0, 0);
    int row = 0;
    const int col = (part % CT) * 16 + (lane & 3) * 4;
    if (part < parts) {
      const int group = part / CT;
      int run = 0, hi = p.runs - 1;  // the first run with more groups up to it
      while (run < hi) {
        const int mid = (run + hi) >> 1;
        if (s_end[mid] > group) hi = mid;
        else run = mid + 1;
      }
      cut = s_cut[run];
      const int rows = cut.w >> 16, last = cut.w & 0xffff;
      row = (group - (run ? s_end[run - 1] : 0)) * 8 + (lane >> 2);
      const int r = row < rows ? row : rows - 1;
      for (int i0 = run + sub * U; i0 <= last; i0 += W * U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ml[u] = make_float2(-INFINITY, 0.f);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + u <= last) {
            const int64_t at = (static_cast<int64_t>(i0 + u) * 2 + (i0 + u == run ? 1 : 0)) * MT;
            ml[u] = *reinterpret_cast<const float2*>(p.part_ml + (at + r) * 2);
            v[u] = *reinterpret_cast<const float4*>(p.part_o + at * D + attn_piece_at<MT>(r, col));
          }
        }
        attn_join<U>(ml, v, m, l, o);
      }
    }
    if (W > 1) {
      s_ml[warp][lane] = make_float2(m, l);
      s_o[warp][lane] = o;
      __syncthreads();
      if (sub != 0 || part >= parts) return;
      for (int w = 1; w < W; ++w) {
        const float2 ml[1] = {s_ml[warp + w][lane]};
        const float4 v[1] = {s_o[warp + w][lane]};
        attn_join<1>(ml, v, m, l, o);
      }
    }
    if (row < cut.w >> 16) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int at = cut.z + row, i = at / p.group, g = at - i * p.group;
      T* dst = static_cast<T*>(p.out) + (static_cast<int64_t>(cut.x) + i) * p.out_stride +
               static_cast<int64_t>(cut.y * p.group + g) * D + col;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
    }
    if (W > 1) return;
  }
}

}  // namespace gdn
