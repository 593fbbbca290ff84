// Attention of larger drafted trees and prompt chunks over a paged cache on the 5th-generation tensor
// cores, for sm_103a.
//
// With R query rows a kv head the operator does R flops a byte of the cache, so from some tens of
// rows on the register products of gdn_attn_kernel bound it, and from about 256 rows the tensor
// cores' rate does. A CTA works on two score streams x = 0, 1 of 128 query rows, each with its own
// scores and accumulators in tensor memory, and takes tiles of 128 tokens:
//
//     S_x = Q_x K^T (tcgen05)  ->  four warps: running maximum m, P = 2^(S c - m c), sum l
//     O_x += P V  (tcgen05, P from tensor memory, where it takes the place of S_x)
//
// so that the products of one stream run while the warps of the other take exponentials. A unit has
// up to 256 rows. With more than 128 ("dual") both streams see every token tile, and one load of K
// and V serves 256 rows; with fewer ("split") the streams take alternate token tiles of the same
// rows, and their (m, l, O) are added up at the unit's end.
// O stays unnormalised in tensor memory. It is scaled down only when a row's maximum has grown by
// more than 2^8 since its last reference: until then P <= 2^8 relative to the reference, which
// costs no precision in fp32 and 16-bit floats (their relative error does not depend on the size;
// 2^8 and kWeightLog2 together are inside fp16's range), and most tiles skip the round trip through the registers.
//
// Roles: warps 0-3 and 4-7 one stream each; warps 8-11 copy Q, K and V tiles (TMA boxes inside the
// pages, or 16-byte cp.async for any page size; 128-byte-swizzled rows), K and V through a ring of
// STAGES tiles, the next unit's Q as soon as the last scores of this one are done; an elected thread
// of warp 12 issues the products. The hand-offs are mbarriers; every wait is bounded, and when one
// expires the status word says so and all roles run out.
//
// What bounds it: with many rows the chain of a stream from one tile's scores to the next's, about 3000
// cycles (softmax 1500, the products of both kinds 1024 one after the other because P lies over S,
// hand-offs the rest), of which two streams fill the tensor pipe to 59%, and the start, the pieces of cut
// units and the join. Trees of 64 in 8 sequences of 32768, 32 heads on 4: 215 to 222 us, 1.22 to 1.26
// PFLOP/s, 62 to 65% of the measured cuBLAS rate, the clock held down by the power limit; 196 to 202 us in loops too
// short for that (173 us for each 32768 tokens more, 81%). With few
// rows HBM and the ends: trees of 3 to 16 in 16 sequences of 500 to 8192, 32 heads on 8: 58 us, 5.1
// TB/s. Tensor memory is full (S and O of two streams), so a third stream, or P beside S, has no room;
// one pass over the scores instead of two, the row in registers, two warps a row, handing P over in
// halves and scores in halves of 64 tokens were slower or no faster.
#pragma once
#include "gdn_attn_kernel.cuh"

namespace gdn {

constexpr int kTcTile = 128;  // tokens of a tile, and rows of a stream
constexpr int kTcRows = 256;  // rows of a unit
constexpr int kTcThreads = 416;
constexpr float kTcGrowth = 8.f;  // log2 of the growth of a maximum that O is not scaled for

template <int D>
struct AttnTcPlan {
  static constexpr int TILE = kTcTile * D * 2;  // Q of a stream, or a tile of K or V
  // the ring: as many tiles as fit; with D = 64 enough to keep the CTA alone on its SM, since it
  // takes all of the tensor memory
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int LAG = 2;  // cp.async tiles in flight behind the one just issued
  static constexpr int Q = 0;
  static constexpr int RING = 2 * TILE;
  static constexpr int BYTES = RING + STAGES * TILE;
  static constexpr int DYN_SMEM = BYTES + 1024;  // slack for 1024-byte alignment
  static constexpr uint32_t COL_S = 0, COL_O = 256, TMEM_COLS = 512;
  // mbarriers
  static constexpr int FULL = 0, FREE = STAGES, S_FULL = 2 * STAGES, P_FULL = S_FULL + 2, O_FULL = P_FULL + 2,
                       Q_FULL = O_FULL + 2, Q_FREE = Q_FULL + 1, JOIN = Q_FREE + 1, NBAR = JOIN + 1;
};

// Which of tokens tok .. tok + 31 the new row i of sequence s sees, as bits.
__device__ __forceinline__ uint32_t sees32(const AttnParams& p, const AttnSeq& s, int i, int tok) {
  if (tok + 32 <= s.ctx && tok + 32 <= s.len) return ~0u;
  if (tok >= s.len) return 0u;
  const int o = tok - s.ctx;  // > -32, or all of them are context
  uint32_t w = ~0u;
  if (o > -32) {
    if (!p.mask) {
      const int n = i - o + 1;
      w = n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
    } else {
      const uint64_t* row = p.mask + (static_cast<int64_t>(s.first) + i) * p.mask_words;
      if (o >= 0) {
        const int at = o >> 6, sh = o & 63;
        const uint64_t lo = at < p.mask_words ? row[at] : 0, hi = at + 1 < p.mask_words ? row[at + 1] : 0;
        w = static_cast<uint32_t>((lo >> sh) | (sh ? hi << (64 - sh) : 0));
      } else {
        w = (static_cast<uint32_t>(row[0]) << -o) | ((1u << -o) - 1u);
      }
    }
  }
  const int lim = s.len - tok;
  return lim < 32 ? w & ((1u << lim) - 1u) : w;
}

// A wait that did not succeed at once, with its time limit. Out of line: the roles' loops share the
// instruction caches, and their size is what the issuing warp feels first.
__device__ __noinline__ bool tc_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort, unsigned* status) {
  const uint64_t t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait_hint(bar, parity, 100000u)) {
    if (*abort) return false;
    if (tc::globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

struct TcShared {
  uint32_t bars;  // shared address of the mbarriers
  volatile uint32_t* abort;
  unsigned* status;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // Bounded wait by a whole warp, with one answer.
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
    const bool ok = tc::mbar_try_wait(bar(i), parity);
    return __all_sync(0xffffffffu, ok) || __all_sync(0xffffffffu, ok || tc_wait_slow(bar(i), parity, abort, status));
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
gdn_attn_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const AttnParams p) {
  using Plan = AttnTcPlan<D>;
  constexpr int MT = kTcRows, TILE = Plan::TILE, NS = Plan::STAGES, LAG = Plan::LAG;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t s_bar[Plan::NBAR];
  __shared__ uint32_t s_tmem, s_abort;
  __shared__ AttnWalk<MT, kTcTile> s_walk;
  __shared__ float2 s_ml[2][kTcTile];  // split units: (m, l) of both streams
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedParams& c = p.cache;
  const int run = blockIdx.x;
  const TcShared sh{tc::smem_u32(s_bar), &s_abort, p.status};

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(sh.bar(Plan::FULL + i), 128);
      tc::mbar_init(sh.bar(Plan::FREE + i), 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(sh.bar(Plan::S_FULL + x), 1);
      tc::mbar_init(sh.bar(Plan::P_FULL + x), 4);
      tc::mbar_init(sh.bar(Plan::O_FULL + x), 1);
    }
    tc::mbar_init(sh.bar(Plan::Q_FULL), 128);
    tc::mbar_init(sh.bar(Plan::Q_FREE), 1);
    tc::mbar_init(sh.bar(Plan::JOIN), 256);
    tc::mbar_fence_init();
  }
  if (warp == 12) tc::tmem_alloc(tc::smem_u32(&s_tmem), Plan::TMEM_COLS);
  tc::grid_dependency_wait();  // so far nothing has touched global memory
  if (warp == 0) {
    AttnWalk<MT, kTcTile> found;
    found.begin(p, attn_start<MT, kTcTile>(p, run));
    if (lane == 0) s_walk = found;
  }
  if (threadIdx.x == 0 && !p.whole) p.cut[run] = make_int4(0, 0, 0, -1);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  tc::allow_dependent_launch();  // the join waits for this grid's end before it reads anything
  const uint32_t tmem = s_tmem;
  AttnWalk<MT, kTcTile> w = s_walk;

  if (warp < 8) {
    // ---- one row a thread: softmax, and the unit's end -----------------------------------
    const int x = warp >> 2, lrow = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's quarter of the lanes
    const uint32_t s_addr = tmem + lanes + Plan::COL_S + x * kTcTile, o_addr = tmem + lanes + Plan::COL_O;
    const float cl = p.scale_log2;
    const Pair cl2 = pair_of(cl, cl);
    uint32_t s_ph = 0, o_ph = 0, j_ph = 0;
    bool ok = true, pending = false;  // pending: the other stream may still read this one's O
    for (; ok && w.any; w.next(p)) {
      const AttnSeq& s = w.s;
      const int R = s.n * p.group;
      const bool split = R - w.qt * MT <= kTcTile;
      const int row = w.qt * MT + (split ? 0 : x * kTcTile) + lrow;
      const bool has = row < R;
      const int i = has ? row / p.group : 0, g = has ? row - i * p.group : 0;
      const bool used = __any_sync(0xffffffffu, has);  // any row of the warp
      const int step = split ? 2 : 1;
      float m = -INFINITY, l = 0.f;
      for (int t = w.t0 + (split ? x : 0); t < w.t1; t += step) {
        ok = sh.wait_warp(Plan::S_FULL + x, s_ph);
        s_ph ^= 1;
        if (!ok) break;
        tc::fence_after_sync();
        if (used) {
          const int tok = t * kTcTile;
          uint32_t r0[32], r1[32];
          if (tok + kTcTile > s.ctx || tok + kTcTile > s.len) {  // scores of unseen tokens become -inf
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const uint32_t vis = sees32(p, s, i, tok + 32 * k);
              if (__all_sync(0xffffffffu, vis == ~0u)) continue;
              tc::tmem_ld32(s_addr + 32 * k, r0);
              tc::tmem_ld_wait32(r0);
#pragma unroll
              for (int e = 0; e < 32; ++e) r0[e] = (vis >> e) & 1 ? r0[e] : 0xFF800000u;
              tc::tmem_st32(s_addr + 32 * k, r0);
            }
            tc::tmem_st_wait();
          }
          float mx[2] = {-INFINITY, -INFINITY};
          auto top_of = [&](const uint32_t (&r)[32]) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              mx[0] = fmaxf(mx[0], fmaxf(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
              mx[1] = fmaxf(mx[1], fmaxf(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])));
            }
          };
          tc::tmem_ld32(s_addr, r0);
          tc::tmem_ld_wait32(r0);
          tc::tmem_ld32(s_addr + 32, r1);
          top_of(r0);
          tc::tmem_ld_wait32(r1);
          tc::tmem_ld32(s_addr + 64, r0);
          top_of(r1);
          tc::tmem_ld_wait32(r0);
          tc::tmem_ld32(s_addr + 96, r1);
          top_of(r0);
          tc::tmem_ld_wait32(r1);
          tc::tmem_ld32(s_addr, r0);  // the second pass begins
          top_of(r1);
          const float top = fmaxf(mx[0], mx[1]);
          // a new reference for the row where its maximum has outgrown the old one (or there is none)
          const bool grown = top * cl > m * cl + kTcGrowth, fresh = m == -INFINITY;
          const float f = grown && !fresh ? exp2_approx((m - top) * cl) : 1.f;
          if (grown || fresh) m = top;
          if (__any_sync(0xffffffffu, f != 1.f)) {
            l *= f;
            tc::tmem_ld_wait32(r0);
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              tc::tmem_ld32(o_addr + x * D + 32 * k, r1);
              tc::tmem_ld_wait32(r1);
#pragma unroll
              for (int e = 0; e < 32; ++e) r1[e] = __float_as_uint(__uint_as_float(r1[e]) * f);
              tc::tmem_st32(o_addr + x * D + 32 * k, r1);
            }
          }
          const float nb = m == -INFINITY ? 0.f : (kWeightLog2<T> == 0.f ? -m * cl : kWeightLog2<T> - m * cl);
          const Pair nb2 = pair_of(nb, nb);
          Pair sum[2] = {0, 0};
          auto weights = [&](const uint32_t (&r)[32], int k) {  // over a part of S that has been read
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a, b;
              parts_of(fma2(pair_of(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), cl2, nb2), a, b);
              a = exp2_approx(a);
              b = exp2_approx(b);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair_of(a, b));
              pk[e >> 1] = pack2<T>(a, b);
            }
            tc::tmem_st16u(s_addr + 16 * k, pk);
          };
          tc::tmem_ld_wait32(r0);
          tc::tmem_ld32(s_addr + 32, r1);
          weights(r0, 0);
          tc::tmem_ld_wait32(r1);
          tc::tmem_ld32(s_addr + 64, r0);
          weights(r1, 1);
          tc::tmem_ld_wait32(r0);
          tc::tmem_ld32(s_addr + 96, r1);
          weights(r0, 2);
          tc::tmem_ld_wait32(r1);
          weights(r1, 3);
          float sa, sb;
          parts_of(add2(sum[0], sum[1]), sa, sb);
          l += sa + sb;
          tc::tmem_st_wait();
        }
        if (pending) {  // the products that follow overwrite O
          pending = false;
          ok = sh.wait_warp(Plan::JOIN, j_ph ^ 1);
          if (!ok) break;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sh.bar(Plan::P_FULL + x));
      }
      if (!ok) break;
      if (pending) {  // a unit in which this stream had no tile
        pending = false;
        ok = sh.wait_warp(Plan::JOIN, j_ph ^ 1);
        if (!ok) break;
      }
      // ---- the unit's end: rows out, or a piece of them into the workspace --------------------
      const bool whole = w.t0 == 0 && w.t1 == s.tiles, two = split && w.t0 + 1 < w.t1;
      ok = sh.wait_warp(Plan::O_FULL + x, o_ph);
      if (split && ok) {  // both streams' O, and both (m, l) for each stream's warps
        s_ml[x][lrow] = make_float2(m, l);
        tc::mbar_arrive(sh.bar(Plan::JOIN));
        ok = sh.wait_warp(Plan::O_FULL + (x ^ 1), o_ph) && sh.wait_warp(Plan::JOIN, j_ph);
        j_ph ^= 1;
      }
      o_ph ^= 1;
      if (!ok) break;
      tc::fence_after_sync();
      float f0 = 1.f, f1 = 0.f;
      if (split) {
        const float2 a = s_ml[0][lrow], b = s_ml[1][lrow];
        m = fmaxf(a.x, b.x);
        const float base = m == -INFINITY ? 0.f : m;
        f0 = exp2_approx((a.x - base) * cl);
        f1 = exp2_approx((b.x - base) * cl);
        l = a.y * f0 + b.y * f1;
      }
      const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      f0 *= inv;
      f1 *= inv;
      // a dual stream has its rows; the warps of a split unit have half of the columns each
      const int c0 = split ? x * (D / 2) : 0, c1 = split ? c0 + D / 2 : D, xo = split ? 0 : x;
      const int prow = (split ? 0 : x * kTcTile) + lrow;
      const int64_t part = (static_cast<int64_t>(run) * 2 + (w.t0 == 0 ? 1 : 0)) * MT + prow;
      // each lane stores whole 32-byte sectors of its own row
      char* dst = whole ? reinterpret_cast<char*>(static_cast<T*>(p.out) + (static_cast<int64_t>(s.first) + i) * p.out_stride +
                                                  static_cast<int64_t>(w.kvh * p.group + g) * D)
                        : reinterpret_cast<char*>(p.part_o + (part - prow) * D + attn_piece_at<MT>(prow, 0));
      const bool wide = !whole || p.out_wide;
      if (used) {
#pragma unroll 1
        for (int col = c0; col < c1; col += 16) {
          uint32_t r[16], o2[16];
          tc::tmem_ld16u(o_addr + xo * D + col, r);
          if (two) tc::tmem_ld16u(o_addr + D + col, o2);
          tc::tmem_ld_wait16(r);
          if (two) {
            tc::tmem_ld_wait16(o2);
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(fmaf(__uint_as_float(o2[e]), f1, __uint_as_float(r[e]) * f0));
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f0);
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = pack2<T>(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          }
          if (has) {
            store32(dst + col * (whole ? 2 : MT * 4), r, wide);
            if (!whole) store32(dst + (col + 8) * (MT * 4), r + 8, true);
          }
        }
      }
      if (split) {  // this stream's warps have read the other's O
        tc::fence_before_sync();
        tc::mbar_arrive(sh.bar(Plan::JOIN));
        pending = true;
        j_ph ^= 1;
      }
      if (has && !whole && (!split || x == 0))  // m in units of log2 e, as the join takes it
        *reinterpret_cast<float2*>(p.part_ml + part * 2) = make_float2(m == -INFINITY ? m : m * cl, l);
      if (threadIdx.x == 0 && w.t0 == 0 && w.t1 < s.tiles)
        p.cut[run] = w.cut(p);
    }
  } else if (warp < 12) {
    // ---- copies of Q, K and V --------------------------------------------------------------
    // A warp copies 32 tokens of every tile. Where a page holds whole boxes of p.box tokens and all
    // 32 tokens are there, a lane a box starts a TMA copy; else the warp copies by 16 bytes, with
    // zeros for the tokens that are not there.
    constexpr int CH = D / 8, ROWS = 32 / CH;
    const int lw = warp - 8;
    // keys and values leave L2 before the pieces of cut units, which the join reads again: trees of 3 to 16
    // 62 us, 66 without
    const uint64_t policy = tc::policy_evict_first();
    int n = 0;       // tiles issued
    int landed = 0;  // tiles whose arrival is made; those of TMA copies are made at once
    int units = 0;
    bool ok = true;
    auto land = [&](int upto) {
      tc::fence_proxy_async();
      for (; landed < upto; ++landed) tc::mbar_arrive(sh.bar(Plan::FULL + landed % NS));
    };
    // 32 rows of 16-byte pieces to rows lw * 32 .. of the tile at dst; lane r knows row r's source (null: zeros)
    auto copy_rows = [&](uint32_t dst, const T* mine) {
#pragma unroll 4
      for (int j = 0; j < 32 / ROWS; ++j) {
        const int r = j * ROWS + lane / CH, ch = lane % CH;
        const uint64_t src = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), r);
        cp_async_16(dst + (ch >> 3) * (kTcTile * 128) + tc::sw128(lw * 32 + r, (ch & 7) * 16),
                    reinterpret_cast<const T*>(src ? src : reinterpret_cast<uint64_t>(p.q)) + (src ? 8 * ch : 0), src != 0);
      }
    };
    for (; ok && w.any; w.next(p)) {
      const int R = w.s.n * p.group, left = R - w.qt * MT;  // rows of the unit: left, at most MT
      const int32_t* table = c.block_table + w.b * c.table_stride;
      const T* kbase = static_cast<const T*>(c.k) + w.kvh * c.k_head;
      const T* vbase = static_cast<const T*>(c.v) + w.kvh * c.v_head;
      auto load = [&](const CUtensorMap* map, const T* base, int64_t page_stride, int64_t token_stride, const TokenPlace& place) {
        const int slot = n % NS;
        if (n >= NS) ok = sh.wait_warp(Plan::FREE + slot, ((n / NS) - 1) & 1);
        if (!ok) return;
        const uint32_t dst = sbase + Plan::RING + slot * TILE;
        if (p.box && __all_sync(0xffffffffu, place.page >= 0)) {
          if (landed < n) {
            tc::cp_async_wait_all();
            land(n);
          }
          const uint32_t bar = sh.bar(Plan::FULL + slot);
          if (lane == 0) tc::mbar_arrive_expect_tx(bar, 32 * D * 2);
          else tc::mbar_arrive(bar);
          __syncwarp();
          constexpr int HALVES = D / 64;
          const int box = lane / HALVES, half = lane % HALVES, first = (box * p.box) & 31;
          const int page = __shfl_sync(0xffffffffu, place.page, first), at = __shfl_sync(0xffffffffu, place.place, first);
          if (box * p.box < 32)
            tc::tma_load_4d(dst + half * (kTcTile * 128) + (lw * 32 + first) * 128, map, 64 * half, w.kvh, at, page, bar, policy);
          ++n;
          ++landed;
          return;
        }
        copy_rows(dst, place.page >= 0 ? base + place.page * page_stride + place.place * token_stride : nullptr);
        tc::cp_async_commit();
        ++n;
        if (n - landed > LAG) {
          asm volatile("cp.async.wait_group %0;" ::"n"(LAG) : "memory");
          land(n - LAG);
        }
      };
      // the order of the tiles: K0, (Q), K1, V0, K2, V1, ..., V(n-1)
      TokenPlace next = token_place(p, table, w.t0 * kTcTile + lw * 32 + lane, w.s.len), prev = next;
      for (int t = w.t0; t <= w.t1 && ok; ++t) {
        const TokenPlace cur = next;
        next = token_place(p, table, (t + 1) * kTcTile + lw * 32 + lane, t + 1 < w.t1 ? w.s.len : 0);
        if (t < w.t1) load(&k_map, kbase, c.k_page, c.k_token, cur);
        if (t == w.t0 && ok) {  // the first tile is under way meanwhile
          ok = units == 0 || sh.wait_warp(Plan::Q_FREE, (units - 1) & 1);
          if (!ok) break;
#pragma unroll 1
          for (int y = 0; y < (left > kTcTile ? 2 : 1); ++y) {
            const int rr = y * kTcTile + lw * 32 + lane, row = w.qt * MT + rr, i = row / p.group;
            copy_rows(sbase + Plan::Q + y * TILE,
                      rr < left ? static_cast<const T*>(p.q) + (static_cast<int64_t>(w.s.first) + i) * p.q_stride +
                                      static_cast<int64_t>(w.kvh * p.group + row - i * p.group) * D
                                : nullptr);
          }
          tc::cp_async_commit();
          tc::cp_async_wait_all();
          land(n);
          tc::mbar_arrive(sh.bar(Plan::Q_FULL));
          ++units;
        }
        if (t > w.t0 && ok) load(&v_map, vbase, c.v_page, c.v_token, prev);
        prev = cur;
      }
    }
    tc::cp_async_wait_all();
    if (ok) land(n);
  } else {
    // ---- products --------------------------------------------------------------------------
    // The whole warp walks and waits, and one elected thread issues: the descriptors then stay in
    // uniform registers. (With a lane-0 branch around it all, an MMA took 160 cycles to issue,
    // 2.5 times its own 64.)
    constexpr uint32_t fmt = std::is_same<T, __half>::value ? tc::kF16 : tc::kBF16;
    constexpr uint32_t id_s = tc::idesc_f16(128, kTcTile, fmt, false, false), id_o = tc::idesc_f16(128, D, fmt, false, true);
    int base = 0;
    uint32_t q_ph = 0, p_ph = 0;  // p_ph: a bit a stream
    bool ok = true;
    for (; ok && w.any; w.next(p)) {
      const int n = w.t1 - w.t0;
      const bool split = w.s.n * p.group - w.qt * MT <= kTcTile;
      ok = sh.wait_warp(Plan::Q_FULL, q_ph);
      q_ph ^= 1;
      auto scores = [&](int x, int j) {
        if (!ok) return;
        const int at = base + (j == 0 ? 0 : 2 * j - 1), slot = at % NS;
        ok = sh.wait_warp(Plan::FULL + slot, (at / NS) & 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t a = tc::desc_sw128(sbase + Plan::Q + (split ? 0 : x * TILE), 16, 1024);
        const uint64_t b = tc::desc_sw128(sbase + Plan::RING + slot * TILE, 16, 1024);
        const uint32_t d = tmem + Plan::COL_S + x * kTcTile;
        const bool last = split || x == 1;  // of the stream(s) that use the tile
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (kTcTile * 128) + (k & 3) * 32) >> 4;
            tc::mma_f16(d, a + off, b + off, id_s, k > 0);
          }
          tc::mma_commit(sh.bar(Plan::S_FULL + x));
          if (last) tc::mma_commit(sh.bar(Plan::FREE + slot));
          if (last && j == n - 1) tc::mma_commit(sh.bar(Plan::Q_FREE));
        }
        __syncwarp();
      };
      auto values = [&](int x, int j) {
        if (!ok) return;
        const int at = base + (j == n - 1 ? 2 * n - 1 : 2 * j + 2), slot = at % NS;
        ok = sh.wait_warp(Plan::FULL + slot, (at / NS) & 1) && sh.wait_warp(Plan::P_FULL + x, (p_ph >> x) & 1);
        p_ph ^= 1u << x;
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t b = tc::desc_sw128(sbase + Plan::RING + slot * TILE, kTcTile * 128, 1024);
        const uint32_t d = tmem + Plan::COL_O + x * D, a = tmem + Plan::COL_S + x * kTcTile;
        const bool first = split ? j < 2 : j == 0;
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < kTcTile / 16; ++k) tc::mma_f16_ts(d, a + 8 * k, b + ((k * 2048) >> 4), id_o, !first || k > 0);
          if (split || x == 1) tc::mma_commit(sh.bar(Plan::FREE + slot));
          if (split ? j + 2 >= n : j == n - 1) tc::mma_commit(sh.bar(Plan::O_FULL + x));
          if (split && n == 1) tc::mma_commit(sh.bar(Plan::O_FULL + 1));  // a stream without tiles is told too
        }
        __syncwarp();
      };
      if (split) {
        scores(0, 0);
        if (n > 1) scores(1, 1);
        for (int j = 0; j < n && ok; ++j) {
          values(j & 1, j);
          if (j + 2 < n) scores(j & 1, j + 2);
        }
      } else {
        scores(0, 0);
        scores(1, 0);
        for (int j = 0; j < n && ok; ++j)
          for (int x = 0; x < 2; ++x) {
            values(x, j);
            if (j + 1 < n) scores(x, j + 1);
          }
      }
      base += 2 * n;
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (s_abort) {  // products and copies in flight land before the memory is given up
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (warp == 12) tc::tmem_dealloc(tmem, Plan::TMEM_COLS);
}

}  // namespace gdn
