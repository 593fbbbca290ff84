// Attention of larger drafted trees and prompt chunks over a paged cache on the 5th-generation tensor
// cores, for sm_103a.
//
// With R query rows a kv head the operator does R flops a byte of the cache, so from some tens of
// rows on the register products of gdn_attn_kernel bound it, and from about 256 rows the tensor
// cores' rate does. A CTA works on two score streams x = 0, 1, each with 128 query rows and its own
// accumulators in tensor memory, and takes tiles of 128 tokens:
//
//     S_x = Q_x K^T (tcgen05)  ->  four warps: running maximum m, P = 2^(S c - m c), sum l
//     O_x += P V  (tcgen05, P from tensor memory, where it takes the place of S_x)
//
// so that the products of one stream run while the warps of the other take exponentials.
// Two ways to feed the streams:
//   kSplit = false: 256 rows, both streams on every token tile; one load of K and V for 256 rows.
//   kSplit = true : up to 128 rows, the streams on alternate token tiles of the same rows; their
//                   (m, l, O) are added up at the unit's end.
// O stays unnormalised in tensor memory. It is scaled down only when a row's maximum has grown by
// more than 2^8 since its last reference: until then P <= 2^8 relative to the reference, which
// costs no precision in fp32 and 16-bit floats (their relative error does not depend on the size;
// 2^8 is far inside fp16's range), and most tiles skip the round trip through the registers.
//
// Roles: warps 0-3 and 4-7 one stream each; warps 8-11 copy K and V tiles (TMA boxes
// inside the pages, or 16-byte cp.async for any page size; 128-byte-swizzled rows) through a ring of
// STAGES tiles; a thread of warp 12 issues the
// products. The hand-offs are mbarriers; every wait is bounded, and when one expires the status
// word says so and all roles run out.
#pragma once
#include "gdn_attn_kernel.cuh"

namespace gdn {

constexpr int kTcTile = 128;  // tokens of a tile, and rows of a stream
constexpr int kTcThreads = 416;
constexpr float kTcGrowth = 8.f;  // log2 of the growth of a maximum that O is not scaled for

template <int D>
struct AttnTcPlan {
  static constexpr int TILE = kTcTile * D * 2;  // Q of a stream, or a tile of K or V
  // the ring: as many tiles as fit beside Q; with D = 64 enough to keep the CTA alone on its SM,
  // since it takes all of the tensor memory
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int LAG = 2;  // copies in flight behind the one just issued
  static constexpr int Q = 0;
  static constexpr int RING = 2 * TILE;
  static constexpr int BYTES = RING + STAGES * TILE;
  static constexpr int DYN_SMEM = BYTES + 1024;  // slack for 1024-byte alignment
  static constexpr uint32_t COL_S = 0, COL_O = 256, TMEM_COLS = 512;
  // mbarriers
  static constexpr int FULL = 0, FREE = STAGES, S_FULL = 2 * STAGES, P_FULL = S_FULL + 2, O_FULL = P_FULL + 2,
                       Q_FULL = O_FULL + 2, X_FULL = Q_FULL + 1, X_FREE = X_FULL + 1, NBAR = X_FREE + 1;
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

struct TcShared {
  uint32_t bars;  // shared address of the mbarriers
  volatile uint32_t* abort;
  unsigned* status;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // Bounded wait of one thread.
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    if (tc::mbar_try_wait(bar(i), parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait_hint(bar(i), parity, 100000u)) {
      if (*abort) return false;
      if (tc::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
    return true;
  }
  // The same by a whole warp, with one answer.
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(i, parity));
  }
};

template <typename T, int D, bool kSplit>
__global__ void __launch_bounds__(kTcThreads, 1)
gdn_attn_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const AttnParams p) {
  using Plan = AttnTcPlan<D>;
  constexpr int MT = kSplit ? kTcTile : 2 * kTcTile, TILE = Plan::TILE, NS = Plan::STAGES, LAG = Plan::LAG;
  extern __shared__ uint8_t dyn[];
  __shared__ int64_t s_scan[kTcThreads / 32];
  __shared__ AttnStart s_start;
  __shared__ __align__(8) uint64_t s_bar[Plan::NBAR];
  __shared__ uint32_t s_tmem, s_abort;
  __shared__ float s_ml[2][kTcTile];
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
    tc::mbar_init(sh.bar(Plan::Q_FULL), 256);
    tc::mbar_init(sh.bar(Plan::X_FULL), 128);
    tc::mbar_init(sh.bar(Plan::X_FREE), 128);
    tc::mbar_fence_init();
    if (!p.whole) p.cut[run] = make_int4(0, 0, 0, -1);
  }
  if (warp == 12) tc::tmem_alloc(tc::smem_u32(&s_tmem), Plan::TMEM_COLS);
  tc::fence_before_sync();
  const AttnStart st = attn_start<MT, kTcTile, kTcThreads>(p, run, s_scan, &s_start);
  tc::fence_after_sync();
  tc::allow_dependent_launch();  // the join waits for this grid's end before it reads anything
  const uint32_t tmem = s_tmem;
  AttnWalk<MT, kTcTile> w(st);

  if (warp < 8) {
    // ---- one row a thread: softmax, and the unit's end -----------------------------------
    const int x = warp >> 2, lrow = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's quarter of the lanes
    const uint32_t s_addr = tmem + lanes + Plan::COL_S + x * kTcTile, o_addr = tmem + lanes + Plan::COL_O + x * D;
    const float cl = p.scale_log2;
    uint32_t s_ph = 0, o_ph = 0;
    bool ok = true;
    while (ok && w.next(p)) {
      const AttnSeq& s = w.s;
      const int R = s.n * p.group, row = w.qt * MT + (kSplit ? 0 : x * kTcTile) + lrow;
      const bool has = row < R;
      const int i = has ? row / p.group : 0, g = has ? row - i * p.group : 0;
      const int64_t head = (static_cast<int64_t>(s.first) + i) * p.q_stride + static_cast<int64_t>(w.kvh * p.group + g) * D;
      {  // the row of Q (of its stream; or half of it each, where the streams share the rows)
        constexpr int PER = kSplit ? D / 16 : D / 8;
        uint8_t* q = smem + Plan::Q + (kSplit ? 0 : x * TILE);
        const int c0 = kSplit ? x * PER : 0;
        uint4 v[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
          v[j] = has ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + head + 8 * (c0 + j)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < PER; ++j)
          *reinterpret_cast<uint4*>(q + ((c0 + j) >> 3) * (kTcTile * 128) + tc::sw128(lrow, ((c0 + j) & 7) * 16)) = v[j];
        tc::fence_proxy_async();
        tc::mbar_arrive(sh.bar(Plan::Q_FULL));
      }
      const bool used = __any_sync(0xffffffffu, has);                       // any row of the warp
      const bool mine = kSplit ? w.t0 + x < w.t1 : w.qt * MT + x * kTcTile < R;  // any tile of the stream
      float m = -INFINITY, l = 0.f;
      for (int t = w.t0 + (kSplit ? x : 0); mine && t < w.t1; t += kSplit ? 2 : 1) {
        ok = sh.wait_warp(Plan::S_FULL + x, s_ph);
        s_ph ^= 1;
        if (!ok) break;
        tc::fence_after_sync();
        if (used) {
          const int tok = t * kTcTile;
          const bool tail = tok + kTcTile > s.ctx || tok + kTcTile > s.len;
          uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t r[32];
          if (tail) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              vis[k] = sees32(p, s, i, tok + 32 * k);
              tc::tmem_ld32(s_addr + 32 * k, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], (vis[k] >> e) & 1 ? __uint_as_float(r[e]) : -INFINITY);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tc::tmem_ld32(s_addr + 32 * k, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(r[e]));
            }
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // a new reference for the row where its maximum has outgrown the old one (or there is none)
          const bool grown = top * cl > m * cl + kTcGrowth, fresh = m == -INFINITY;
          if (__any_sync(0xffffffffu, grown && !fresh)) {
            const float f = grown && !fresh ? exp2_approx((m - top) * cl) : 1.f;
            l *= f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              tc::tmem_ld32(o_addr + 32 * k, r);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tc::tmem_st32(o_addr + 32 * k, r);
            }
          }
          if (grown || fresh) m = top;
          const float nb = m == -INFINITY ? 0.f : -m * cl;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            tc::tmem_ld32(s_addr + 32 * k, r);
            tc::tmem_ld_wait();
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a = exp2_approx(fmaf(__uint_as_float(r[e]), cl, nb));
              float b = exp2_approx(fmaf(__uint_as_float(r[e + 1]), cl, nb));
              if (tail) {
                a = (vis[k] >> e) & 1 ? a : 0.f;
                b = (vis[k] >> (e + 1)) & 1 ? b : 0.f;
              }
              sum[(e >> 1) & 3] += a + b;
              pk[e >> 1] = pack2<T>(a, b);
            }
            tc::tmem_st16u(s_addr + 16 * k, pk);  // over the part of S that has been read
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tc::tmem_st_wait();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sh.bar(Plan::P_FULL + x));
      }
      if (!ok) break;
      ok = sh.wait_warp(Plan::O_FULL + x, o_ph);
      o_ph ^= 1;
      if (!ok) break;
      tc::fence_after_sync();
      // ---- the unit's end: the row out, or a piece of it into the workspace
      const bool whole = w.t0 == 0 && w.t1 == s.tiles, two = kSplit && w.t0 + 1 < w.t1;
      const int64_t part = (static_cast<int64_t>(run) * 2 + (w.t0 == 0 ? 1 : 0)) * MT + (kSplit ? 0 : x * kTcTile) + lrow;
      T* out = static_cast<T*>(p.out) + (static_cast<int64_t>(s.first) + i) * p.out_stride +
               static_cast<int64_t>(w.kvh * p.group + g) * D;
      float mm = m, ll = l, f0 = 1.f, f1 = 0.f;
      constexpr int HALF = D / 2;  // columns that the second stream hands over at a time
      float* xch = reinterpret_cast<float*>(smem + TILE);  // [HALF][128]
      if (two) {
        if (x == 1) {
          s_ml[0][lrow] = m;
          s_ml[1][lrow] = l;
        }
      }
      auto write32 = [&](int col, const float* a, float inv) {  // 32 columns of the row
        if (!has) return;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(out + col + e) =
                make_uint4(pack2<T>(a[e] * inv, a[e + 1] * inv), pack2<T>(a[e + 2] * inv, a[e + 3] * inv),
                           pack2<T>(a[e + 4] * inv, a[e + 5] * inv), pack2<T>(a[e + 6] * inv, a[e + 7] * inv));
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(p.part_o + part * D + col + e) = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
        }
      };
#pragma unroll 1
      for (int h = 0; h < 2 && ok; ++h) {
        if (two && x == 1) {
          if (h == 1) {  // the first half has been taken
            ok = sh.wait_warp(Plan::X_FREE, 0);  // two phases a unit
            if (!ok) break;
          }
#pragma unroll
          for (int k = 0; k < HALF / 32; ++k) {
            uint32_t r[32];
            tc::tmem_ld32(o_addr + h * HALF + 32 * k, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) xch[(32 * k + e) * kTcTile + lrow] = __uint_as_float(r[e]);
          }
          tc::mbar_arrive(sh.bar(Plan::X_FULL));
        } else if (mine && !(kSplit && x == 1)) {
          if (two) {
            ok = sh.wait_warp(Plan::X_FULL, h);
            if (!ok) break;
            if (h == 0) {
              const float m1 = s_ml[0][lrow];
              mm = fmaxf(m, m1);
              const float base = mm == -INFINITY ? 0.f : mm;
              f0 = exp2_approx((m - base) * cl);
              f1 = exp2_approx((m1 - base) * cl);
              ll = l * f0 + s_ml[1][lrow] * f1;
            }
          }
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll
          for (int k = 0; k < HALF / 32; ++k) {
            uint32_t r[32];
            float a[32];
            tc::tmem_ld32(o_addr + h * HALF + 32 * k, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              a[e] = __uint_as_float(r[e]);
              if (two) a[e] = a[e] * f0 + xch[(32 * k + e) * kTcTile + lrow] * f1;
            }
            write32(h * HALF + 32 * k, a, inv);
          }
          if (two) tc::mbar_arrive(sh.bar(Plan::X_FREE));
        }
      }
      if (!ok) break;
      if (two) {
        // the streams leave together: Q and the hand-over space are free for both
        ok = sh.wait_warp(Plan::X_FREE, 1);
        if (!ok) break;
      }
      if (has && !whole && mine && (!kSplit || x == 0)) {
        p.part_ml[part * 2] = mm == -INFINITY ? mm : mm * cl;  // in units of log2 e, as the join takes them
        p.part_ml[part * 2 + 1] = ll;
      }
      if (threadIdx.x == 0 && w.t0 == 0 && w.t1 < s.tiles)
        p.cut[run] = make_int4(s.first, s.n, w.unit, run_of(st.end + (s.tiles - w.t1) - 1, st.total, st.runs));
    }
  } else if (warp < 12) {
    // ---- copies of K and V -----------------------------------------------------------------
    constexpr int CH = D / 8, ROWS = 32 / CH;
    // A warp copies 32 tokens of every tile. Where a page holds whole boxes of p.box tokens and all
    // 32 tokens are there, a lane a box starts a TMA copy; else the warp copies by 16 bytes, with
    // zeros for the tokens that are not there.
    const int lw = warp - 8;
    int n = 0;       // tiles issued
    int landed = 0;  // tiles whose arrival is made; those of TMA copies are made at once
    bool ok = true;
    auto land = [&](int upto) {
      tc::fence_proxy_async();
      for (; landed < upto; ++landed) tc::mbar_arrive(sh.bar(Plan::FULL + landed % NS));
    };
    while (ok && w.next(p)) {
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
          const int box = lane / HALVES, half = lane % HALVES, first = box * p.box & 31;
          const int page = __shfl_sync(0xffffffffu, place.page, first), at = __shfl_sync(0xffffffffu, place.place, first);
          if (box * p.box < 32)
            tc::tma_load_4d(dst + half * (kTcTile * 128) + (lw * 32 + first) * 128, map, 64 * half, w.kvh, at, page, bar);
          ++n;
          ++landed;
          return;
        }
#pragma unroll 4
        for (int j = 0; j < 32 / ROWS; ++j) {
          const int r = j * ROWS + lane / CH, ch = lane % CH;
          const int page = __shfl_sync(0xffffffffu, place.page, r), at = __shfl_sync(0xffffffffu, place.place, r);
          const bool real = page >= 0;
          cp_async_16(dst + (ch >> 3) * (kTcTile * 128) + tc::sw128(lw * 32 + r, (ch & 7) * 16),
                      base + (real ? page : 0) * page_stride + at * token_stride + 8 * ch, real);
        }
        tc::cp_async_commit();
        ++n;
        if (n - landed > LAG) {
          asm volatile("cp.async.wait_group %0;" ::"n"(LAG) : "memory");
          land(n - LAG);
        }
      };
      TokenPlace next = token_place(p, table, w.t0 * kTcTile + lw * 32 + lane, w.s.len), prev = next;
      for (int t = w.t0; t <= w.t1 && ok; ++t) {
        const TokenPlace cur = next;
        next = token_place(p, table, (t + 1) * kTcTile + lw * 32 + lane, t + 1 < w.t1 ? w.s.len : 0);
        if (t < w.t1) load(&k_map, kbase, c.k_page, c.k_token, cur);
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
    while (ok && w.next(p)) {
      const int n = w.t1 - w.t0;
      const int streams = kSplit ? 2 : (w.qt * MT + kTcTile < w.s.n * p.group ? 2 : 1);
      ok = sh.wait_warp(Plan::Q_FULL, q_ph);
      q_ph ^= 1;
      // tiles are loaded in the order K0, K1, V0, K2, V1, ..., V(n-1)
      auto scores = [&](int x, int j) {
        if (!ok) return;
        const int at = base + (j == 0 ? 0 : 2 * j - 1), slot = at % NS;
        ok = sh.wait_warp(Plan::FULL + slot, (at / NS) & 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t a = tc::desc_sw128(sbase + Plan::Q + (kSplit ? 0 : x * TILE), 16, 1024);
        const uint64_t b = tc::desc_sw128(sbase + Plan::RING + slot * TILE, 16, 1024);
        const uint32_t d = tmem + Plan::COL_S + x * kTcTile;
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * (kTcTile * 128) + (k & 3) * 32) >> 4;
            tc::mma_f16(d, a + off, b + off, id_s, k > 0);
          }
          tc::mma_commit(sh.bar(Plan::S_FULL + x));
          if (kSplit || x == streams - 1) tc::mma_commit(sh.bar(Plan::FREE + slot));
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
        const bool first = kSplit ? j < 2 : j == 0;
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < kTcTile / 16; ++k) tc::mma_f16_ts(d, a + 8 * k, b + ((k * 2048) >> 4), id_o, !first || k > 0);
          if (kSplit || x == streams - 1) tc::mma_commit(sh.bar(Plan::FREE + slot));
          if (kSplit ? j + 2 >= n : j == n - 1) tc::mma_commit(sh.bar(Plan::O_FULL + x));
          // a stream without tiles is told too: it must not run ahead into the next unit's Q
          if (kSplit ? n == 1 : streams == 1 && j == n - 1) tc::mma_commit(sh.bar(Plan::O_FULL + 1));
        }
        __syncwarp();
      };
      if (kSplit) {
        scores(0, 0);
        if (n > 1) scores(1, 1);
        for (int j = 0; j < n && ok; ++j) {
          values(j & 1, j);
          if (j + 2 < n) scores(j & 1, j + 2);
        }
      } else {
        for (int x = 0; x < streams; ++x) scores(x, 0);
        for (int j = 0; j < n && ok; ++j)
          for (int x = 0; x < streams; ++x) {
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
