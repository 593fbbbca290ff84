// Shared parts of the attention kernels over a paged cache: the split of the work over the
// CTAs and the join of its parts.
//
// A unit is one tile of query rows of one (sequence, kv head). The rows of a kv head are
// r = i (nq / nkv) + g for new token i and head g of its group, so that all heads that read
// a key share its load. A unit walks its sequence's tokens in tiles of KT. The CTAs are dealt
// out to members, by their work: member j of J (J = the most row tiles of a kv head, at most 8)
// has the row tiles j, j + J, ... So CTAs that read the same keys for different rows run side by
// side, and the second read finds them in L2. (In one order over (sequence, kv head, row tile) the
// row tiles of a kv head came one after the other: with two of them every key came from HBM twice.)
// A member's tiles in a row, (sequence, kv head, row tile, token tile), are cut into as many equal
// runs as it has CTAs: the load is even whatever the lengths, one long sequence fills the
// card, and no length is needed on the host. A unit that lies in one run is written by it. A
// unit that is cut leaves a partial (m, l, o) of every piece in the workspace,
//
//     m = max_t x_t,   l = sum_t 2^(x_t - m),   o = sum_t 2^(x_t - m) v_t
//
// (x in units of log2 e, m any reference near the maximum; l and o times 2^kWeightLog2), and
// gdn_attn_join_kernel adds the pieces up in their order, with weights 2^(m_piece - max m). A run has at most two cut units, its
// first (slot 0) and its last (slot 1), so the workspace does not grow with the batch. Where the
// units are short and many the runs are cut at units and the join falls away.
#pragma once
#include "gdn_norm_rope_kernel.cuh"

namespace gdn {

struct AttnParams {
  const void* q;
  void* out;
  PagedParams cache;
  const uint64_t* mask;  // [rows][mask_words] or null
  int mask_words;
  int nq, nkv, group;
  float scale_log2;  // scale * log2 e
  int64_t q_stride, out_stride;
  int out_wide;    // out's head rows lie on 32-byte boundaries
  int runs;        // CTAs of the attention kernel
  int box;         // tokens of a TMA box inside a page, 0: pages do not hold whole boxes
  int whole;       // runs are cut at units only: nothing to join
  float* part_ml;  // [runs][2][MT][2]: m and l
  float* part_o;   // [runs][2][D / 8][MT][8]
  int4* cut;       // [runs]: the unit that begins in the run and is cut (AttnWalk::cut; w < 0: none)
  unsigned* status;
};

struct AttnSeq {
  int first, n;  // its new rows
  int ctx, len;  // tokens before them, and with them (as many as the table holds)
  int tiles;     // token tiles, at least 1
  int qtiles;    // row tiles of a kv head
};

template <int MT, int KT>
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b, bool report) {
  const PagedParams& c = p.cache;
  AttnSeq s;
  s.first = c.cu_rows ? c.cu_rows[b] : b;
  const int end = c.cu_rows ? c.cu_rows[b + 1] : b + 1;
  s.ctx = c.ctx_lens[b];
  s.n = end - s.first;
  const bool ends = !c.cu_rows || ((b != 0 || s.first == 0) && (b != c.B - 1 || end == c.rows));
  if (s.first < 0 || end < s.first || end > c.rows || s.ctx < 0 || !ends) {
    if (report) atomicOr(p.status, kStatusBadSeqlens);
    if (s.first < 0 || end < s.first || end > c.rows || s.ctx < 0) s.n = s.ctx = 0;
  }
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page_size;  // < 2^31
  int64_t len = static_cast<int64_t>(s.ctx) + s.n;
  if (len > cap) {
    if (report && s.n > 0) atomicOr(p.status, kStatusBadPage);
    len = cap;
  }
  s.len = static_cast<int>(len);
  s.tiles = s.len > 0 ? (s.len + KT - 1) / KT : 1;
  s.qtiles = (s.n * p.group + MT - 1) / MT;
  return s;
}

constexpr int kAttnMembers = 8;

// Row tiles of a kv head that member j of `members` has.
__device__ __forceinline__ int attn_member_tiles(const AttnSeq& s, int j, int members) {
  return s.qtiles > j ? (s.qtiles - j - 1) / members + 1 : 0;
}

// What the start and the end of a unit cost (its Q, first pages and tiles, its rows out), in tokens. The
// runs count it in front of the unit's own; without it those with many short units end last: one token
// of 64 sequences of 100 to 16000 348 us, with 128 to 512 tokens 337, 333, 332, 332; trees of 3 to 16
// 60.4, 58.8, 58.4, 58.4, 58.7.
constexpr int kAttnUnitTokens = 384;

// What the runs count: token tiles and units' starts, or units.
template <int KT>
__device__ __forceinline__ int64_t attn_cost(const AttnParams& p, const AttnSeq& s, int j, int members) {
  return static_cast<int64_t>(p.whole ? 1 : s.tiles + kAttnUnitTokens / KT) * attn_member_tiles(s, j, members) * p.nkv;
}

// The same as time, by which the members get their CTAs: in gdn_attn_tc_kernel a tile costs a
// row tile that fills more than one stream about 3/2 of another (3000 and 1950 cycles).
template <int MT, int KT>
__device__ __forceinline__ int64_t attn_weight(const AttnParams& p, const AttnSeq& s, int j, int members) {
  const int64_t cost = attn_cost<KT>(p, s, j, members);
  if (MT <= KT || cost == 0) return cost;
  const int last = s.qtiles - 1;
  const bool small = last % members == j && s.n * p.group - last * MT <= MT / 2;
  return 3 * cost - (small ? attn_cost<KT>(p, s, last, last + 1) : 0);
}

// Inclusive prefix of `x` over the warp, and the sum over it.
__device__ __forceinline__ int64_t warp_prefix(int64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// a * b / c for a, c >= 0, b > 0, in 32 bits where that holds the product.
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  const uint64_t x = static_cast<uint64_t>(a) * static_cast<uint64_t>(b);
  return (x | static_cast<uint64_t>(c)) >> 32 ? static_cast<int64_t>(x / static_cast<uint64_t>(c))
                                              : static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(c));
}

// Where a run starts: sequence, unit and tile of it, and how many tiles it has.
struct AttnStart {
  int b;
  int member, members;
  int64_t within;      // tiles of sequence b before the run
  int64_t end, total;  // the member's tiles up to the run's end, and in all
  int64_t count;       // tiles of the run
  int first, runs;     // the member's first run, and its runs that have tiles
};

// Run i of `runs` has the tiles [total i / runs, total (i + 1) / runs).
__device__ __forceinline__ int64_t run_begin(int64_t i, int64_t total, int runs) { return mul_div(total, i, runs); }

// The run that holds tile `at`.
__device__ __forceinline__ int run_of(int64_t at, int64_t total, int runs) {
  int64_t i = mul_div(at, runs, total);
  while (run_begin(i + 1, total, runs) <= at) ++i;
  while (run_begin(i, total, runs) > at) --i;
  return static_cast<int>(i);
}

// Where the block's run starts, found by one warp, a lane a sequence (the block's barrier after its
// set-up is then the only one; a search by all threads took several).
template <int MT, int KT>
__device__ __forceinline__ AttnStart attn_start(const AttnParams& p, int run) {
  const int B = p.cache.B, lane = threadIdx.x & 31;
  const bool report = run == 0;
  // the most row tiles, and all members' weight
  int most = 0;
  int64_t work = 0;
  AttnSeq own{};  // this lane's sequence, where there are at most 32
#pragma unroll 4
  for (int b = lane; b < B; b += 32) {
    own = attn_seq<MT, KT>(p, b, report);
    most = own.qtiles > most ? own.qtiles : most;
    work += attn_weight<MT, KT>(p, own, 0, 1);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const int64_t all = warp_sum(work);
  const int members = most < kAttnMembers ? most : kAttnMembers;
  // member j has the runs j + floor((p.runs - members) weight of members < j / all) and on, at least one
  int64_t before = 0, total = 0;
  int member = 0, first = 0, next = p.runs;
  if (members == 1) {
    int64_t cost = 0;
    for (int b = lane; b < B; b += 32) cost += attn_cost<KT>(p, B <= 32 ? own : attn_seq<MT, KT>(p, b, false), 0, 1);
    total = warp_sum(cost);
  } else {
    for (int j = 0; j < members; ++j) {
      int64_t weight = 0, cost = 0;
      for (int b = lane; b < B; b += 32) {
        const AttnSeq s = B <= 32 ? own : attn_seq<MT, KT>(p, b, false);
        weight += attn_weight<MT, KT>(p, s, j, members);
        cost += attn_cost<KT>(p, s, j, members);
      }
      total = warp_sum(cost);
      const int begin = j + static_cast<int>(mul_div(before, p.runs - members, all));
      before += warp_sum(weight);
      const int end = j + 1 + static_cast<int>(mul_div(before, p.runs - members, all));
      if (run >= begin && run < end) {
        member = j;
        first = begin;
        next = end;
        break;
      }
    }
  }
  const int runs = total < next - first ? static_cast<int>(total) : next - first;  // no run is empty
  AttnStart st{0, member, members, 0, 0, total, 0, first, runs};
  if (run - first >= runs) return st;
  const int64_t begin = run_begin(run - first, total, runs);
  st.end = run_begin(run - first + 1, total, runs);
  st.count = st.end - begin;
  int64_t upto = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int64_t cost = 0;
    if (b0 + lane < B) cost = attn_cost<KT>(p, B <= 32 ? own : attn_seq<MT, KT>(p, b0 + lane, false), member, members);
    const int64_t end_b = upto + warp_prefix(cost);
    const unsigned m = __ballot_sync(0xffffffffu, end_b > begin);
    if (m) {  // the first sequence that ends behind the run's first tile
      const int l = __ffs(m) - 1;
      st.b = b0 + l;
      st.within = begin - __shfl_sync(0xffffffffu, end_b - cost, l);
      break;
    }
    upto = __shfl_sync(0xffffffffu, end_b, 31);
  }
  return st;
}

// Walks a run: the unit pieces in their order. The warp that has found the start takes the first
// step; then every thread of a role walks by itself.
template <int MT, int KT>
struct AttnWalk {
  AttnStart st;
  int b;
  int64_t within, left;
  bool any;    // there is a piece
  AttnSeq s;   // its sequence
  int kvh, qt;
  int t0, t1;  // its token tiles
  __device__ __forceinline__ void begin(const AttnParams& p, const AttnStart& start) {
    st = start;
    b = st.b;
    within = st.within;
    left = st.count;
    next(p);
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    const int member = st.member, members = st.members;
    while (left > 0) {
      s = attn_seq<MT, KT>(p, b, false);
      const int64_t cost = attn_cost<KT>(p, s, member, members);
      if (within >= cost) {
        within -= cost;
        ++b;
        continue;
      }
      int unit;
      if (p.whole) {
        unit = static_cast<int>(within);
        t0 = 0;
        t1 = s.tiles;
        ++within;
        --left;
      } else {
        const int span = s.tiles + kAttnUnitTokens / KT;
        unit = within >> 32 ? static_cast<int>(within / span) : static_cast<int>(static_cast<uint32_t>(within) / static_cast<uint32_t>(span));
        const int at = static_cast<int>(within - static_cast<int64_t>(unit) * span);
        const int take = left < span - at ? static_cast<int>(left) : span - at;
        within += take;
        left -= take;
        t0 = at > kAttnUnitTokens / KT ? at - kAttnUnitTokens / KT : 0;
        t1 = at + take - kAttnUnitTokens / KT;
        if (t1 <= t0) continue;  // the run ends in front of the unit's first tile
      }
      const int mine = attn_member_tiles(s, member, members);
      kvh = unit / mine;
      qt = (unit - kvh * mine) * members + member;
      any = true;
      return;
    }
    any = false;
  }
  // What the join has to know where the unit begins in run `run` and is cut: the sequence's first row, kv
  // head, first of its rows there, and the rows of the unit (from bit 16) with the last run.
  __device__ __forceinline__ int4 cut(const AttnParams& p) const {
    const int left = s.n * p.group - qt * MT;
    return make_int4(s.first, kvh, qt * MT,
                     (left < MT ? left : MT) << 16 | (st.first + run_of(st.end + (s.tiles - t1) - 1, st.total, st.runs)));
  }
};

// ---- 16-bit element types ---------------------------------------------------------------
// The weights 2^(x - m) are rounded to the cache's type for the second product, the only form in which the
// tensor cores take them beside 16-bit values; l sums them in fp32 before. That costs up to 2^-8 (bf16) or
// 2^-11 (fp16) of a weight: against 64 bits the output of 64 drafted rows over 32768 is off by 2.3e-3 of its
// size in bf16, 1.7e-3 if it were rounded only once. fp16 also has few exponents: as numbers up to 1, weights
// below 2^-14 lose bits and those below 2^-25 are gone, and a row may have 10^5 of them. So all of a row's
// weights, and with them l and o, are 2^kWeightLog2 times as large, which the division by l takes out
// again; what is gone then is below 2^-31 of the largest. The rest of fp16's 2^16 is for what a weight may
// exceed 1 by (2^8, with the tensor-core kernel's old references) and a factor of 4 for the rounding of
// exponents, reached where |x| is 2^24 and fp32 holds a score itself to no more. 2^8, with references that
// are kept to 2^4 for it, took 38.6 instead of 36.7 us for 33 drafted rows over 65536 tokens.
template <typename T>
constexpr float kWeightLog2 = 0.f;
template <>
constexpr float kWeightLog2<__half> = 6.f;

// 2^x on the special function unit (relative error about 2^-22; 0 for -inf).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- pieces of cut units ----------------------------------------------------------------
// A piece's o in the workspace: [D / 8][MT][8], so that threads with a row each write whole lines.
template <int MT>
__device__ __forceinline__ int attn_piece_at(int row, int col) {
  return ((col >> 3) * MT + row) * 8 + (col & 7);
}

// Adds U pieces to (m, l, o), in their order.
template <int U>
__device__ __forceinline__ void attn_join(const float2 (&ml)[U], const float4 (&v)[U], float& m, float& l, float4& o) {
  float mn = m;
#pragma unroll
  for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
  const float base = mn == -INFINITY ? 0.f : mn, f = exp2_approx(m - base);
  m = mn;
  l *= f;
  o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float g = exp2_approx(ml[u].x - base);
    l = fmaf(ml[u].y, g, l);
    o.x = fmaf(v[u].x, g, o.x);
    o.y = fmaf(v[u].y, g, o.y);
    o.z = fmaf(v[u].z, g, o.z);
    o.w = fmaf(v[u].w, g, o.w);
  }
}

}  // namespace gdn
