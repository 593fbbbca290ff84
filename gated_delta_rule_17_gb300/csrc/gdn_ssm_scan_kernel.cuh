// The scan over prompts in chunks of 128 tokens on the tensor cores (tcgen05), for sm_103a.
//
// Within a chunk, with g_t = d_t a, suf_t = sum of g over the chunk's tokens behind t, and total their sum:
//
//     o_i = e^{total - suf_i} q_i S + sum_{j <= i} (q_i . k_j) e^{suf_j - suf_i} d_j v_j + skip v_i
//     S  <- e^{total} S + sum_j k_j (d_j e^{suf_j} v_j)^T
//
// A unit is 64 value columns of a head, and a CTA takes two units of one key head (two halves of a head of
// 128, or two heads of 64) through a sequence, or a segment of one. Their products share the operands:
//
//     G = Q K^T (128 x 128)      once for both units
//     O2 = Q S16                 N = 128: both units side by side
//     O1 = A V                   A = G under the mask
//     L = K^T V'                 V' = d e^{suf} v as bf16 hi + lo, so that the fp32 state keeps 16 bits of it
//
// The decays need no exponential a pair (i, j): with V = V' (hi) and e^{-suf_i} on the rows of O1, A is
// the same for both heads, and bf16 has fp32's exponents. That holds while the chunk's decay stays within
// kSsmSpan. A head whose chunk decays further has an A of its own, with d_j e^{suf_j - suf_i}, and V = v: beside the diagonal as
// (d_j e^{suf_j - b}) e^{b - suf_i} about the decay b behind every 16 columns, where neither factor passes 1 or d, on it pair by pair; and
// O2's rows are scaled before O1 comes on top. Operands of 16 bits cost the output little beside its own rounding: it is off by 1.9e-3 of
// its size in the mean, 1.7e-3 if it were rounded only once; the state is off by 4e-6.
//
// Roles: warps 0-7, a thread a row of S and of the outputs (warps 0-3 unit 0, 4-7 unit 1), S in registers; warps 8-15 make
// the operands, V' of their unit and half of A; warp 16 copies Q and K (TMA) and issues the products. Order on the tensor
// pipe: O2, L, O1 of a chunk, then G of the next. So the update of S, the only step that the next chunk's O2 waits
// for, runs under G, making A under O2, the rows' way out under L.
//
// 4 x 8192 tokens of 32 heads of 128 x 128 on 16: 188 us, 206 to 216 with a few heads whose chunks decay by more than kSsmSpan; HBM alone
// would take 122, the products at their least 35. There is a CTA for 128 of the 152 SMs, and a chunk takes it 2.9 us. The tensor pipe is
// busy for 29% of it, the issue slots for 43%, loads and stores keep shared memory for 40% and the products' operands (288 KB a chunk)
// and copies for as much again; the rest is the roles' hand-offs. Copies of v and x by rows instead of by TMA, rows out by plain stores, one buffer of K,
// and O begun from skip v each took 8% to half as long again. A segment's first pass takes 0.6 of the second's time.
#pragma once
#include <cstddef>
#include <type_traits>
#include "gdn_ssm_common.cuh"

namespace gdn {

constexpr int kSsmChunk = 128;
constexpr int kSsmThreads = 640;
// Registers of a thread by role. Five warpgroups are launched with 96 each, which they share out: 2 x 128 + 2 x 88 + 48 = 5 x 96.
constexpr int kSsmRowRegs = 128, kSsmOperandRegs = 88, kSsmIssueRegs = 48;
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Nats that a chunk may decay for its decays to go into its operands. These and their sums are then up to e^50 = 5.2e21 times above or below
// their size, which leaves 6.6e16 of fp32's range (and, below, of bf16's) to the sums of |q.k| d |v| and |k| d |v| over a chunk. With 140 nats,
// the most that values about one take, it would be 1.3e8, and values of a hundred would pass it. Fewer chunks are wide then: ragged prompts
// 411, 406, 419 us with 140 nats, 416, 422, 421 with 100, 422, 440, 421 with 80.
constexpr float kSsmSpan = 100.f;

// A CTA's part: a sequence, a segment of it, and the item of the sequence's first segment.
struct SsmPlace {
  int seq, seg, segs, first;
};

// What the roles tell one another beside tiles.
struct SsmSmall {
  uint64_t bar[22];
  alignas(16) float suf[2][kSsmChunk], d[2][kSsmChunk];  // of each unit's tokens
  float total[2][2];                         // by chunk parity: each unit's decay
  float behind[2][8];                        // in chunks of wide decay: log2 of the decay behind each 16 tokens
  uint32_t tmem, abort;
  SsmPlace place;
};

static_assert(offsetof(SsmSmall, suf) % 16 == 0 && offsetof(SsmSmall, d) % 16 == 0, "four tokens' are read and written at once");

struct SsmPlan {
  static constexpr int BLOCK = 128 * 128;  // 128 rows of 64 16-bit values
  static constexpr int Q = 0, K = 2 * BLOCK, VHI = K + 4 * BLOCK, VLO = VHI + 2 * BLOCK, S16 = VLO + 2 * BLOCK, ROWS = S16 + 2 * BLOCK,
                       SMALL = ROWS + 2 * BLOCK, DYN_SMEM = SMALL + static_cast<int>(sizeof(SsmSmall));
  static constexpr uint32_t COL_G = 0, COL_O = 128, COL_L = 384, TMEM_COLS = 512;  // O: a buffer of 128 for even and odd chunks
  // mbarriers: copies (Q_FULL, K_FULL + buffer, X_FULL + chunk parity, X_LANDED), products (G_FULL, Q_FREE, L_FULL, O_FULL + buffer) and
  // warps' signals. A wait by parity takes the phase before for its own unless that one is known to be over, and waits for ever where the
  // phase behind its own may be over too; so each role either waits for every phase of a barrier, or the comment at its wait says what
  // it knows them by.
  static constexpr int Q_FULL = 0, K_FULL = 1, G_FULL = 3, Q_FREE = 4, L_FULL = 5, X_FULL = 6, X_LANDED = 8, O_FULL = 9, GATES = 11, V_READY = 12,
                       A_READY = 13, S_READY = 14, GATES_READ = 15, STAGED = 16, O_READ = 17, STEPS_READ = 19, STEPS_SET = 20, NBAR = 22;
  static_assert(sizeof(SsmSmall::bar) == NBAR * 8 && SMALL % 16 == 0 && DYN_SMEM <= 227 * 1024, "");
  static __device__ __forceinline__ int arrivals(int i) { return i < GATES ? 1 : i == GATES ? 2 : i >= STEPS_SET ? 4 : 8; }
};

struct SsmScanParams {
  SsmParams s;
  int pairs;      // CTAs of a sequence, or of a segment of one
  int sms;
  int segment;    // chunks of a segment; 0: whole sequences
  float* states;  // segments: [item][nv][DK][DV], item i the state that segment i starts from: S_0 of the first, the end of the first from
                  // S_0, and behind it each segment's end from zero
  float* decays;  // [item][nv]: the decay over segment i, as a logarithm
};

// Found by one warp. Sequences go by themselves, packed ones the longest first, or (where `segment` is given, and the longest of them would
// keep most SMs waiting) in segments: then the state at the end of each segment but the last is worked out first, which takes a
// little over half of a segment's time again. The warp has a lane for a sequence, so that packed batches of more than 32 go in their given
// order and whole: a prompt of 32768 among 31 of 100, 8 heads of 128 x 64 on 2: 142 us, among 32 of them 675.
__device__ __forceinline__ SsmPlace ssm_place(const SsmScanParams& params, int item) {
  const Rows& b = params.s.batch;
  const int lane = threadIdx.x & 31, seg = params.segment;
  if (!b.cu) {
    const int n = seg ? ((b.T + kSsmChunk - 1) / kSsmChunk + seg - 1) / seg : 1;
    return {item / n, item % n, n, item - item % n};
  }
  if (b.B > 32) return {item < b.B ? item : -1, 0, 1, item};
  int chunks = 0;
  if (lane < b.B) {
    const int start = b.start(lane), end = b.end(lane);
    if (rows_held(start, end, b.rows)) chunks = (end - start + kSsmChunk - 1) / kSsmChunk;
  }
  const int longest = __reduce_max_sync(0xffffffffu, chunks), total = __reduce_add_sync(0xffffffffu, chunks);
  const float even = static_cast<float>(total) * params.pairs / params.sms, whole = fmaxf(even, longest);
  SsmPlace r{-1, 0, 1, item};
  unsigned found;
  if (seg && whole > 1.2f * (1.6f * even + 1.6f * seg + 4.f)) {
    const int n = (chunks + seg - 1) / seg;
    int before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before -= n;
    found = __ballot_sync(0xffffffffu, item >= before && item < before + n);
    const int src = found ? __ffs(found) - 1 : 0;
    r.first = __shfl_sync(0xffffffffu, before, src);
    r.segs = __shfl_sync(0xffffffffu, n, src);
    r.seg = item - r.first;
  } else {
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < 32; ++o) {
      const int other = __shfl_sync(0xffffffffu, chunks, o);
      rank += other > chunks || (other == chunks && o < lane);
    }
    found = __ballot_sync(0xffffffffu, rank == item);
  }
  r.seq = found && __ffs(found) - 1 < b.B ? __ffs(found) - 1 : -1;
  return r;
}

constexpr int kSsmWaits = 1 << 18;  // tries of up to 10 us each before a wait gives up

struct SsmShared {
  uint32_t bars;
  volatile uint32_t* abort;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  // Bounded wait by a whole warp, with one answer. A warp that gave up waits no more but walks on, and may then take another way than
  // its neighbours. So a barrier without a limit is one that a warp comes to as often whichever way it takes. (Counted, not timed: the
  // clock and a call cost every wait code, of which the roles share the instruction caches.)
  __device__ __forceinline__ void wait(int i, uint32_t parity, bool& ok) const {
    if (!ok) return;
    bool there = tc::mbar_try_wait(bar(i), parity);
#pragma unroll 1
    for (int k = 0; k < kSsmWaits && !there && !*abort; ++k) there = tc::mbar_try_wait_hint(bar(i), parity, 10000u);
    ok = __all_sync(0xffffffffu, there);
    if (!ok) *abort = 1;
  }
  __device__ __forceinline__ void arrive(int i) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar(i));
  }
};

// A value that the compiler takes to change, so that it does not write a role's loop twice for the two of a flag.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ float ssm_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Whether a unit's chunk decays by more than kSsmSpan (the same for all roles).
__device__ __forceinline__ bool ssm_wide(float total) { return !(total >= -kSsmSpan); }

// kOut false: the states at the ends of the segments, without outputs.
template <int DK, int DV, bool kOut>
__global__ void __launch_bounds__(kSsmThreads, 1)
gdn_ssm_scan_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap out_map,
                    const SsmScanParams params) {
  using P = SsmPlan;
  constexpr int SLICES = DV / 64, KB = DK / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = tc::smem_u32(smem);
  SsmSmall& small = *reinterpret_cast<SsmSmall*>(smem + P::SMALL);
  const SsmParams& p = params.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SsmShared sh{tc::smem_u32(small.bar), &small.abort};

  const int pair = static_cast<int>(blockIdx.x % static_cast<unsigned>(params.pairs)), item = static_cast<int>(blockIdx.x / static_cast<unsigned>(params.pairs));
  const int heads = p.nv / p.nk, units = heads * SLICES, per_key = (units + 1) / 2;  // of a key head
  const int kh = pair / per_key;
  tc::grid_dependency_wait();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.batch.B; i += kSsmThreads) p.batch.report(i, p.status);
  if (warp == 0) {
    const SsmPlace found = ssm_place(params, item);
    if (lane == 0) small.place = found;
  }
  __syncthreads();
  const SsmPlace place = small.place;
  if (place.seq < 0 || (!kOut && place.seg == place.segs - 1)) return;
  const int seq = place.seq, begin = p.batch.start(seq), end = p.batch.end(seq);
  if (!rows_held(begin, end, p.batch.rows) || begin == end) return;
  if (sbase & 1023) {  // the swizzle goes by the address; the alignment that smem is declared with gives it
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const int start = begin + place.seg * params.segment * kSsmChunk;
  const int tokens = place.seg < place.segs - 1 ? params.segment * kSsmChunk : end - start, chunks = (tokens + kSsmChunk - 1) / kSsmChunk;

  if (threadIdx.x == 0) {
    small.abort = 0;
    for (int i = 0; i < P::NBAR; ++i) tc::mbar_init(sh.bar(i), P::arrivals(i));
    tc::mbar_fence_init();
  }
  if (warp == 16) tc::tmem_alloc(tc::smem_u32(&small.tmem), P::TMEM_COLS);
  if (KB == 1)  // keys of 64: the products of K^T take 128 rows, the second half zeros
    for (int i = threadIdx.x; i < 2 * P::BLOCK / 16; i += kSsmThreads)
      *reinterpret_cast<uint4*>(smem + P::K + (i / (P::BLOCK / 16) * 2 + 1) * P::BLOCK + i % (P::BLOCK / 16) * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = small.tmem;
  bool ok = true;

  if (warp < 16) {
    const int group = warp >> 3, x = (warp >> 2) & 1, t = threadIdx.x & 127;  // the unit, and the row of it
    const int is_real = 2 * (pair % per_key) + x < units;
    const bool real = is_real;
    const int unit = 2 * (pair % per_key) + (real ? x : 0), h = kh * heads + unit / SLICES, col = h * DV + unit % SLICES * 64;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's quarter of the lanes
    if (group == 0) {
      // ---- a row of S, and of the outputs ------------------------------------------------
      more_registers<kSsmRowRegs>();
      const float skip = p.skip ? p.skip[h] : 0.f;
      const int64_t in_head = static_cast<int64_t>(t) * DV + unit % SLICES * 64;
      float* S = ssm_state<DK, DV>(p, seq, h) + in_head;
      auto kept = [&](int i) { return params.states + (static_cast<int64_t>(i) * p.nv + h) * (DK * DV) + in_head; };
      const bool held = real && t < DK;
      float s[64];
      auto load = [&](const float* from, float keep) {  // s keep + from
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(from + i);
          s[i] = fmaf(s[i], keep, v.x);
          s[i + 1] = fmaf(s[i + 1], keep, v.y);
          s[i + 2] = fmaf(s[i + 2], keep, v.z);
          s[i + 3] = fmaf(s[i + 3], keep, v.w);
        }
      };
      auto save = [&](float* to) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      };
#pragma unroll
      for (int i = 0; i < 64; ++i) s[i] = 0.f;
      if (held) {
        if constexpr (kOut) {
          // of a segment: what the segments before it leave, one after the other
#pragma unroll 1
          for (int i = place.segs == 1 ? 0 : min(place.seg, 1); i <= place.seg; ++i)
            load(place.segs == 1 ? S : kept(place.first + i), i > 1 ? __expf(params.decays[static_cast<int64_t>(place.first + i - 1) * p.nv + h]) : 0.f);
        } else if (place.seg == 0) {
          load(S, 0.f);
          save(kept(item));  // the last segment writes its end over S_0
        }
      }
      float decay = 0.f;
      uint8_t* s16 = smem + P::S16 + x * P::BLOCK;
      uint8_t* rows = smem + P::ROWS + x * P::BLOCK;
      const Pair by_v = pair_of(skip, skip);
      // the factors of chunk c: of the row's sums, of the state before it, and of its products with V'; and of the state in the sums
      struct Factors {
        float row, keep, grow, to16;
      };
      auto factors = [&](int c) {
        sh.wait(P::GATES, c & 1, ok);
        const float suf = small.suf[x][t], total = small.total[c & 1][x];
        const bool wide = ssm_wide(total);
        sh.arrive(P::GATES_READ);
        const float mid = wide ? 0.f : 0.5f * total;
        Factors f;
        f.row = wide ? 1.f : __expf(mid - suf);
        f.keep = __expf(total);
        f.grow = __expf(mid);
        f.to16 = wide ? 1.f : f.grow;  // e^{total - mid}
        if (!kOut) decay += total;
        return f;
      };
      Factors now = factors(0);
      float scale = 0.f;  // of the row's outputs in the chunk before
      for (int c = 0; c <= chunks; ++c) {
        const uint32_t ph = c & 1;
        if (kOut && c < chunks) {  // S for the products, with what it decays by beside V' where they share an accumulator
          const Pair by = pair_of(now.to16, now.to16);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) parts_of(mul2(pair_of(s[8 * i + 2 * e], s[8 * i + 2 * e + 1]), by), y[2 * e], y[2 * e + 1]);
            *reinterpret_cast<uint4*>(s16 + tc::sw128(t, 16 * i)) = pack16<__nv_bfloat16>(y);
          }
          tc::fence_proxy_async();
          tc::fence_before_sync();
          sh.arrive(P::S_READY);
        }
        if (!kOut && c < chunks) {  // L has been read
          tc::fence_before_sync();
          sh.arrive(P::S_READY);
        }
        if (kOut && c > 0) {  // the rows of the chunk before
          const uint32_t from = tmem + lanes + P::COL_O + 64 * x, off = (c & 1) ? 0 : 128;  // its buffer
          sh.wait(P::X_FULL + (ph ^ 1), ((c - 1) >> 1) & 1, ok);
          sh.wait(P::O_FULL + (ph ^ 1), ((c - 1) >> 1) & 1, ok);
          tc::fence_after_sync();
          const Pair by = pair_of(scale, scale);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t o[16], w[8];
            tc::tmem_ld16u(from + off + 16 * i, o);
            Pair v[8];
            unpack16<__nv_bfloat16>(*reinterpret_cast<const uint4*>(rows + tc::sw128(t, 32 * i)), *reinterpret_cast<Pair(*)[4]>(&v[0]));
            unpack16<__nv_bfloat16>(*reinterpret_cast<const uint4*>(rows + tc::sw128(t, 32 * i + 16)), *reinterpret_cast<Pair(*)[4]>(&v[4]));
            tc::tmem_ld_wait16(o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fma2(pair_of(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), by, mul2(v[e], by_v));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float y[2];
              parts_of(v[e], y[0], y[1]);
              w[e] = pack2<__nv_bfloat16>(y[0], y[1]);
            }
            *reinterpret_cast<uint4*>(rows + tc::sw128(t, 32 * i)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(rows + tc::sw128(t, 32 * i + 16)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          tc::fence_before_sync();
          sh.arrive(P::O_READ + (ph ^ 1));
          // out by one copy (by plain stores of eight lanes a row the scan of 4 x 8192 took half as long again), the last chunk of a
          // sequence by its rows, of which the copy would write those behind it too
          const int at = (c - 1) * kSsmChunk, n = tokens - at;
          if (n >= kSsmChunk) {
            tc::fence_proxy_async();
            sh.arrive(P::STAGED);
          } else {
            __syncwarp();
#pragma unroll 1
            for (int i = lane >> 3; i < 32; i += 4) {
              const int r = (t & 96) + i;
              const uint4 v = *reinterpret_cast<const uint4*>(rows + tc::sw128(r, 16 * (lane & 7)));
              if (ok && real && r < n) *reinterpret_cast<uint4*>(p.out + (start + at + r) * p.out_stride + col + 8 * (lane & 7)) = v;
            }
          }
        }
        if (c < chunks) {
          scale = now.row;
          const Pair by = pair_of(now.keep, now.keep), in = pair_of(now.grow, now.grow);
          if (c + 1 < chunks) now = factors(c + 1);
          sh.wait(P::L_FULL, ph, ok);
          tc::fence_after_sync();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t l[32];
            tc::tmem_ld32(tmem + lanes + P::COL_L + 64 * x + 32 * i, l);
            tc::tmem_ld_wait32(l);
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              parts_of(fma2(pair_of(s[32 * i + e], s[32 * i + e + 1]), by, mul2(pair_of(__uint_as_float(l[e]), __uint_as_float(l[e + 1])), in)),
                       s[32 * i + e], s[32 * i + e + 1]);
          }
        }
      }
      if (ok && held) {
        if (kOut && place.seg == place.segs - 1) save(S);
        if (!kOut) {
          save(kept(item + 1));
          if (t == 0 && unit % SLICES == 0) params.decays[static_cast<int64_t>(item) * p.nv + h] = decay;
        }
      }
    } else {
      // ---- operands --------------------------------------------------------------------------
      fewer_registers<kSsmOperandRegs>();
      const int r0 = t & 96, quarter = warp & 3;  // the warp's tokens: r0 + 4 i + lane / 8, eight lanes a row
      const __nv_bfloat16* v = p.v + static_cast<int64_t>(start + r0 + (lane >> 3)) * p.v_stride + col + 8 * (lane & 7);
      uint8_t* hi[2];  // a lane's place in V' for even and odd i
#pragma unroll
      for (int i = 0; i < 2; ++i) hi[i] = smem + P::VHI + x * P::BLOCK + tc::sw128(r0 + 4 * i + (lane >> 3), 16 * (lane & 7));
      uint4 word[8];  // a chunk's v, ahead
      // Half of the next chunk's words come while A is made, where there are registers for no more, but not beside wide decays, whose A
      // reads shared memory behind these loads: without it ragged prompts took 362 us for 337, and 448 for 405 with wide decays (461 where
      // those fetch early too)
      auto fetch = [&](int c, auto first, auto last, bool now) {  // words first .. last - 1
        constexpr int from = decltype(first)::value, to = decltype(last)::value;
        const int left = opaque(is_real) && now ? tokens - c * kSsmChunk - r0 - (lane >> 3) : 0;
        const __nv_bfloat16* at = v + static_cast<int64_t>(c * kSsmChunk + 4 * from) * p.v_stride;
#pragma unroll
        for (int i = from; i < to; ++i) {
          if (left > 4 * i) word[i] = *reinterpret_cast<const uint4*>(at);
          at += 4 * p.v_stride;
        }
      };
      auto clear = [&] {
#pragma unroll
        for (int i = 0; i < 8; ++i) word[i] = make_uint4(0, 0, 0, 0);
      };
      clear();
      using None = std::integral_constant<int, 0>;
      using Half = std::integral_constant<int, 4>;
      using All = std::integral_constant<int, 8>;
      fetch(0, None{}, All{}, true);
      uint32_t set = 0;    // phase of STEPS_SET
      bool own_v = false;  // whether O1 of the chunk before took v itself for this unit
      for (int c = 0; c < chunks; ++c) {
        const uint32_t ph = c & 1;
        const int n = min(kSsmChunk, tokens - c * kSsmChunk);
        if (n < kSsmChunk) {  // rows of K behind the sequence are someone else's, or nobody's: as zeros they are no NaN
          sh.wait(P::K_FULL + ph, (c >> 1) & 1, ok);  // (the phase before: L_FULL of chunk c - 2, which has read that K)
#pragma unroll 1
          for (int i = threadIdx.x - 256; i < (kSsmChunk - n) * 8 * KB; i += 256) {
            const int r = n + i / (8 * KB), w = i % (8 * KB);
            *reinterpret_cast<uint4*>(smem + P::K + (2 * ph + w / 8) * P::BLOCK + r * 128 + w % 8 * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        sh.wait(P::GATES, ph, ok);
        const bool wide = ssm_wide(small.total[ph][x]), any = wide || ssm_wide(small.total[ph][x ^ 1]);
        const float suf = small.suf[x][t], d = small.d[x][t], f = d * __expf(wide ? suf : fmaf(-0.5f, small.total[ph][x], suf));
        const float f_hi = __bfloat162float(__float2bfloat16_rn(f));
        const uint32_t both = pack2<__nv_bfloat16>(f_hi, f - f_hi);
        if (c > 0) {  // V is free
          sh.wait(P::L_FULL, ph ^ 1, ok);
          // (the phase before: L of chunk c - 1 was issued behind O_READ of chunk c - 3)
          if (kOut && !own_v) sh.wait(P::O_FULL + (ph ^ 1), ((c - 1) >> 1) & 1, ok);
        }
        own_v = wide;
        // V' = v f in pairs of bf16: with f = f_hi + f_lo, hi = v f_hi rounded, lo = (v f_hi - hi, exact) + v f_lo
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t other = __shfl_sync(0xffffffffu, both, 4 * i + (lane >> 3));
          const __nv_bfloat162 fh = as_bf162(__byte_perm(other, 0, 0x1010)), fl = as_bf162(__byte_perm(other, 0, 0x3232));
          const uint32_t w[4] = {word[i].x, word[i].y, word[i].z, word[i].w};
          uint32_t a4[4], b4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 e = as_bf162(w[k]), high = __hmul2_rn(e, fh);
            a4[k] = as_u32(high);
            b4[k] = as_u32(__hfma2(e, fl, __hfma2(e, fh, __hneg2(high))));
          }
          uint8_t* at = hi[i & 1] + i / 2 * 1024;
          *reinterpret_cast<uint4*>(at) = make_uint4(a4[0], a4[1], a4[2], a4[3]);
          *reinterpret_cast<uint4*>(at + (P::VLO - P::VHI)) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
        }
        tc::fence_proxy_async();
        sh.arrive(P::V_READY);
        clear();
        fetch(c + 1, None{}, Half{}, c + 1 < chunks && !any);
        if (!kOut) sh.arrive(P::STEPS_READ);
        if constexpr (kOut) {
          sh.wait(P::G_FULL, ph, ok);
          // A: row t, columns 32 i .. 32 i + 31, of which it sees those up to itself. Half of it in place of this half of G;
          // where a decay is wide and the units are two heads, the 32 columns of both units in place of those of G, once both have them.
          // For that the two warps of these rows meet at a barrier once a block, in every chunk. (With waits of the bounded kind in its
          // place the ragged prompts take 465 us for 410, as the two no longer run through the code together.)
          const bool own_a = any && SLICES == 1;
          const float own = suf * kLog2e;
          if (wide) {  // d e^{suf - behind} in the place of d, and log2 of d e^{suf} in that of suf, once the rows' warps have it
            const float last = __shfl_sync(0xffffffffu, suf, lane | 15);
            sh.wait(P::GATES_READ, ph, ok);  // (the phase before: GATES of this chunk came behind it)
            small.d[x][t] = d * __expf(suf - last);
            small.suf[x][t] = own + __log2f(d);
            if ((lane & 15) == 15) small.behind[x][t >> 4] = own;
            sh.arrive(P::STEPS_SET + x);
            sh.wait(P::STEPS_SET + x, set, ok);
            set ^= 1;
          }
          tc::fence_after_sync();
          // block i of 32 columns, `spread` with a wide decay's factors
          auto block = [&](int i, bool spread, uint32_t (&k16)[16]) {
            uint32_t r[32];
            float f[2] = {1.f, 1.f};
            if (spread && i < quarter) {
              f[0] = ssm_exp2(small.behind[x][2 * i] - own);
              f[1] = ssm_exp2(small.behind[x][2 * i + 1] - own);
            }
            if (i <= quarter && __any_sync(0xffffffffu, f[1] > 0.f)) {
              tc::tmem_ld32(tmem + lanes + P::COL_G + 32 * i, r);
              tc::tmem_ld_wait32(r);
              if (spread && i < quarter) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const Pair row = pair_of(f[e / 16], f[e / 16]);
                  float c4[4], y[4];
                  load4(&small.d[x][32 * i + e], c4);
#pragma unroll
                  for (int k = 0; k < 4; k += 2)
                    parts_of(mul2(mul2(pair_of(__uint_as_float(r[e + k]), __uint_as_float(r[e + k + 1])), pair_of(c4[k], c4[k + 1])), row), y[k], y[k + 1]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) r[e + k] = __float_as_uint(y[k]);
                }
              } else if (spread) {
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * ssm_exp2(small.suf[x][32 * i + e] - own));
              }
              if (i == quarter) {
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = e <= lane ? r[e] : 0u;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) k16[e / 2] = pack2<__nv_bfloat16>(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) k16[e] = 0;
            }
          };
          if (own_a) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t k16[16];
              block(i, wide, k16);
              if (i <= quarter) tc::named_barrier(7 + quarter, 64);
              tc::tmem_st16u(tmem + lanes + P::COL_G + 32 * i + 16 * x, k16);
            }
          } else {
            if (SLICES == 1)
#pragma unroll 1
              for (int i = 0; i <= quarter; ++i) tc::named_barrier(7 + quarter, 64);
#pragma unroll 1
            for (int i = 2 * x; i < 2 * x + 2; ++i) {
              uint32_t k16[16];
              block(i, SLICES == 2 && wide, k16);
              tc::tmem_st16u(tmem + lanes + P::COL_G + 32 * x + 16 * i, k16);
            }
          }
          sh.arrive(P::STEPS_READ);
          if (wide) {  // O2's rows take the decay before them
            const float f = __expf(small.total[ph][x] - suf);
            const uint32_t o = tmem + lanes + P::COL_O + ph * 128 + 64 * x;
            sh.wait(P::Q_FREE, ph, ok);  // (the phase before: G of this chunk was issued behind it)
            tc::fence_after_sync();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t r[16];
              tc::tmem_ld16u(o + 16 * i, r);
              tc::tmem_ld_wait16(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tc::tmem_st16u(o + 16 * i, r);
            }
          }
          tc::tmem_st_wait();
          tc::fence_before_sync();
          sh.arrive(P::A_READY);
        }
        if (c + 1 < chunks) {
          fetch(c + 1, None{}, Half{}, any);
          fetch(c + 1, Half{}, All{}, true);
        }
      }
    }
  } else {
    // ---- copies and products, by one warp of the last four ----------------------------------------
    fewer_registers<kSsmIssueRegs>();
    if (warp == 16) {
      constexpr uint32_t id_g = tc::idesc_f16(128, 128, tc::kBF16, false, false), id_o = tc::idesc_f16(128, 128, tc::kBF16, false, true),
                         id_o64 = tc::idesc_f16(128, 64, tc::kBF16, false, true), id_l = tc::idesc_f16(128, 128, tc::kBF16, true, true);
      auto copy = [&](const CUtensorMap* map, int to, int bar, int c) {
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(sh.bar(bar), KB * P::BLOCK);
#pragma unroll
          for (int i = 0; i < KB; ++i) tc::tma_load_2d(sbase + to + i * P::BLOCK, map, kh * DK + 64 * i, start + c * kSsmChunk, sh.bar(bar));
        }
        __syncwarp();
      };
      if (kOut) copy(&q_map, P::Q, P::Q_FULL, 0);
      copy(&k_map, P::K, P::K_FULL, 0);
      const uint64_t q_k = tc::desc_sw128(sbase + P::Q, 16, 1024), s_mn = tc::desc_sw128(sbase + P::S16, P::BLOCK, 1024);
      const uint64_t v_mn = tc::desc_sw128(sbase + P::ROWS, P::BLOCK, 1024);
      const uint64_t hi_mn = tc::desc_sw128(sbase + P::VHI, P::BLOCK, 1024), lo_mn = tc::desc_sw128(sbase + P::VLO, P::BLOCK, 1024);
      for (int c = 0; c < chunks && ok; ++c) {
        const uint32_t ph = c & 1;
        const int kt = P::K + ph * 2 * P::BLOCK;
        const uint64_t k_k = tc::desc_sw128(sbase + kt, 16, 1024), k_mn = tc::desc_sw128(sbase + kt, P::BLOCK, 1024);
        if (kOut) sh.wait(P::Q_FULL, ph, ok);
        sh.wait(P::K_FULL + ph, (c >> 1) & 1, ok);
        if (!ok) break;
        tc::fence_after_sync();
        if (kOut && tc::elect_one()) {
#pragma unroll 2
          for (int i = 0; i < DK / 16; ++i) {
            const uint32_t off = ((i >> 2) * P::BLOCK + (i & 3) * 32) >> 4;
            tc::mma_f16(tmem + P::COL_G, q_k + off, k_k + off, id_g, i > 0);
          }
          tc::mma_commit(sh.bar(P::G_FULL));
        }
        __syncwarp();
        if (c + 1 < chunks) {
          if (c > 0) sh.wait(P::L_FULL, ph ^ 1, ok);  // the products of the chunk before have read the other K
          if (!ok) break;
          copy(&k_map, P::K + (ph ^ 1) * 2 * P::BLOCK, P::K_FULL + (ph ^ 1), c + 1);
        }
        auto state = [&] {  // L
          if (tc::elect_one()) {
#pragma unroll 2
            for (int i = 0; i < 8; ++i) tc::mma_f16(tmem + P::COL_L, k_mn + ((i * 2048) >> 4), hi_mn + ((i * 2048) >> 4), id_l, i > 0);
#pragma unroll 2
            for (int i = 0; i < 8; ++i) tc::mma_f16(tmem + P::COL_L, k_mn + ((i * 2048) >> 4), lo_mn + ((i * 2048) >> 4), id_l, 1);
            tc::mma_commit(sh.bar(P::L_FULL));
          }
          __syncwarp();
        };
        sh.wait(P::S_READY, ph, ok);  // and L has been read
        if constexpr (kOut) {
          if (c > 1) sh.wait(P::O_READ + ph, ((c >> 1) - 1) & 1, ok);
          if (!ok) break;
          const bool wide[2] = {ssm_wide(small.total[ph][0]), ssm_wide(small.total[ph][1])}, any = wide[0] || wide[1];
          const uint32_t o = tmem + P::COL_O + ph * 128;  // the chunk's buffer
          tc::fence_after_sync();
          if (tc::elect_one()) {
#pragma unroll 2
            for (int i = 0; i < DK / 16; ++i) {
              const uint32_t off = ((i >> 2) * P::BLOCK + (i & 3) * 32) >> 4;
              tc::mma_f16(o, q_k + off, s_mn + ((i * 2048) >> 4), id_o, i > 0);
            }
            tc::mma_commit(sh.bar(P::Q_FREE));
          }
          __syncwarp();
          sh.wait(P::V_READY, ph, ok);
          if (!ok) break;
          tc::fence_after_sync();
          state();  // L before O1: the next state then waits for neither A nor O1
          if (c + 1 < chunks) {
            sh.wait(P::Q_FREE, ph, ok);
            if (!ok) break;
            copy(&q_map, P::Q, P::Q_FULL, c + 1);
          }
          sh.wait(P::A_READY, ph, ok);
          if (any) sh.wait(P::X_FULL + ph, (c >> 1) & 1, ok);  // (the phase before: O_READ of chunk c - 2, whose rows had v)
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            if (!any || SLICES == 2) {
              const uint64_t b_mn = any ? v_mn : hi_mn;
#pragma unroll 2
              for (int i = 0; i < 8; ++i) tc::mma_f16_ts(o, tmem + P::COL_G + 8 * i + (i & 4) * 8, b_mn + ((i * 2048) >> 4), id_o, 1);
            } else {
              for (int u = 0; u < 2; ++u)
#pragma unroll 2
                for (int i = 0; i < 8; ++i)
                  tc::mma_f16_ts(o + 64 * u, tmem + P::COL_G + 32 * (i >> 1) + 16 * u + 8 * (i & 1), (wide[u] ? v_mn : hi_mn) + ((u * P::BLOCK + i * 2048) >> 4), id_o64, 1);
            }
            tc::mma_commit(sh.bar(P::O_FULL + ph));
          }
          __syncwarp();
        } else {
          sh.wait(P::V_READY, ph, ok);
          if (!ok) break;
          tc::fence_after_sync();
          if (c + 2 < chunks && tc::elect_one()) {
            for (int i = 0; i < KB; ++i) tc::tma_prefetch_2d(&k_map, kh * DK + 64 * i, start + (c + 2) * kSsmChunk);
            for (int x = 0; x < min(2, units - 2 * (pair % per_key)); ++x)
              tc::tma_prefetch_2d(&v_map, kh * heads * DV + (2 * (pair % per_key) + x) * 64, start + (c + 2) * kSsmChunk);
          }
          __syncwarp();
          state();
        }
      }
    } else if (warp < 19) {
      // ---- gates, a warp a unit, four tokens a lane -----------------------------------------------
      const int x = warp - 17;
      const int is_real = 2 * (pair % per_key) + x < units, unit = 2 * (pair % per_key) + (is_real ? x : 0), h = kh * heads + unit / SLICES;
      const float a = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
      float z[4];
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = c * kSsmChunk + 4 * lane + i;
          z[i] = 0.f;
          if (opaque(is_real) && r < tokens) {
            const int64_t at = (start + r) * p.dt_stride + h;
            z[i] = p.dt_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.dt)[at]) : static_cast<const float*>(p.dt)[at];
          }
        }
      };
      fetch(0);
      for (int c = 0; c < chunks; ++c) {
        const uint32_t ph = c & 1;
        float d[4], suf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = z[i] + bias;
          d[i] = !(opaque(is_real) && c * kSsmChunk + 4 * lane + i < tokens) ? 0.f : opaque(p.softplus) ? fmaxf(y, 0.f) + log1pf(__expf(-fabsf(y))) : y;
        }
        if (c + 1 < chunks) fetch(c + 1);
        // a token's decay; from e^-200 on it is none in fp32, and as no more than that the sums behind it keep their last bits for the
        // tokens before it
        auto gate = [&](int i) {
          const float g = d[i] * a;
          return g < -200.f ? -200.f : g;
        };
        suf[3] = 0.f;
#pragma unroll
        for (int i = 3; i > 0; --i) suf[i - 1] = gate(i) + suf[i];
        float incl = gate(0) + suf[0];  // from this lane's first token to the chunk's last
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, incl, o);
          if (lane + o < 32) incl += y;
        }
        float behind = __shfl_down_sync(0xffffffffu, incl, 1);
        if (lane == 31) behind = 0.f;
        if (c > 0) {  // the chunk's before are used
          sh.wait(P::GATES_READ, ph ^ 1, ok);
          sh.wait(P::STEPS_READ, ph ^ 1, ok);
        }
        *reinterpret_cast<float4*>(&small.d[x][4 * lane]) = make_float4(d[0], d[1], d[2], d[3]);
        *reinterpret_cast<float4*>(&small.suf[x][4 * lane]) = make_float4(suf[0] + behind, suf[1] + behind, suf[2] + behind, suf[3] + behind);
        if (lane == 0) small.total[ph][x] = incl;
        sh.arrive(P::GATES);
      }
    } else if (kOut) {
      // ---- the rows: out what is there of the chunk before, then v in its place; and what comes two chunks on, into L2 ---------
      const int left = min(2, units - 2 * (pair % per_key)), col = kh * heads * DV + 2 * (pair % per_key) * 64;
      for (int c = 0; c < chunks; ++c) {
        const int at = start + c * kSsmChunk, ahead = at + 2 * kSsmChunk, n = tokens - c * kSsmChunk;
        const int full = n < kSsmChunk ? P::X_LANDED : P::X_FULL + (c & 1);
        if (c > 0) sh.wait(P::STAGED, (c & 1) ^ 1, ok);
        if (!ok) break;
        if (tc::elect_one()) {
          if (c > 0) {
            for (int x = 0; x < left; ++x) tc::tma_store_2d(&out_map, col + 64 * x, at - kSsmChunk, sbase + P::ROWS + x * P::BLOCK);
            tc::tma_store_commit();
            tc::tma_store_wait_read();
          }
          tc::mbar_arrive_expect_tx(sh.bar(full), left * P::BLOCK);
          for (int x = 0; x < left; ++x) {
            tc::tma_load_2d(sbase + P::ROWS + x * P::BLOCK, &v_map, col + 64 * x, at, sh.bar(full));
            if (c + 2 < chunks) tc::tma_prefetch_2d(&v_map, col + 64 * x, ahead);
          }
          if (c + 2 < chunks)
            for (int i = 0; i < KB; ++i) {
              tc::tma_prefetch_2d(&q_map, kh * DK + 64 * i, ahead);
              tc::tma_prefetch_2d(&k_map, kh * DK + 64 * i, ahead);
            }
        }
        __syncwarp();
        if (n < kSsmChunk) {  // where O1 takes v itself, rows behind the sequence are zeros before anyone has them, so that they are no NaN
          sh.wait(P::X_LANDED, 0, ok);
          sh.wait(P::GATES, c & 1, ok);  // (the phase before: STAGED of chunk c - 1, whose rows have the factors of c; none comes after)
          if (!ok) break;
          if (ssm_wide(small.total[c & 1][0]) || ssm_wide(small.total[c & 1][1]))
#pragma unroll 4
            for (int i = lane; i < (kSsmChunk - n) * 8 * left; i += 32)
              *reinterpret_cast<uint4*>(smem + P::ROWS + (i & 8) / 8 * (left - 1) * P::BLOCK + (n + i / (8 * left)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async();
          sh.arrive(P::X_FULL + (c & 1));
        }
      }
      if (tokens % kSsmChunk == 0) sh.wait(P::STAGED, (chunks - 1) & 1, ok);
      if (ok && tokens % kSsmChunk == 0 && tc::elect_one()) {
        for (int x = 0; x < left; ++x) tc::tma_store_2d(&out_map, col + 64 * x, start + tokens - kSsmChunk, sbase + P::ROWS + x * P::BLOCK);
        tc::tma_store_commit();
        tc::tma_store_wait_read();
      }
      __syncwarp();
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (small.abort) {  // products and copies in flight land before the memory is given up
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (warp == 16) tc::tmem_dealloc(tmem, P::TMEM_COLS);
}

}  // namespace gdn
