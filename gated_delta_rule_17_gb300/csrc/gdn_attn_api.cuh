// Host side of the entry points in include/gdn_attention.h: argument checks (each rejection
// names the guard) and launches. Included by gdn_api.cu, whose error message, launch count,
// device table and status word it shares.
#pragma once

namespace {

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

int launched(int launches) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  g_launches = launches;
  return GDN_OK;
}

int check_head_dim(int d) {
  if (d != 64 && d != 128) return fail(GDN_ERR_UNSUPPORTED, "head_dim = %d is neither 64 nor 128", d);
  return GDN_OK;
}

int check_rope(const gdn_rope_t* r, int d, gdn::RopeParams* out, int* interleaved) {
  *out = gdn::RopeParams{};
  *interleaved = 0;
  if (!r || r->rot == 0) return GDN_OK;
  if (r->rot < 0 || r->rot > d || r->rot % 8)
    return fail(GDN_ERR_ARG, "rot = %d must be a multiple of 8 in 0..head_dim", r->rot);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(GDN_ERR_ARG, "interleaved must be 0 or 1");
  if (!r->cos || !r->sin) return fail(GDN_ERR_ARG, "a rotation table pointer is NULL");
  if (!aligned16(r->cos) || !aligned16(r->sin)) return fail(GDN_ERR_ARG, "cos and sin must be 16-byte aligned");
  if (r->positions < 0) return fail(GDN_ERR_ARG, "the rotation table's positions = %d is negative", r->positions);
  if (r->stride < r->rot / 2 || r->stride % 4)
    return fail(GDN_ERR_ARG, "rotation table stride %lld must be >= rot / 2 and a multiple of 4", (long long)r->stride);
  out->cos = r->cos;
  out->sin = r->sin;
  out->stride = r->stride;
  out->positions = r->positions;
  out->rot = r->rot;
  *interleaved = r->interleaved;
  return GDN_OK;
}

int check_stride(int64_t stride, int64_t least, const char* name) {
  if (stride < least || stride % 8)
    return fail(GDN_ERR_ARG, "%s row stride %lld must be >= %lld and a multiple of 8", name, (long long)stride,
                (long long)least);
  return GDN_OK;
}

template <int N>
using IntC = std::integral_constant<int, N>;

// Head rows a lane group takes of a token with `heads` heads at most.
int norm_unroll(int heads, int d) {
  const int slots = 256 / d;
  return heads <= slots ? 1 : heads <= 2 * slots ? 2 : gdn::kNormUnroll;
}
// Calls f with it at compile time.
template <typename F>
void by_unroll(int unroll, F&& f) {
  if (unroll == 1) f(IntC<1>{});
  else if (unroll == 2) f(IntC<2>{});
  else f(IntC<gdn::kNormUnroll>{});
}

int norm_chunks(int heads, int d, int unroll) {
  const int per = unroll * (32 / (d / 8));
  return (heads + per - 1) / per;
}

// The checks that the forward and the backward share; fills all but the gradients' fields.
int norm_setup(const void* q, const void* k, const int32_t* positions, const gdn_rope_t* rope, const float* q_weight,
               const float* k_weight, float eps, void* q_out, void* k_out, int rows, int nq, int nkv, int d, int dtype,
               const gdn_norm_strides_t* st, int unroll, gdn::NormRopeParams* p, int* interleaved) {
  *p = gdn::NormRopeParams{};
  if (rows < 0) return fail(GDN_ERR_ARG, "rows = %d is negative", rows);
  if (nq < 0 || nkv < 0 || nq + static_cast<int64_t>(nkv) < 1)
    return fail(GDN_ERR_ARG, "head counts nq = %d, nkv = %d: neither negative, one at least positive", nq, nkv);
  if (int rc = check_head_dim(d)) return rc;
  if (dtype != GDN_BF16 && dtype != GDN_F16 && dtype != GDN_F32) return fail(GDN_ERR_UNSUPPORTED, "dtype %d is unknown", dtype);
  if (!(eps >= 0.f)) return fail(GDN_ERR_ARG, "eps must not be negative");
  if (int rc = check_rope(rope, d, &p->rope, interleaved)) return rc;
  const int64_t wq = static_cast<int64_t>(nq) * d, wk = static_cast<int64_t>(nkv) * d;
  p->q_stride = st ? st->q : wq;
  p->k_stride = st ? st->k : wk;
  p->q_out_stride = st ? st->q_out : wq;
  p->k_out_stride = st ? st->k_out : wk;
  p->q_grad_stride = st ? st->q_grad : wq;
  p->k_grad_stride = st ? st->k_grad : wk;
  if (nq) {
    if (int rc = check_stride(p->q_stride, wq, "q")) return rc;
    if (int rc = check_stride(p->q_out_stride, wq, "q_out")) return rc;
  }
  if (nkv) {
    if (int rc = check_stride(p->k_stride, wk, "k")) return rc;
    if (int rc = check_stride(p->k_out_stride, wk, "k_out")) return rc;
  }
  p->q_chunks = norm_chunks(nq, d, unroll);
  p->chunks = p->q_chunks + norm_chunks(nkv, d, unroll);
  if (static_cast<int64_t>(rows) * p->chunks > INT32_MAX - (1 << 20))
    return fail(GDN_ERR_UNSUPPORTED, "%d rows of %d + %d heads exceed the item range", rows, nq, nkv);
  if (rows == 0) return GDN_OK;
  if ((nq && (!q || !q_out)) || (nkv && (!k || !k_out))) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
    return fail(GDN_ERR_ARG, "q, k and their outputs must be 16-byte aligned");
  if (!aligned16(q_weight) || !aligned16(k_weight)) return fail(GDN_ERR_ARG, "weights must be 16-byte aligned");
  if (p->rope.rot && !positions) return fail(GDN_ERR_ARG, "a rotation needs positions");
  p->q = q;
  p->k = k;
  p->q_out = q_out;
  p->k_out = k_out;
  p->positions = positions;
  p->q_weight = q_weight;
  p->k_weight = k_weight;
  p->rows = rows;
  p->nq = nq;
  p->nkv = nkv;
  p->eps = eps;
  return GDN_OK;
}

// Calls f(T{}, D, interleaved) with compile-time element type, head size and pairing.
template <typename F>
void by_head(int d, int interleaved, F&& f) {
  if (d == 64) interleaved ? f(IntC<64>{}, std::true_type{}) : f(IntC<64>{}, std::false_type{});
  else interleaved ? f(IntC<128>{}, std::true_type{}) : f(IntC<128>{}, std::false_type{});
}
template <typename F>
void by_type16(int dtype, F&& f) {
  dtype == GDN_BF16 ? f(__nv_bfloat16{}) : f(__half{});
}
template <typename F>
void by_type(int dtype, F&& f) {
  if (dtype == GDN_F32) f(float{});
  else by_type16(dtype, f);
}

int check_paged(const gdn_paged_t* c, int nkv, int d, gdn::PagedParams* p) {
  *p = gdn::PagedParams{};
  if (!c) return fail(GDN_ERR_ARG, "the cache is NULL");
  if (c->B < 0 || c->rows < 0) return fail(GDN_ERR_ARG, "B = %d or rows = %d is negative", c->B, c->rows);
  if (c->page_size < 1 || c->num_pages < 0 || c->max_pages < 0)
    return fail(GDN_ERR_ARG, "page_size = %d, num_pages = %d or max_pages = %d is out of range", c->page_size, c->num_pages,
                c->max_pages);
  if (static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX - 65536)
    return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size exceeds the 2^31 token range");
  if (c->table_stride < c->max_pages)
    return fail(GDN_ERR_ARG, "block_table row stride %lld is below max_pages = %d", (long long)c->table_stride, c->max_pages);
  for (const int64_t s : {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head})
    if (s < 0 || s % 8) return fail(GDN_ERR_ARG, "cache stride %lld must be a multiple of 8", (long long)s);
  if (nkv > 1 && (c->k_head < d || c->v_head < d)) return fail(GDN_ERR_ARG, "cache head strides are below head_dim = %d", d);
  if (!c->cu_rows && c->rows != c->B)
    return fail(GDN_ERR_ARG, "without cu_rows there is one row a sequence: rows = %d, B = %d", c->rows, c->B);
  if (c->rows > 0 && c->B == 0) return fail(GDN_ERR_ARG, "%d rows of no sequence", c->rows);
  if (c->rows == 0) return GDN_OK;
  if (!c->k || !c->v || !c->block_table || !c->ctx_lens) return fail(GDN_ERR_ARG, "a required cache pointer is NULL");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(GDN_ERR_ARG, "the caches must be 16-byte aligned");
  p->k = c->k;
  p->v = c->v;
  p->k_page = c->k_page;
  p->k_token = c->k_token;
  p->k_head = c->k_head;
  p->v_page = c->v_page;
  p->v_token = c->v_token;
  p->v_head = c->v_head;
  p->num_pages = c->num_pages;
  p->page_size = c->page_size;
  p->block_table = c->block_table;
  p->table_stride = c->table_stride;
  p->max_pages = c->max_pages;
  p->B = c->B;
  p->rows = c->rows;
  p->ctx_lens = c->ctx_lens;
  p->cu_rows = c->cu_rows;
  return GDN_OK;
}

// ---- attention -----------------------------------------------------------------------
constexpr int kAttnCtasPerSm = 2;  // of gdn_attn_kernel; gdn_attn_tc_kernel has an SM to itself

// The kernel for the rows that a kv head may have (new rows of a sequence x heads of a group). With
// 16 or fewer one block of register products does: 79 us against 82 on tcgen05 at 16 rows, 16
// sequences of 4096 to 8192 tokens, 8 kv heads; 58 against 72 for 128 sequences of 200 to 400. Above,
// tcgen05 does: 83 against 112 (two blocks of 16) or 106 (blocks of 32) at 24 rows.
enum AttnKind { kAttn16, kAttnTc };
constexpr int kAttnKindRows[] = {gdn::kAttnRows, gdn::kTcRows};
AttnKind attn_kind(int64_t rows, float scale) {
  // the tensor-core kernel keeps its maxima in unscaled scores, which a scale <= 0 would turn round
  return rows <= gdn::kAttnRows || !(scale > 0.f) ? kAttn16 : kAttnTc;
}

int attn_runs(AttnKind kind, int sms) {
  const int runs = kind != kAttnTc ? sms * kAttnCtasPerSm : sms;
  return runs < gdn::kJoinRuns ? runs : gdn::kJoinRuns;
}

// Whether to give the CTAs whole units. That costs the tiles by which the busiest CTA then has more
// than an even share (and what the units' lengths differ by, which the host does not know: hence
// the limit on them), and saves the join and the pieces' way through memory, worth about seven
// tiles. Measured whole and cut, graph replays: 8 sequences of 500 tokens, 8 kv heads, one row each
// 12.3 and 12.9 us, 64 of 500 32 and 35, one of 500 12.3 and 10.5, 8 of 1000 19 and 15; trees of 16 in
// 32 sequences of 980 31 and 36, in 8 of 480 11.5 and 16.4.
bool attn_whole(AttnKind kind, int sms, const gdn::AttnParams& p, int most) {
  const int64_t tile = kind == kAttn16 ? gdn::kAttnTile : gdn::kTcTile;
  const int64_t tiles = (static_cast<int64_t>(p.cache.max_pages) * p.cache.page_size + tile - 1) / tile;
  if (tiles > 16) return false;
  // two bounds on the row tiles of a kv head: by all rows, and by the most of a sequence
  const int64_t rows = kAttnKindRows[kind], group = p.group, B = p.cache.B;
  const int64_t by_all = p.cache.rows * group / rows + B, by_most = B * ((most * group + rows - 1) / rows);
  const int64_t units = p.nkv * (by_all < by_most ? by_all : by_most);
  const int64_t ctas = attn_runs(kind, sms);
  return (units + ctas - 1) / ctas * tiles - units * tiles / ctas <= 7;
}

struct AttnLayout {
  size_t cut, ml, o, total;
};
AttnLayout attn_layout(AttnKind kind, int sms, int d) {
  const size_t runs = attn_runs(kind, sms), rows = runs * 2 * kAttnKindRows[kind];
  AttnLayout l;
  l.cut = 0;
  l.ml = align256(runs * sizeof(int4));
  l.o = l.ml + align256(rows * 2 * sizeof(float));
  l.total = l.o + align256(rows * d * sizeof(float));
  return l;
}

// Tokens of a TMA box: the largest power of two that divides the page size, from 8 (the rows of a
// swizzle atom) to the 32 of a copying warp; 0 where there is none.
int attn_box(int page_size) {
  int box = page_size & -page_size;
  if (box > 32) box = 32;
  return box >= 8 ? box : 0;
}

// A cache as [pages][page_size][heads][d] with boxes of 64 values, one head, `box` tokens.
bool cache_map(CUtensorMap* m, const void* base, int64_t page, int64_t token, int64_t head, const gdn::PagedParams& c,
               int nkv, int d, int box, int dtype) {
  auto fn = encode_fn();
  if (!fn) return false;
  // a dimension of one takes any stride; the encoder wants one that is not zero
  auto bytes = [&](int64_t stride, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? stride : d) * 2; };
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(nkv), static_cast<cuuint64_t>(c.page_size),
                        static_cast<cuuint64_t>(c.num_pages)};
  cuuint64_t strides[3] = {bytes(head, nkv), bytes(token, c.page_size), bytes(page, c.num_pages)};
  cuuint32_t boxes[4] = {64, 1, static_cast<cuuint32_t>(box), 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, dtype == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may start while the kernel before it in the stream ends: all of these kernels wait
// for it (tc::grid_dependency_wait) before they read or write global memory.
template <typename... A, typename... B>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t s, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D, int MT>
cudaError_t launch_join(cudaError_t e, int sms, const gdn::AttnParams& p, cudaStream_t s) {
  if (e != cudaSuccess || p.whole) return e;
  return launch_early(gdn::gdn_attn_join_kernel<T, D, MT>, dim3(static_cast<unsigned>(sms * gdn::kJoinCtasPerSm)),
                      32 * gdn::kJoinWarps, 0, s, p);
}

template <typename T, int D>
cudaError_t launch_attn(AttnKind kind, int sms, const gdn::AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.runs));
  if (kind == kAttn16)
    return launch_join<T, D, gdn::kAttnRows>(
        launch_early(gdn::gdn_attn_kernel<T, D>, grid, gdn::kAttnThreads, gdn::AttnPlan<D>::DYN_SMEM, s, p), sms, p, s);
  return launch_join<T, D, gdn::kTcRows>(
      launch_early(gdn::gdn_attn_tc_kernel<T, D>, grid, gdn::kTcThreads, gdn::AttnTcPlan<D>::DYN_SMEM, s, k, v, p), sms, p, s);
}

}  // namespace

extern "C" {

int gdn_head_norm_rope(const void* q, const void* k, const int32_t* positions, const gdn_rope_t* rope,
                       const float* q_weight, const float* k_weight, float eps, void* q_out, void* k_out, int rows,
                       int nq, int nkv, int d, int dtype, const gdn_norm_strides_t* strides, void* stream) {
  g_err[0] = 0;
  g_launches = 0;
  gdn::NormRopeParams p;
  int next = 0;
  if (int rc = check_head_dim(d)) return rc;  // norm_unroll divides by it
  const int unroll = norm_unroll(nq > nkv ? nq : nkv, d);
  if (int rc = norm_setup(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out, rows, nq, nkv, d, dtype, strides,
                          unroll, &p, &next))
    return rc;
  if (rows == 0) return GDN_OK;
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  p.status = dev->status;
  const int warps = gdn::kNormThreads / 32;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(rows) * p.chunks + warps - 1) / warps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_type(dtype, [&](auto t) {
    by_head(d, next, [&](auto dim, auto pairs) {
      by_unroll(unroll, [&](auto u) {
        gdn::gdn_head_norm_rope_kernel<decltype(t), dim.value, pairs.value, u.value><<<grid, gdn::kNormThreads, 0, s>>>(p);
      });
    });
  });
  return launched(1);
}

size_t gdn_head_norm_rope_backward_workspace_bytes(int rows, int nq, int nkv, int d) {
  (void)nq;
  (void)nkv;
  if (rows <= 0 || (d != 64 && d != 128)) return 0;
  return (static_cast<size_t>(plan_sms()) * gdn::kNormBwdCtasPerSm + 2) * d * sizeof(float);
}

int gdn_head_norm_rope_backward(const void* q, const void* k, const int32_t* positions, const gdn_rope_t* rope,
                                const float* q_weight, const float* k_weight, float eps, const void* q_grad,
                                const void* k_grad, void* dq, void* dk, float* dq_weight, float* dk_weight, int rows,
                                int nq, int nkv, int d, int dtype, const gdn_norm_strides_t* strides, void* workspace,
                                size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  g_launches = 0;
  gdn::NormRopeParams p;
  int next = 0;
  if (int rc = norm_setup(q, k, positions, rope, q_weight, k_weight, eps, dq, dk, rows, nq, nkv, d, dtype, strides,
                          gdn::kNormUnroll, &p, &next))
    return rc;
  if (nq)
    if (int rc = check_stride(p.q_grad_stride, static_cast<int64_t>(nq) * d, "q_grad")) return rc;
  if (nkv)
    if (int rc = check_stride(p.k_grad_stride, static_cast<int64_t>(nkv) * d, "k_grad")) return rc;
  const bool sums = dq_weight || dk_weight;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // sums over no rows
    for (float* w : {dq_weight, dk_weight})
      if (w) {
        cudaError_t e = cudaMemsetAsync(w, 0, static_cast<size_t>(d) * sizeof(float), s);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
      }
    return GDN_OK;
  }
  if ((nq && !q_grad) || (nkv && !k_grad)) return fail(GDN_ERR_ARG, "an incoming gradient pointer is NULL");
  if (!aligned16(q_grad) || !aligned16(k_grad)) return fail(GDN_ERR_ARG, "q_grad and k_grad must be 16-byte aligned");
  const size_t need = gdn_head_norm_rope_backward_workspace_bytes(rows, nq, nkv, d);
  if (workspace && sums) {
    if (workspace_bytes < need)
      return fail(GDN_ERR_ARG, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, need);
    if (!aligned256(workspace)) return fail(GDN_ERR_ARG, "workspace must be 256-byte aligned");
  }
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  p.status = dev->status;
  p.q_grad = q_grad;
  p.k_grad = k_grad;
  void* ws = sums ? workspace : nullptr;
  if (sums && !ws) {
    cudaError_t e = cudaMallocAsync(&ws, need, s);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaMallocAsync(%zu): %s", need, cudaGetErrorString(e));
  }
  p.partials = static_cast<float*>(ws);
  // the grid's CTAs in proportion to the steps that a token's heads take, at least one each; a token's
  // heads are cut into as many runs as it takes to give every warp one
  const int slots = dev->sms * gdn::kNormBwdCtasPerSm, warps = gdn::kNormBwdThreads / 32;
  const int step = 256 / d * (dtype == GDN_F32 ? 1 : 2);
  const int q_steps = (nq + step - 1) / step, k_steps = (nkv + step - 1) / step;
  auto side = [&](int steps, int* parts, int* per) -> int {
    *parts = *per = 1;
    if (!steps) return 0;
    int share = static_cast<int>(static_cast<int64_t>(slots) * steps / (q_steps + k_steps));
    if (share < 1) share = 1;
    int64_t cuts = (static_cast<int64_t>(share) * warps + rows - 1) / rows;
    if (cuts > steps) cuts = steps;
    const int run = (steps + static_cast<int>(cuts) - 1) / static_cast<int>(cuts);
    *per = run * step;
    *parts = (steps + run - 1) / run;
    const int64_t need = (static_cast<int64_t>(rows) * *parts + warps - 1) / warps;
    return need < share ? static_cast<int>(need) : share;
  };
  p.q_ctas = side(q_steps, &p.q_parts, &p.q_per);
  const int grid = p.q_ctas + side(k_steps, &p.k_parts, &p.k_per);
  by_type(dtype, [&](auto t) {
    by_head(d, next, [&](auto dim, auto pairs) {
      gdn::gdn_head_norm_rope_bwd_kernel<decltype(t), dim.value, pairs.value><<<grid, gdn::kNormBwdThreads, 0, s>>>(p);
    });
  });
  if (sums) {
    const float* parts = p.partials;
    launch_early(gdn::gdn_norm_weight_sum_kernel, dim3(static_cast<unsigned>(d / 32), 2), 1024, 0, s, parts, d, p.q_ctas,
                 grid, dq_weight, dk_weight);  // a refusal is launched()'s to report
  }
  int rc = launched(sums ? 2 : 1);
  if (sums && !workspace) {
    cudaError_t e = cudaFreeAsync(ws, s);
    if (e != cudaSuccess && rc == GDN_OK) rc = fail(GDN_ERR_CUDA, "cudaFreeAsync: %s", cudaGetErrorString(e));
  }
  return rc;
}

int gdn_paged_append(const void* k, const void* v, const gdn_paged_t* cache, const int32_t* positions,
                     const gdn_rope_t* rope, int norm, const float* k_weight, float eps, int nkv, int d, int dtype,
                     int64_t k_stride, int64_t v_stride, void* stream) {
  g_err[0] = 0;
  g_launches = 0;
  gdn::AppendParams p{};
  int next = 0;
  if (nkv < 1) return fail(GDN_ERR_ARG, "nkv = %d must be positive", nkv);
  if (int rc = check_head_dim(d)) return rc;
  if (dtype != GDN_BF16 && dtype != GDN_F16) return fail(GDN_ERR_UNSUPPORTED, "dtype %d is neither bf16 nor fp16", dtype);
  if (norm != 0 && norm != 1) return fail(GDN_ERR_ARG, "norm must be 0 or 1");
  if (!norm && k_weight) return fail(GDN_ERR_ARG, "k_weight is given without norm");
  if (!(eps >= 0.f)) return fail(GDN_ERR_ARG, "eps must not be negative");
  if (int rc = check_rope(rope, d, &p.rope, &next)) return rc;
  if (int rc = check_paged(cache, nkv, d, &p.cache)) return rc;
  const int64_t w = static_cast<int64_t>(nkv) * d;
  p.k_stride = k_stride ? k_stride : w;
  p.v_stride = v_stride ? v_stride : w;
  if (int rc = check_stride(p.k_stride, w, "k")) return rc;
  if (int rc = check_stride(p.v_stride, w, "v")) return rc;
  const int unroll = norm_unroll(nkv, d);
  p.chunks = norm_chunks(nkv, d, unroll);
  const int64_t items = static_cast<int64_t>(cache->rows) * p.chunks;
  if (items > INT32_MAX - (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "%d rows of %d heads exceed the item range", cache->rows, nkv);
  if (cache->rows == 0) return GDN_OK;
  if (!k || !v) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_weight)) return fail(GDN_ERR_ARG, "k, v and k_weight must be 16-byte aligned");
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  p.k = k;
  p.v = v;
  p.positions = positions;
  p.k_weight = k_weight;
  p.nkv = nkv;
  p.norm = norm;
  p.eps = eps;
  p.status = dev->status;
  const int warps = gdn::kNormThreads / 32;
  const unsigned grid = static_cast<unsigned>((items + warps - 1) / warps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_type16(dtype, [&](auto t) {
    by_head(d, next, [&](auto dim, auto pairs) {
      by_unroll(unroll, [&](auto u) {
        gdn::gdn_paged_append_kernel<decltype(t), dim.value, pairs.value, u.value><<<grid, gdn::kNormThreads, 0, s>>>(p);
      });
    });
  });
  return launched(1);
}

size_t gdn_tree_attention_workspace_bytes(int nq, int nkv, int d) {
  if (nq <= 0 || nkv <= 0 || (d != 64 && d != 128)) return 0;
  size_t most = 0;
  for (AttnKind kind : {kAttn16, kAttnTc}) {
    const size_t n = attn_layout(kind, plan_sms(), d).total;
    if (n > most) most = n;
  }
  return most;
}

int gdn_tree_attention(const void* q, const gdn_paged_t* cache, const uint64_t* mask, int mask_words, float scale,
                       void* out, int nq, int nkv, int d, int dtype, int64_t q_stride, int64_t out_stride,
                       int max_rows, void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  g_launches = 0;
  gdn::AttnParams p{};
  if (nq < 1 || nkv < 1) return fail(GDN_ERR_ARG, "head counts nq = %d, nkv = %d must be positive", nq, nkv);
  if (nq % nkv) return fail(GDN_ERR_UNSUPPORTED, "nq = %d is not a multiple of nkv = %d", nq, nkv);
  if (int rc = check_head_dim(d)) return rc;
  if (dtype != GDN_BF16 && dtype != GDN_F16) return fail(GDN_ERR_UNSUPPORTED, "dtype %d is neither bf16 nor fp16", dtype);
  p.scale_log2 = scale * 1.4426950408889634f;  // log2 e
  if (!(p.scale_log2 - p.scale_log2 == 0.f)) return fail(GDN_ERR_ARG, "scale must be finite, and so its product with log2 e");
  if (mask && mask_words < 1) return fail(GDN_ERR_ARG, "mask_words = %d must be positive", mask_words);
  if (max_rows < 0) return fail(GDN_ERR_ARG, "max_rows = %d is negative", max_rows);
  if (int rc = check_paged(cache, nkv, d, &p.cache)) return rc;
  const int64_t w = static_cast<int64_t>(nq) * d;
  p.q_stride = q_stride ? q_stride : w;
  p.out_stride = out_stride ? out_stride : w;
  if (int rc = check_stride(p.q_stride, w, "q")) return rc;
  if (int rc = check_stride(p.out_stride, w, "out")) return rc;
  if (static_cast<int64_t>(cache->rows) * nq > INT32_MAX - 4096)
    return fail(GDN_ERR_UNSUPPORTED, "%d rows of %d heads exceed the 2^31 row range", cache->rows, nq);
  if (cache->rows == 0) return GDN_OK;
  if (!q || !out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(GDN_ERR_ARG, "q and out must be 16-byte aligned");
  const size_t need = gdn_tree_attention_workspace_bytes(nq, nkv, d);
  if (workspace) {
    if (workspace_bytes < need)
      return fail(GDN_ERR_ARG, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, need);
    if (!aligned256(workspace)) return fail(GDN_ERR_ARG, "workspace must be 256-byte aligned");
  }
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = workspace;
  if (!ws) {
    cudaError_t e = cudaMallocAsync(&ws, need, s);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaMallocAsync(%zu): %s", need, cudaGetErrorString(e));
  }
  p.q = q;
  p.out = out;
  p.out_wide = reinterpret_cast<uintptr_t>(out) % 32 == 0 && p.out_stride % 16 == 0;
  p.mask = mask;
  p.mask_words = mask_words;
  p.nq = nq;
  p.nkv = nkv;
  p.group = nq / nkv;
  p.status = dev->status;
  const int most = !cache->cu_rows ? 1 : (max_rows && max_rows < cache->rows ? max_rows : cache->rows);
  const AttnKind kind = attn_kind(static_cast<int64_t>(most) * p.group, scale);
  p.runs = attn_runs(kind, dev->sms);
  p.whole = attn_whole(kind, dev->sms, p, most);
  CUtensorMap maps[2] = {};
  if (kind == kAttnTc) {
    // strides that TMA cannot take (or no pages at all) leave the copies to the threads
    p.box = cache->num_pages > 0 ? attn_box(cache->page_size) : 0;
    if (p.box && (!cache_map(&maps[0], cache->k, cache->k_page, cache->k_token, cache->k_head, p.cache, nkv, d, p.box, dtype) ||
                  !cache_map(&maps[1], cache->v, cache->v_page, cache->v_token, cache->v_head, p.cache, nkv, d, p.box, dtype)))
      p.box = 0;
  }
  const AttnLayout l = attn_layout(kind, dev->sms, d);
  p.cut = reinterpret_cast<int4*>(static_cast<char*>(ws) + l.cut);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + l.ml);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + l.o);
  cudaError_t e = cudaSuccess;
  by_type16(dtype, [&](auto t) {
    e = d == 64 ? launch_attn<decltype(t), 64>(kind, dev->sms, p, maps[0], maps[1], s)
                : launch_attn<decltype(t), 128>(kind, dev->sms, p, maps[0], maps[1], s);
  });
  int rc = e != cudaSuccess ? fail(GDN_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e)) : launched(p.whole ? 1 : 2);
  if (!workspace) {
    e = cudaFreeAsync(ws, s);
    if (e != cudaSuccess && rc == GDN_OK) rc = fail(GDN_ERR_CUDA, "cudaFreeAsync: %s", cudaGetErrorString(e));
  }
  return rc;
}

}  // extern "C"
