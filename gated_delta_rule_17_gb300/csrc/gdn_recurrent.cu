// Host side of the entry points in include/gdn_recurrent.h: argument checks (each rejection names the
// guard) and launches. A translation unit of its own, compiled beside gdn_api.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <type_traits>

#include "gdn_recurrent.h"
#include "gdn_host.h"
#include "gdn_conv_kernel.cuh"
#include "gdn_layer_norm_kernel.cuh"
#include "gdn_ssm_scan_kernel.cuh"

namespace {

int fail(int code, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return gdn_host::refuse(code, text);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launched(int launches) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  gdn_host::count(launches);
  return GDN_OK;
}

template <int N>
using IntC = std::integral_constant<int, N>;

template <typename F>
void by_type(int dtype, F&& f) {
  if (dtype == GDN_F32) f(float{});
  else if (dtype == GDN_F16) f(__half{});
  else f(__nv_bfloat16{});
}

int check_type(int dtype) {
  if (dtype != GDN_BF16 && dtype != GDN_F16 && dtype != GDN_F32) return fail(GDN_ERR_UNSUPPORTED, "dtype %d is unknown", dtype);
  return GDN_OK;
}

// A row stride (0: packed) that holds `least` elements and keeps rows on 16 bytes.
int take_stride(int64_t given, int64_t least, const char* name, int64_t* out) {
  *out = given ? given : least;
  if (*out < least || *out % 8)
    return fail(GDN_ERR_ARG, "%s row stride %lld must be >= %lld and a multiple of 8", name, (long long)*out, (long long)least);
  return GDN_OK;
}

int check_flag(int value, const char* name) {
  if (value != 0 && value != 1) return fail(GDN_ERR_ARG, "%s must be 0 or 1", name);
  return GDN_OK;
}

// An output in the place of an input takes its rows' stride too.
struct Same {
  const char *out_name, *in_name;
  const void *out, *in;
  int64_t out_stride, in_stride;
};
int check_same(const Same& s) {
  if (s.out && s.out == s.in && s.out_stride != s.in_stride)
    return fail(GDN_ERR_ARG, "%s in the place of %s needs its row stride: %lld, not %lld", s.out_name, s.in_name, (long long)s.in_stride, (long long)s.out_stride);
  return GDN_OK;
}

int check_batch(int B, int T, const int32_t* cu, gdn::Rows* out) {
  if (B < 0 || T < 0) return fail(GDN_ERR_ARG, "B = %d or T = %d is negative", B, T);
  const int64_t rows = cu ? T : static_cast<int64_t>(B) * T;
  if (rows > INT32_MAX - 65536) return fail(GDN_ERR_UNSUPPORTED, "%lld rows exceed the 2^31 row range", (long long)rows);
  *out = gdn::Rows{cu, B, T, static_cast<int>(rows)};
  return GDN_OK;
}

int check_workspace(const void* ws, size_t given, size_t need) {
  if (!ws) return GDN_OK;
  if (given < need) return fail(GDN_ERR_ARG, "workspace of %zu bytes is smaller than the %zu required", given, need);
  if (!aligned(ws, 256)) return fail(GDN_ERR_ARG, "workspace must be 256-byte aligned");
  return GDN_OK;
}

// The caller's workspace, or one from the stream's pool that release() gives back.
int acquire(void* given, size_t need, cudaStream_t s, void** ws) {
  *ws = given;
  if (given || !need) return GDN_OK;
  cudaError_t e = cudaMallocAsync(ws, need, s);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaMallocAsync(%zu): %s", need, cudaGetErrorString(e));
  return GDN_OK;
}
int release(void* given, void* ws, cudaStream_t s, int rc) {
  if (given || !ws) return rc;
  cudaError_t e = cudaFreeAsync(ws, s);
  if (e != cudaSuccess && rc == GDN_OK) rc = fail(GDN_ERR_CUDA, "cudaFreeAsync: %s", cudaGetErrorString(e));
  return rc;
}

int zero(float* p, int64_t n, cudaStream_t s) {
  if (!p) return GDN_OK;
  cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(n) * sizeof(float), s);
  return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
}

// A launch that may start while the kernel before it in the stream ends; these kernels wait for that
// one (tc::grid_dependency_wait) before they read or write global memory.
template <typename... A, typename... B>
void launch_early(void (*kernel)(A...), int64_t grid, int threads, int shared, cudaStream_t s, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(shared);
  cfg.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, args...);  // a refusal is launched()'s to report
}

// ---- convolution ---------------------------------------------------------------------

constexpr int kConvMaxD = 1 << 26;  // (width + 1) D in 32 bits

template <typename F>
void by_width(int width, F&& f) {
  if (width == 2) f(IntC<2>{});
  else if (width == 3) f(IntC<3>{});
  else f(IntC<4>{});
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Rows of a thread's strip: as few as make `waves` passes of all the threads that the SMs hold (512 each), so that the last pass
// is as full as the others.
int conv_strips(int64_t rows, int words, int sms, int waves, int least) {
  const int64_t strips = static_cast<int64_t>(sms) * 512 * waves / words;
  const int64_t strip = strips > 1 ? (rows + strips - 1) / strips : rows;
  return static_cast<int>(strip < least ? least : strip);
}
int conv_strip(int64_t rows, int words, int sms) { return conv_strips(rows, words, sms, 4, 1); }
// The backward's walk width - 1 rows more and leave partial sums, so they are longer.
int conv_bwd_strip(int64_t rows, int words, int sms) { return conv_strips(rows, words, sms, 2, 16); }

int conv_setup(const void* x, const float* weight, const float* bias, int D, int width, int silu, int dtype, int64_t x_stride,
               gdn::ConvParams* p) {
  if (D < 8 || D % 8 || D > kConvMaxD) return fail(GDN_ERR_UNSUPPORTED, "D = %d is not a multiple of 8 in 8..%d", D, kConvMaxD);
  if (static_cast<int64_t>(p->batch.B) * D > static_cast<int64_t>(INT32_MAX) * 128)  // CTAs of a thread for four channels of a state
    return fail(GDN_ERR_UNSUPPORTED, "%d sequences of %d channels exceed the item range", p->batch.B, D);
  if (width < 2 || width > 4) return fail(GDN_ERR_UNSUPPORTED, "width = %d is not 2, 3 or 4", width);
  if (int rc = check_type(dtype)) return rc;
  if (int rc = check_flag(silu, "silu")) return rc;
  if (int rc = take_stride(x_stride, D, "x", &p->x_stride)) return rc;
  if (!weight) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 16)) return fail(GDN_ERR_ARG, "x, weight and bias must be 16-byte aligned");
  p->x = x;
  p->weight = weight;
  p->bias = bias;
  p->D = D;
  p->silu = silu;
  return GDN_OK;
}

// ---- layer norm ----------------------------------------------------------------------

constexpr int kNormMaxDim = 8192;

// Calls f with the lanes of a group and the words of eight values that each holds.
template <typename F>
void by_dim(int dim, F&& f) {
  if (dim <= 16) f(IntC<2>{}, IntC<1>{});
  else if (dim <= 64) f(IntC<8>{}, IntC<1>{});
  else if (dim <= 128) f(IntC<16>{}, IntC<1>{});
  else if (dim <= 256) f(IntC<32>{}, IntC<1>{});
  else if (dim <= 1024) f(IntC<32>{}, IntC<4>{});
  else if (dim <= 4096) f(IntC<128>{}, IntC<4>{});
  else f(IntC<256>{}, IntC<4>{});
}
// The backward keeps the columns' weights and sums too, so a group takes more lanes, the more with a gate: of one warp up to 256
// values (f gets the lanes and 0), a CTA beyond (threads, and words a thread).
template <bool kGate, typename F>
void by_dim_backward(int dim, F&& f) {
  if (dim <= 16) f(IntC<2>{}, IntC<0>{});
  else if (dim <= 64) f(IntC<8>{}, IntC<0>{});
  else if (dim <= 128) f(IntC<16>{}, IntC<0>{});
  else if (dim <= 256) f(IntC<32>{}, IntC<0>{});
  else if (dim <= 1024) f(IntC<128>{}, IntC<1>{});
  else if constexpr (kGate) dim <= 4096 ? f(IntC<512>{}, IntC<1>{}) : f(IntC<1024>{}, IntC<1>{});
  else dim <= 4096 ? f(IntC<256>{}, IntC<2>{}) : f(IntC<512>{}, IntC<2>{});
}

// CTAs and ring of the backward. The ring's stages fill what an SM's CTAs share of 200 KB, eight at most.
struct NormPlan {
  int ctas, stages, ring;
};
template <bool kGate>
NormPlan norm_plan(int64_t items, int dim, int sms, int element) {
  NormPlan p{};
  by_dim_backward<kGate>(dim, [&](auto lanes, auto words) {
    constexpr int L = lanes.value;
    int per_sm = kGate ? 4 : gdn::kNormSmallCtas;
    int64_t need = items;
    if constexpr (words.value == 0) {
      need = (items + 128 / L - 1) / (128 / L);
    } else {
      const int stage = (kGate ? 3 : 2) * dim * element;
      per_sm = gdn::norm_wide_ctas<L, kGate>;
      p.stages = 200 * 1024 / per_sm / stage;
      if (p.stages > 8) p.stages = 8;
      p.ring = p.stages * stage;
    }
    const int64_t most = static_cast<int64_t>(sms) * per_sm;
    p.ctas = static_cast<int>(need < most ? need : most);
  });
  return p;
}

// Lets a kernel take the ring's shared memory, once a device (the types name the kernel).
template <typename T, int L, int NV, bool G>
int allow_shared(const void* kernel) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (done.load() >> dev & 1)) return GDN_OK;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  if (dev < 64) done.fetch_or(uint64_t{1} << dev);
  return GDN_OK;
}

int layer_norm_setup(const void* x, const void* gate, const float* weight, const float* bias, float eps, int rows, int groups, int dim,
                     int dtype, int rms, int gate_first, const gdn_layer_norm_strides_t* st, gdn::LayerNormParams* p) {
  *p = gdn::LayerNormParams{};
  if (rows < 0) return fail(GDN_ERR_ARG, "rows = %d is negative", rows);
  if (groups < 1) return fail(GDN_ERR_ARG, "groups = %d must be positive", groups);
  if (dim < 8 || dim % 8 || dim > kNormMaxDim)
    return fail(GDN_ERR_UNSUPPORTED, "dim = %d is not a multiple of 8 in 8..%d", dim, kNormMaxDim);
  if (int rc = check_type(dtype)) return rc;
  if (int rc = check_flag(rms, "rms")) return rc;
  if (int rc = check_flag(gate_first, "gate_first")) return rc;
  if (gate_first && !gate) return fail(GDN_ERR_ARG, "gate_first without a gate");
  if (!(eps >= 0.f)) return fail(GDN_ERR_ARG, "eps must not be negative");
  const int64_t width = static_cast<int64_t>(groups) * dim;
  if (int rc = take_stride(st ? st->x : 0, width, "x", &p->x_stride)) return rc;
  if (gate)
    if (int rc = take_stride(st ? st->gate : 0, width, "gate", &p->gate_stride)) return rc;
  if (int rc = take_stride(st ? st->out : 0, width, "out", &p->out_stride)) return rc;
  if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(weight, 16) || !aligned(bias, 16))
    return fail(GDN_ERR_ARG, "x, gate, weight and bias must be 16-byte aligned");
  p->items = static_cast<int64_t>(rows) * groups;
  if (p->items > INT32_MAX - 65536 || width > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%d rows of %d groups exceed the item range", rows, groups);
  if (rows && !x) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  p->x = x;
  p->gate = gate;
  p->weight = weight;
  p->bias = bias;
  p->groups = groups;
  p->dim = dim;
  p->rms = rms;
  p->gate_first = gate_first;
  p->eps = eps;
  return GDN_OK;
}

// ---- state space scan ----------------------------------------------------------------

template <typename F>
void by_state(int dk, int dv, F&& f) {
  if (dk == 64) dv == 64 ? f(IntC<64>{}, IntC<64>{}) : f(IntC<64>{}, IntC<128>{});
  else dv == 64 ? f(IntC<128>{}, IntC<64>{}) : f(IntC<128>{}, IntC<128>{});
}

int ssm_setup(const void* q, const void* k, const void* v, const void* dt, const float* a, const float* dt_bias, const float* skip,
              void* state, void* out, int nk, int nv, int dk, int dv, const gdn_ssm_options_t* o, int64_t rows, gdn::SsmParams* p) {
  if (nk < 1 || nv < 1) return fail(GDN_ERR_ARG, "head counts nk = %d, nv = %d must be positive", nk, nv);
  if (nv % nk) return fail(GDN_ERR_UNSUPPORTED, "nv = %d is not a multiple of nk = %d", nv, nk);
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return fail(GDN_ERR_UNSUPPORTED, "dk = %d or dv = %d is neither 64 nor 128", dk, dv);
  const int64_t wk = static_cast<int64_t>(nk) * dk, wv = static_cast<int64_t>(nv) * dv;
  if (wv > INT32_MAX || wk > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%d heads of %d values exceed a row's range", nv, dv);
  if (int rc = take_stride(o ? o->q : 0, wk, "q", &p->q_stride)) return rc;
  if (int rc = take_stride(o ? o->k : 0, wk, "k", &p->k_stride)) return rc;
  if (int rc = take_stride(o ? o->v : 0, wv, "v", &p->v_stride)) return rc;
  if (int rc = take_stride(o ? o->out : 0, wv, "out", &p->out_stride)) return rc;
  p->dt_stride = o && o->dt ? o->dt : nv;
  if (p->dt_stride < nv) return fail(GDN_ERR_ARG, "dt row stride %lld must be >= nv = %d", (long long)p->dt_stride, nv);
  p->state_is_table = o ? o->state_is_table : 0;
  p->dt_bf16 = o ? o->dt_bf16 : 0;
  p->softplus = o ? o->softplus : 1;
  if (int rc = check_flag(p->state_is_table, "state_is_table")) return rc;
  if (int rc = check_flag(p->dt_bf16, "dt_bf16")) return rc;
  if (int rc = check_flag(p->softplus, "softplus")) return rc;
  if (rows == 0) return GDN_OK;
  if (!q || !k || !v || !dt || !a || !state || !out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(state, p->state_is_table ? 8 : 16))
    return fail(GDN_ERR_ARG, "q, k, v, out and state must be 16-byte aligned");
  if (!aligned(dt, p->dt_bf16 ? 2 : 4) || !aligned(a, 4) || !aligned(dt_bias, 4) || !aligned(skip, 4))
    return fail(GDN_ERR_ARG, "dt, a, dt_bias and skip must be aligned to their elements");
  p->q = static_cast<const __nv_bfloat16*>(q);
  p->k = static_cast<const __nv_bfloat16*>(k);
  p->v = static_cast<const __nv_bfloat16*>(v);
  p->dt = dt;
  p->a = a;
  p->dt_bias = dt_bias;
  p->skip = skip;
  p->state = state;
  p->out = static_cast<__nv_bfloat16*>(out);
  p->nk = nk;
  p->nv = nv;
  return GDN_OK;
}

// [rows][heads * d] bf16 rows as boxes of 64 values and a chunk of tokens.
int ssm_map(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int64_t stride, const char* name) {
  auto fn = gdn_host::encode_fn();
  if (!fn) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[2] = {64, gdn::kSsmChunk}, estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed (%d)", name, static_cast<int>(r));
  return GDN_OK;
}

// CTAs of a sequence: two slices of 64 value columns of one key head each.
int ssm_pairs(int nk, int nv, int dv) { return nk * ((nv / nk * (dv / 64) + 1) / 2); }

// Segments of the scan: how many chunks each (0: whole sequences), the items (sequences or segments) that there may be, and
// the workspace for them.
struct SsmSegments {
  int segment, items;
  size_t states, total;
};
SsmSegments ssm_segments(int64_t B, int64_t T, bool varlen, int pairs, int nv, int dk, int dv, int sms) {
  SsmSegments r{0, static_cast<int>(B), 0, 0};
  const int64_t chunks = (T + gdn::kSsmChunk - 1) / gdn::kSsmChunk;
  if (!varlen) {
    // n segments of `per` chunks: the passes of all CTAs, the first of segments 1 to n - 1 at 0.6 of a chunk's time, and what a pass costs
    // by itself, about three chunks' time
    auto passes = [&](int64_t ctas) { return static_cast<double>((ctas + sms - 1) / sms); };
    double best = passes(B * pairs) * static_cast<double>(chunks);
    for (int n = 2; n <= 32; ++n) {
      const int64_t per = (chunks + n - 1) / n;
      if (per < 4) break;
      const double time = passes(B * pairs * (n - 1)) * (0.6 * static_cast<double>(per) + 3) + passes(B * pairs * n) * static_cast<double>(per) + 3 + 0.1 * n;
      if (time < 0.9 * best) {
        best = time;
        r.segment = static_cast<int>(per);
      }
    }
    if (r.segment) r.items = static_cast<int>(B * ((chunks + r.segment - 1) / r.segment));
  } else if (B > 0 && B <= 32) {
    // the lengths are the device's to see; it takes segments where the longest sequence stands out. Of half the chunks that every SM would
    // have of an even share
    const int64_t per = (chunks * pairs / sms + 1) / 2, segment = per < 8 ? 8 : per;
    if (chunks / B > 0 && chunks > 4 * segment) {
      r.segment = static_cast<int>(segment);
      r.items = static_cast<int>(B + chunks / segment + 1);
    }
  }
  if (r.segment) {
    r.states = align256(static_cast<size_t>(r.items + 1) * nv * dk * dv * sizeof(float));
    r.total = r.states + align256(static_cast<size_t>(r.items) * nv * sizeof(float));
  }
  return r;
}

// Shared memory of the scan's kernels, once a device.
int ssm_attributes() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  if (e == cudaSuccess && dev < 64 && done[dev]) return GDN_OK;
  for (int dk : {64, 128})
    for (int dv : {64, 128})
      by_state(dk, dv, [&](auto K, auto V) {
        for (const void* f : {reinterpret_cast<const void*>(gdn::gdn_ssm_scan_kernel<K.value, V.value, true>),
                              reinterpret_cast<const void*>(gdn::gdn_ssm_scan_kernel<K.value, V.value, false>)})
          if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, gdn::SsmPlan::DYN_SMEM);
      });
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  if (dev < 64) done[dev] = true;
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_causal_conv(const void* x, const float* weight, const float* bias, void* state, void* out, int B, int T, int D, int width,
                    int silu, int dtype, int state_is_table, int64_t x_stride, int64_t out_stride, const int32_t* cu_seqlens,
                    void* stream) {
  gdn_host::begin();
  gdn::ConvParams p{};
  if (int rc = check_batch(B, T, cu_seqlens, &p.batch)) return rc;
  if (int rc = conv_setup(x, weight, bias, D, width, silu, dtype, x_stride, &p)) return rc;
  if (int rc = take_stride(out_stride, D, "out", &p.out_stride)) return rc;
  if (int rc = check_flag(state_is_table, "state_is_table")) return rc;
  if (B && state_is_table && !state) return fail(GDN_ERR_ARG, "a state table without its pointer");
  if (B == 0 || p.batch.rows == 0) return GDN_OK;
  if (!x || !out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (x == out) return fail(GDN_ERR_ARG, "out must not be x: a row's inputs are read by several threads");
  if (!aligned(out, 16) || !aligned(state, state_is_table ? 8 : 16)) return fail(GDN_ERR_ARG, "out and state must be 16-byte aligned");
  p.state = state;
  p.out = out;
  p.state_is_table = state_is_table;
  int sms = 0;
  if (int rc = gdn_host::device(&sms, &p.status)) return rc;
  const int words = D / (dtype == GDN_F32 ? 4 : 8), rows = p.batch.rows;
  p.strip = conv_strip(rows, words, sms);
  if (!cu_seqlens) {  // whole sequences in a strip where they are short
    if (p.strip < T && T <= 16) p.strip = T;
    if (p.strip >= T) {
      p.strip -= p.strip % T;
      p.state_here = 1;
    }
  }
  p.strips = ceil_div(rows, p.strip);
  const int64_t threads = static_cast<int64_t>(p.strips) * words;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool after = state && !p.state_here;
  by_type(dtype, [&](auto t) {
    by_width(width, [&](auto w) {
      launch_early(gdn::gdn_conv_kernel<decltype(t), w.value>, ceil_div(threads, gdn::kConvThreads), gdn::kConvThreads, 0, s, p);
      if (after)
        launch_early(gdn::gdn_conv_state_kernel<decltype(t), w.value>, ceil_div(static_cast<int64_t>(B) * words, gdn::kConvThreads),
                     gdn::kConvThreads, 0, s, p);
    });
  });
  return launched(after ? 2 : 1);
}

size_t gdn_causal_conv_backward_workspace_bytes(int rows, int D, int width) {
  if (rows <= 0 || D < 8 || D % 8 || D > kConvMaxD || width < 2 || width > 4) return 0;
  const int strip = conv_bwd_strip(rows, D / 4, gdn_host::plan_sms());
  return static_cast<size_t>(ceil_div(rows, strip)) * (width + 1) * D * sizeof(float);
}

int gdn_causal_conv_backward(const void* x, const float* weight, const float* bias, const void* h0, const void* dout,
                             const void* dST, void* dx, float* dweight, float* dbias, void* dh0, int B, int T, int D, int width,
                             int silu, int dtype, int64_t x_stride, int64_t dout_stride, int64_t dx_stride,
                             const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_host::begin();
  gdn::ConvParams p{};
  if (int rc = check_batch(B, T, cu_seqlens, &p.batch)) return rc;
  if (int rc = conv_setup(x, weight, bias, D, width, silu, dtype, x_stride, &p)) return rc;
  if (int rc = take_stride(dout_stride, D, "dout", &p.dout_stride)) return rc;
  if (int rc = take_stride(dx_stride, D, "dx", &p.dx_stride)) return rc;
  const int rows = B == 0 ? 0 : p.batch.rows;
  if (rows && (!x || !dout || !dx)) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (rows && (dx == x || dx == dout)) return fail(GDN_ERR_ARG, "dx must not be x or dout: a row's are read by several threads");
  if (!aligned(dout, 16) || !aligned(dx, 16) || !aligned(h0, 16) || !aligned(dST, 16) || !aligned(dh0, 16))
    return fail(GDN_ERR_ARG, "dout, dx, h0, dST and dh0 must be 16-byte aligned");
  const bool sums = dweight || dbias;
  const size_t need = sums ? gdn_causal_conv_backward_workspace_bytes(rows, D, width) : 0;
  if (need)
    if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // sums over no rows
    if (int rc = zero(dweight, static_cast<int64_t>(D) * width, s)) return rc;
    if (int rc = zero(dbias, D, s)) return rc;
    if (B == 0 || !dh0) return GDN_OK;
  }
  int sms = 0;
  if (int rc = gdn_host::device(&sms, &p.status)) return rc;
  p.state = const_cast<void*>(h0);
  p.dout = dout;
  p.dx = dx;
  p.dlast = dST;
  p.dfirst = dh0;
  p.dweight = dweight;
  p.dbias = dbias;
  const int words = D / 4;
  p.strip = conv_bwd_strip(rows, words, sms);
  p.strips = ceil_div(rows, p.strip);
  void* ws = nullptr;
  if (int rc = acquire(need ? workspace : nullptr, need, s, &ws)) return rc;
  p.partials = static_cast<float*>(ws);
  const int sum_ctas = need ? ceil_div(static_cast<int64_t>(width + 1) * D, 32) : 0;
  const int end_ctas = dh0 ? ceil_div(static_cast<int64_t>(B) * words, gdn::kConvSumThreads) : 0;
  by_type(dtype, [&](auto t) {
    by_width(width, [&](auto w) {
      if (rows)
        launch_early(gdn::gdn_conv_bwd_kernel<decltype(t), w.value>, ceil_div(static_cast<int64_t>(p.strips) * words, gdn::kConvThreads),
                     gdn::kConvThreads, 0, s, p);
      if (sum_ctas + end_ctas)
        launch_early(gdn::gdn_conv_bwd_ends_kernel<decltype(t), w.value>, sum_ctas + end_ctas, gdn::kConvSumThreads, 0, s, p, sum_ctas);
    });
  });
  return release(need ? workspace : nullptr, ws, s, launched((rows > 0) + (sum_ctas + end_ctas > 0)));
}

size_t gdn_ssm_scan_workspace_bytes(int B, int T, int nk, int nv, int dk, int dv, int varlen) {
  if (B <= 0 || T <= 0 || nk < 1 || nv < 1 || nv % nk || (dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return 0;
  return ssm_segments(B, T, varlen != 0, ssm_pairs(nk, nv, dv), nv, dk, dv, gdn_host::plan_sms()).total;
}

int gdn_ssm_scan(const void* q, const void* k, const void* v, const void* dt, const float* a, const float* dt_bias, const float* skip,
                 void* state, void* out, int B, int T, int nk, int nv, int dk, int dv, const gdn_ssm_options_t* options,
                 const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_host::begin();
  gdn::SsmParams p{};
  if (int rc = check_batch(B, T, cu_seqlens, &p.batch)) return rc;
  const int rows = B == 0 ? 0 : p.batch.rows;
  if (int rc = ssm_setup(q, k, v, dt, a, dt_bias, skip, state, out, nk, nv, dk, dv, options, rows, &p)) return rc;
  if (rows == 0) return GDN_OK;
  if (out == v || out == q || out == k) return fail(GDN_ERR_ARG, "out must not be q, k or v: rows are read by several CTAs");
  int sms = 0;
  if (int rc = gdn_host::device(&sms, &p.status)) return rc;
  gdn::SsmScanParams sp{};
  sp.pairs = ssm_pairs(nk, nv, dv);
  sp.sms = sms;
  const SsmSegments seg = ssm_segments(B, T, cu_seqlens != nullptr, sp.pairs, nv, dk, dv, sms);
  if (static_cast<int64_t>(seg.items) * sp.pairs > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%d sequences of %d heads exceed the item range", B, nv);
  if (seg.total)
    if (int rc = check_workspace(workspace, workspace_bytes, seg.total)) return rc;
  if (int rc = ssm_attributes()) return rc;
  CUtensorMap q_map, k_map, v_map, out_map;
  if (int rc = ssm_map(&q_map, q, static_cast<int64_t>(nk) * dk, rows, p.q_stride, "q")) return rc;
  if (int rc = ssm_map(&k_map, k, static_cast<int64_t>(nk) * dk, rows, p.k_stride, "k")) return rc;
  if (int rc = ssm_map(&v_map, v, static_cast<int64_t>(nv) * dv, rows, p.v_stride, "v")) return rc;
  if (int rc = ssm_map(&out_map, out, static_cast<int64_t>(nv) * dv, rows, p.out_stride, "out")) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* given = seg.total ? workspace : nullptr;
  void* ws = nullptr;
  if (int rc = acquire(given, seg.total, s, &ws)) return rc;
  sp.s = p;
  sp.segment = seg.segment;
  sp.states = static_cast<float*>(ws);
  sp.decays = seg.total ? reinterpret_cast<float*>(static_cast<char*>(ws) + seg.states) : nullptr;
  const int grid = seg.items * sp.pairs;
  by_state(dk, dv, [&](auto K, auto V) {
    auto go = [&](auto kernel) { launch_early(kernel, grid, gdn::kSsmThreads, gdn::SsmPlan::DYN_SMEM, s, q_map, k_map, v_map, out_map, sp); };
    if (seg.segment) go(gdn::gdn_ssm_scan_kernel<K.value, V.value, false>);
    go(gdn::gdn_ssm_scan_kernel<K.value, V.value, true>);
  });
  return release(given, ws, s, launched(seg.segment ? 2 : 1));
}

int gdn_ssm_decode(const void* q, const void* k, const void* v, const void* dt, const float* a, const float* dt_bias, const float* skip,
                   void* state, void* out, int B, int nk, int nv, int dk, int dv, const gdn_ssm_options_t* options, void* stream) {
  gdn_host::begin();
  gdn::SsmParams p{};
  if (int rc = check_batch(B, 1, nullptr, &p.batch)) return rc;
  if (int rc = ssm_setup(q, k, v, dt, a, dt_bias, skip, state, out, nk, nv, dk, dv, options, B, &p)) return rc;
  if (static_cast<int64_t>(B) * nv > INT32_MAX) return fail(GDN_ERR_UNSUPPORTED, "%d sequences of %d heads exceed the item range", B, nv);
  if (B == 0) return GDN_OK;
  if (out == q || out == k) return fail(GDN_ERR_ARG, "out must not be q or k: a row's are read by several CTAs");
  if (int rc = check_same({"out", "v", out, v, p.out_stride, p.v_stride})) return rc;
  int sms = 0;
  if (int rc = gdn_host::device(&sms, &p.status)) return rc;
  by_state(dk, dv, [&](auto K, auto V) {
    launch_early(gdn::gdn_ssm_decode_kernel<K.value, V.value>, B * nv, gdn::ssm_threads<K.value, V.value>, 0, static_cast<cudaStream_t>(stream), p);
  });
  return launched(1);
}

int gdn_layer_norm(const void* x, const void* gate, const float* weight, const float* bias, float eps, void* out, int rows, int groups,
                   int dim, int dtype, int rms, int gate_first, const gdn_layer_norm_strides_t* strides, void* stream) {
  gdn_host::begin();
  gdn::LayerNormParams p;
  if (int rc = layer_norm_setup(x, gate, weight, bias, eps, rows, groups, dim, dtype, rms, gate_first, strides, &p)) return rc;
  if (rows == 0) return GDN_OK;
  if (!out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned(out, 16)) return fail(GDN_ERR_ARG, "out must be 16-byte aligned");
  for (const auto& a : {Same{"out", "x", out, x, p.out_stride, p.x_stride}, Same{"out", "gate", out, gate, p.out_stride, p.gate_stride}})
    if (int rc = check_same(a)) return rc;
  int sms = 0;
  unsigned* status = nullptr;
  if (int rc = gdn_host::device(&sms, &status)) return rc;
  p.out = out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_type(dtype, [&](auto t) {
    by_dim(dim, [&](auto lanes, auto words) {
      constexpr int L = lanes.value, threads = gdn::norm_threads<L>;
      const int grid = ceil_div(p.items, threads / L * gdn::norm_rows<L, words.value>);
      if (gate) launch_early(gdn::gdn_layer_norm_kernel<decltype(t), L, words.value, true>, grid, threads, 0, s, p);
      else launch_early(gdn::gdn_layer_norm_kernel<decltype(t), L, words.value, false>, grid, threads, 0, s, p);
    });
  });
  return launched(1);
}

size_t gdn_layer_norm_backward_workspace_bytes(int rows, int groups, int dim) {
  if (rows <= 0 || groups < 1 || dim < 8 || dim % 8 || dim > kNormMaxDim) return 0;
  // (without a gate there are as many CTAs as with one, or more)
  return static_cast<size_t>(norm_plan<false>(static_cast<int64_t>(rows) * groups, dim, gdn_host::plan_sms(), 2).ctas) * 2 * dim * sizeof(float);
}

int gdn_layer_norm_backward(const void* x, const void* gate, const float* weight, const float* bias, float eps, const void* dout, void* dx,
                            void* dgate, float* dweight, float* dbias, int rows, int groups, int dim, int dtype, int rms, int gate_first,
                            const gdn_layer_norm_strides_t* strides, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_host::begin();
  gdn::LayerNormParams p;
  if (int rc = layer_norm_setup(x, gate, weight, bias, eps, rows, groups, dim, dtype, rms, gate_first, strides, &p)) return rc;
  const int64_t width = static_cast<int64_t>(groups) * dim;
  if (int rc = take_stride(strides ? strides->dout : 0, width, "dout", &p.dout_stride)) return rc;
  if (gate)
    if (int rc = take_stride(strides ? strides->dgate : 0, width, "dgate", &p.dgate_stride)) return rc;
  if (!gate && dgate) return fail(GDN_ERR_ARG, "dgate without a gate");
  if (rows && (!dout || !dx || (gate && !dgate))) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (!aligned(dout, 16) || !aligned(dx, 16) || !aligned(dgate, 16)) return fail(GDN_ERR_ARG, "dout, dx and dgate must be 16-byte aligned");
  const bool sums = dweight || dbias;
  const size_t need = sums ? gdn_layer_norm_backward_workspace_bytes(rows, groups, dim) : 0;
  if (need)
    if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  for (const auto& a : {Same{"dx", "x", dx, x, p.out_stride, p.x_stride}, Same{"dx", "dout", dx, dout, p.out_stride, p.dout_stride},
                        Same{"dx", "gate", dx, gate, p.out_stride, p.gate_stride}, Same{"dgate", "gate", dgate, gate, p.dgate_stride, p.gate_stride},
                        Same{"dgate", "x", dgate, x, p.dgate_stride, p.x_stride}, Same{"dgate", "dout", dgate, dout, p.dgate_stride, p.dout_stride}})
    if (int rc = check_same(a)) return rc;
  if (dx && dx == dgate) return fail(GDN_ERR_ARG, "dx and dgate must not be the same");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // sums over no rows
    if (int rc = zero(dweight, dim, s)) return rc;
    return zero(dbias, dim, s);
  }
  int sms = 0;
  unsigned* status = nullptr;
  if (int rc = gdn_host::device(&sms, &status)) return rc;
  p.dout = dout;
  p.out = dx;
  p.dgate = dgate;
  void* ws = nullptr;
  if (int rc = acquire(need ? workspace : nullptr, need, s, &ws)) return rc;
  p.partials = static_cast<float*>(ws);
  const int element = dtype == GDN_F32 ? 4 : 2;
  const NormPlan plan = gate ? norm_plan<true>(p.items, dim, sms, element) : norm_plan<false>(p.items, dim, sms, element);
  p.stages = plan.stages;
  p.status = status;
  int rc = GDN_OK;
  by_type(dtype, [&](auto type) {
    using T = decltype(type);
    auto go = [&](auto gated) {
      constexpr bool G = gated.value;
      by_dim_backward<G>(dim, [&](auto lanes, auto words) {
        constexpr int L = lanes.value, NV = words.value;
        if constexpr (NV == 0) {
          launch_early(gdn::gdn_layer_norm_bwd_kernel<T, L, G>, plan.ctas, 128, 0, s, p);
        } else {
          auto kernel = gdn::gdn_layer_norm_bwd_wide_kernel<T, L, NV, G>;
          rc = allow_shared<T, L, NV, G>(reinterpret_cast<const void*>(kernel));
          if (rc == GDN_OK) launch_early(kernel, plan.ctas, L, plan.ring, s, p);
        }
      });
    };
    if (gate) go(std::true_type{});
    else go(std::false_type{});
  });
  if (rc == GDN_OK) {
    if (sums)
      launch_early(gdn::gdn_layer_norm_sum_kernel, ceil_div(2 * dim, 32), 1024, 0, s, static_cast<const float*>(p.partials), plan.ctas, dim, dweight, dbias);
    rc = launched(sums ? 2 : 1);
  }
  return release(need ? workspace : nullptr, ws, s, rc);
}

}  // extern "C"
