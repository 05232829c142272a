// C ABI of the Float8 linear library (declared in include/fp8_linear.h):
// argument validation on the host, then asynchronous launches on the
// caller's stream.  Nothing here allocates or synchronizes; the only state
// is the per-device address of the no-allocation entry point's scratch
// array, looked up once per device.
#include "fp8l_internal.h"

#include <atomic>
#include <mutex>

namespace {

bool bad_dim(int64_t d) { return d < 0 || (d % 16) != 0 || d > (int64_t)1 << 30; }

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// FP8L_TENSORWISE or FP8L_ROWWISE, optionally with the FP8L_E5M2 flag
bool bad_scaling(int scaling) { return (scaling & ~(FP8L_ROWWISE | FP8L_E5M2)) != 0; }

// Dimensions are capped at 2^30 so that every 32-bit index in the kernels
// stays in range (addresses are formed in 64 bits), and a matrix at 2^40
// elements; a quantized one further, so that each launch has fewer than 2^32
// threads (quantize_fits).
constexpr int64_t kMaxElems = (int64_t)1 << 40;
// GEMM operands and outputs are addressed through buffer resources with
// 32-bit byte offsets: each must stay below 2^31 bytes.
constexpr int64_t kMaxGemmBytes = ((int64_t)1 << 31) - 1;

bool bad_gemm_sizes(int64_t m, int64_t n, int64_t k) {
  return m * k > kMaxGemmBytes || n * k > kMaxGemmBytes || 2 * m * n > kMaxGemmBytes;
}

// C[m,n] = A[m,k] . B[n,k]^T: a pointer may be NULL only where its matrix
// is empty; the scales are read whenever an output element is written.
int check_gemm_operands(const void *a, const float *sa, const void *b,
                        const float *sb, const void *c, int64_t m, int64_t n,
                        int64_t k) {
  if ((!a && m * k > 0) || (!b && n * k > 0) || (!c && m * n > 0)) return FP8L_EINVAL;
  if ((!sa || !sb) && m * n > 0) return FP8L_EINVAL;
  if (misaligned(a) || misaligned(b) || misaligned(c)) return FP8L_EALIGN;
  if ((reinterpret_cast<uintptr_t>(sa) & 3u) || (reinterpret_cast<uintptr_t>(sb) & 3u))
    return FP8L_EALIGN;
  return FP8L_OK;
}

// ---- scratch of fp8_linear_quantize_noalloc -------------------------------
// One array per GPU, held until the process ends; every noalloc call on a
// GPU uses that GPU's copy.  Host code never passes the array's name to a
// kernel (on the host it is only a stand-in for the symbol): it passes the
// device address that hipGetSymbolAddress returns for the device, taken
// once per device with that device current and kept in g_scratch.
static __device__ __align__(256) uint8_t scratch[FP8L_NOALLOC_MAX_WORKSPACE];

constexpr int kMaxDevices = 64;
std::atomic<void *> g_scratch[kMaxDevices];
std::mutex g_scratch_mu;

// The scratch address on the device of `stream` (the current device for the
// default stream); FP8L_EHIP if it cannot be found.
int scratch_address(hipStream_t stream, void **out) {
  int dev = -1;
  if (stream) {
    hipDevice_t d;
    if (hipStreamGetDevice(stream, &d) != hipSuccess) return FP8L_EHIP;
    dev = (int)d;
  } else if (hipGetDevice(&dev) != hipSuccess) {
    return FP8L_EHIP;
  }
  if (dev < 0 || dev >= kMaxDevices) return FP8L_EHIP;
  void *p = g_scratch[dev].load(std::memory_order_acquire);
  if (!p) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch[dev].load(std::memory_order_relaxed);
    if (!p) {
      int cur = -1;
      if (hipGetDevice(&cur) != hipSuccess) return FP8L_EHIP;
      if (cur != dev && hipSetDevice(dev) != hipSuccess) return FP8L_EHIP;
      const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (cur != dev && hipSetDevice(cur) != hipSuccess) return FP8L_EHIP;
      if (e != hipSuccess || !p) return FP8L_EHIP;
      g_scratch[dev].store(p, std::memory_order_release);
    }
  }
  *out = p;
  return FP8L_OK;
}

// Argument checks shared by the quantize entry points (everything but the
// workspace); FP8L_OK if the call is valid.
int check_quantize_args(const void *x, int64_t rows, int64_t cols, int scaling, const void *q,
                        const void *qt, const float *scale, const float *scale_t,
                        const float *amax_out) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(rows) || bad_dim(cols) || rows * cols > kMaxElems) return FP8L_ESHAPE;
  if (!fp8l::quantize_fits(rows, cols, scaling)) return FP8L_ESHAPE;
  const bool empty = rows == 0 || cols == 0;
  // scale vectors may be NULL only where they have no entries (rowwise, 0 rows
  // or 0 columns); tensorwise scales always have one entry
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  if ((!scale && (!rw || rows > 0)) || (!scale_t && (!rw || cols > 0))) return FP8L_EINVAL;
  if (!empty && (!x || !q || !qt)) return FP8L_EINVAL;
  if (misaligned(x) || misaligned(q) || misaligned(qt)) return FP8L_EALIGN;
  if ((reinterpret_cast<uintptr_t>(scale) & 3u) || (reinterpret_cast<uintptr_t>(scale_t) & 3u) ||
      (reinterpret_cast<uintptr_t>(amax_out) & 3u))
    return FP8L_EALIGN;
  return FP8L_OK;
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Checks shared by the norm entry points.
int check_norm(int64_t rows, int64_t cols, int kind, int dtype, int pdtype) {
  if ((kind != FP8L_LAYERNORM && kind != FP8L_RMSNORM) ||
      (dtype != FP8L_BF16 && dtype != FP8L_F32) || (pdtype != FP8L_BF16 && pdtype != FP8L_F32))
    return FP8L_EINVAL;
  if (rows < 0 || rows > (int64_t)1 << 30 || cols < 1 || cols > FP8L_NORM_MAX_COLS)
    return FP8L_ESHAPE;
  return FP8L_OK;
}

// A buffer of a call (none where p is NULL).
struct Span {
  const void *p;
  int64_t bytes;
};

// Whether one of the outputs spans[0..outs) meets another of the n spans.  (A
// workspace counts as an output, with the bytes that the call asks for.)
template <int N>
bool overlapping(const Span (&spans)[N], int outs) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < N; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(spans[i].p);
      const uintptr_t b = reinterpret_cast<uintptr_t>(spans[j].p);
      if (a && b && spans[i].bytes > 0 && spans[j].bytes > 0 &&
          a < b + (uintptr_t)spans[j].bytes && b < a + (uintptr_t)spans[i].bytes)
        return true;
    }
  return false;
}

bool bad_act(int act, int pdtype) {
  return act < FP8L_ACT_NONE || act > FP8L_ACT_RELU2 || (pdtype != FP8L_BF16 && pdtype != FP8L_F32);
}

bool bad_finite(float v) { return !(v >= -3.402823466e38f && v <= 3.402823466e38f); }

// Checks of a residual norm's descriptor shared by its entry points, and the
// launchers' form of it.
int check_resnorm(const fp8l_resnorm *r, fp8l::ResIn &in) {
  if (!r) return FP8L_EINVAL;
  const int s = check_norm(r->rows, r->cols, r->kind, r->dtype, r->pdtype);
  if (s != FP8L_OK) return s;
  if ((r->norms & ~(FP8L_POST_NORM | FP8L_PRE_NORM)) || r->norms == 0) return FP8L_EINVAL;
  if (bad_finite(r->alpha) || (r->rows > 0 && (!r->b || !r->s))) return FP8L_EINVAL;
  const bool post = (r->norms & FP8L_POST_NORM) != 0, pre = (r->norms & FP8L_PRE_NORM) != 0;
  const bool rms = r->kind == FP8L_RMSNORM;
  in = {r->b, r->x, post ? r->post_w : nullptr, post ? r->post_b : nullptr,
        pre ? r->pre_w : nullptr, pre ? r->pre_b : nullptr, r->gate, r->pdtype == FP8L_F32,
        r->dtype == FP8L_F32, rms, post, pre, r->alpha, r->eps, r->rows, r->cols, r->s,
        pre ? r->y : nullptr, post && !rms ? r->mean_post : nullptr,
        post ? r->rstd_post : nullptr, pre && !rms ? r->mean_pre : nullptr,
        pre ? r->rstd_pre : nullptr};
  for (const void *p : {in.b, in.x, in.post_w, in.post_b, in.pre_w, in.pre_b, in.gate,
                        (const void *)in.s, (const void *)in.y})
    if (misaligned(p)) return FP8L_EALIGN;
  for (const float *f : {in.mean_post, in.rstd_post, in.mean_pre, in.rstd_pre})
    if (misaligned4(f)) return FP8L_EALIGN;
  return FP8L_OK;
}

bool bad_eps(float eps) { return !(eps >= 0.f && eps <= 3.402823466e38f); }

}  // namespace

extern "C" {

size_t fp8_linear_workspace_bytes(int64_t rows, int64_t cols, int scaling) {
  if (bad_dim(rows) || bad_dim(cols)) return 0;
  if (bad_scaling(scaling)) return 0;
  return fp8l::quantize_workspace_bytes(rows, cols, scaling);
}

int fp8_linear_quantize(const void *x, int64_t rows, int64_t cols, int scaling,
                        void *q, void *qt, float *scale, float *scale_t,
                        float *amax_out, void *workspace, size_t workspace_bytes,
                        void *stream) {
  const int s = check_quantize_args(x, rows, cols, scaling, q, qt, scale, scale_t, amax_out);
  if (s != FP8L_OK) return s;
  const size_t need = fp8l::quantize_workspace_bytes(rows, cols, scaling);
  if (need > 0 && !workspace) return FP8L_EINVAL;
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(workspace)) return FP8L_EALIGN;
  hipError_t e = fp8l::quantize_launch(x, rows, cols, scaling, q, qt, scale, scale_t,
                                       amax_out, workspace,
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_quantize_noalloc(const void *x, int64_t rows, int64_t cols, int scaling,
                                void *q, void *qt, float *scale, float *scale_t,
                                float *amax_out, void *stream) {
  const int s = check_quantize_args(x, rows, cols, scaling, q, qt, scale, scale_t, amax_out);
  if (s != FP8L_OK) return s;
  // checked before any HIP call: an oversized request fails on the host
  if (fp8l::quantize_workspace_bytes(rows, cols, scaling) > FP8L_NOALLOC_MAX_WORKSPACE)
    return FP8L_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  void *ws = nullptr;
  const int sa = scratch_address(st, &ws);
  if (sa != FP8L_OK) return sa;
  // every partial maximum the cast reads is written by this call's amax
  // pass first, so the array needs no clearing between calls
  hipError_t e = fp8l::quantize_launch(x, rows, cols, scaling, q, qt, scale, scale_t, amax_out,
                                       ws, st);
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_fwd(const void *xq, const float *sx, const void *wq,
                   const float *sw, int64_t M, int64_t N, int64_t K,
                   int scaling, void *out, void *stream) {
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, N, K)) return FP8L_ESHAPE;
  int s = check_gemm_operands(xq, sx, wq, sw, out, M, N, K);
  if (s != FP8L_OK) return s;
  const int vec = scaling == FP8L_ROWWISE;
  hipError_t e = fp8l::gemm_launch(static_cast<const uint8_t *>(xq), sx,
                                   static_cast<const uint8_t *>(wq), sw, vec, 0, M, N, K,
                                   static_cast<uint16_t *>(out),
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_bwd(const void *dyq, const float *sdy, const void *dytq,
                   const float *sdyt, const void *wtq, const float *swt,
                   const void *xtq, const float *sxt, int64_t M, int64_t N,
                   int64_t K, int scaling, void *grad_x, void *grad_w,
                   void *stream) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8L_ESHAPE;
  // grad_x: [M,K] from [M,N] x [K,N]; grad_w: [N,K] from [N,M] x [K,M]
  if (bad_gemm_sizes(M, K, N) || bad_gemm_sizes(N, K, M)) return FP8L_ESHAPE;
  if (!grad_x && !grad_w) return FP8L_EINVAL;
  int s;
  if (grad_x && (s = check_gemm_operands(dyq, sdy, wtq, swt, grad_x, M, K, N)) != FP8L_OK)
    return s;
  if (grad_w && (s = check_gemm_operands(dytq, sdyt, xtq, sxt, grad_w, N, K, M)) != FP8L_OK)
    return s;
  const int vec = (scaling & FP8L_ROWWISE) != 0;
  const int fa = (scaling & FP8L_E5M2) != 0;     // dY operands in E5M2
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (grad_x)  // [M,K] = dYq[M,N] . WTq[K,N]^T
    e = fp8l::gemm_launch(static_cast<const uint8_t *>(dyq), sdy,
                          static_cast<const uint8_t *>(wtq), swt, vec, fa, M, K, N,
                          static_cast<uint16_t *>(grad_x), st);
  if (e == hipSuccess && grad_w)  // [N,K] = dYTq[N,M] . XTq[K,M]^T
    e = fp8l::gemm_launch(static_cast<const uint8_t *>(dytq), sdyt,
                          static_cast<const uint8_t *>(xtq), sxt, vec, fa, N, K, M,
                          static_cast<uint16_t *>(grad_w), st);
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_amax(const void *x, int64_t rows, int64_t cols, float *amax_out,
                    void *workspace, size_t workspace_bytes, void *stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols > kMaxElems) return FP8L_ESHAPE;
  if (!amax_out || (rows * cols > 0 && !x)) return FP8L_EINVAL;
  const size_t need = fp8l::quantize_workspace_bytes(rows, cols, FP8L_TENSORWISE);
  if (need > 0 && !workspace) return FP8L_EINVAL;
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(x) || misaligned(workspace) || (reinterpret_cast<uintptr_t>(amax_out) & 3u))
    return FP8L_EALIGN;
  hipError_t e = fp8l::amax_launch(x, rows, cols, amax_out, workspace,
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_quantize_scaled(const void *x, int64_t rows, int64_t cols, const float *scale,
                               void *q, void *qt, void *stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols > kMaxElems) return FP8L_ESHAPE;
  if (rows * cols == 0) return FP8L_OK;
  if (!fp8l::quantize_fits(rows, cols, FP8L_TENSORWISE)) return FP8L_ESHAPE;
  if (!x || !scale || !q || !qt) return FP8L_EINVAL;
  if (misaligned(x) || misaligned(q) || misaligned(qt) ||
      (reinterpret_cast<uintptr_t>(scale) & 3u))
    return FP8L_EALIGN;
  hipError_t e = fp8l::quantize_scaled_launch(x, rows, cols, scale, q, qt,
                                              static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_bwd_w_f32(const void *dytq, const float *sdyt, const void *xtq,
                         const float *sxt, int64_t M, int64_t N, int64_t K, int scaling,
                         float *grad_w, void *stream) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8L_ESHAPE;
  // [N,K] fp32 = dYTq[N,M] . XTq[K,M]^T: 4-byte outputs under the same
  // 32-bit offset limit
  if (bad_gemm_sizes(N, K, M) || 4 * N * K > kMaxGemmBytes) return FP8L_ESHAPE;
  int s = check_gemm_operands(dytq, sdyt, xtq, sxt, grad_w, N, K, M);
  if (s != FP8L_OK) return s;
  hipError_t e = fp8l::gemm_f32_launch(static_cast<const uint8_t *>(dytq), sdyt,
                                       static_cast<const uint8_t *>(xtq), sxt,
                                       (scaling & FP8L_ROWWISE) != 0,
                                       (scaling & FP8L_E5M2) != 0, N, K, M, grad_w,
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_gemm_grouped(const fp8l_gemm_problem *problems, int count, int scaling,
                            void *stream) {
  if (!problems || count < 1 || count > FP8L_MAX_GROUP) return FP8L_EINVAL;
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  fp8l::GemmDesc d[FP8L_MAX_GROUP];
  for (int i = 0; i < count; ++i) {
    const fp8l_gemm_problem &p = problems[i];
    if (bad_dim(p.m) || bad_dim(p.n) || bad_dim(p.k)) return FP8L_ESHAPE;
    if (bad_gemm_sizes(p.m, p.n, p.k)) return FP8L_ESHAPE;
    int s = check_gemm_operands(p.a, p.sa, p.b, p.sb, p.c, p.m, p.n, p.k);
    if (s != FP8L_OK) return s;
    d[i] = {static_cast<const uint8_t *>(p.a), p.sa, static_cast<const uint8_t *>(p.b), p.sb,
            p.c, p.m, p.n, p.k};
  }
  // outputs pairwise disjoint
  for (int i = 0; i < count; ++i)
    for (int j = i + 1; j < count; ++j) {
      const uintptr_t a0 = reinterpret_cast<uintptr_t>(problems[i].c);
      const uintptr_t a1 = a0 + (uintptr_t)(2 * problems[i].m * problems[i].n);
      const uintptr_t b0 = reinterpret_cast<uintptr_t>(problems[j].c);
      const uintptr_t b1 = b0 + (uintptr_t)(2 * problems[j].m * problems[j].n);
      if (a0 < b1 && b0 < a1) return FP8L_EINVAL;
    }
  hipError_t e = fp8l::gemm_group_launch(d, count, (scaling & FP8L_ROWWISE) != 0,
                                         (scaling & FP8L_E5M2) != 0,
                                         static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_bwd_x_acc(const void *dyq, const float *sdy, const void *wtq, const float *swt,
                         int64_t M, int64_t N, int64_t K, int scaling, void *grad_x,
                         void *stream) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, K, N)) return FP8L_ESHAPE;
  int s = check_gemm_operands(dyq, sdy, wtq, swt, grad_x, M, K, N);
  if (s != FP8L_OK) return s;
  hipError_t e = fp8l::gemm_acc_launch(static_cast<const uint8_t *>(dyq), sdy,
                                       static_cast<const uint8_t *>(wtq), swt,
                                       (scaling & FP8L_ROWWISE) != 0,
                                       (scaling & FP8L_E5M2) != 0, M, K, N,
                                       static_cast<uint16_t *>(grad_x),
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

size_t fp8_swiglu_workspace_bytes(int64_t rows, int64_t hidden, int scaling) {
  if (bad_dim(rows) || bad_dim(hidden) || bad_scaling(scaling)) return 0;
  return fp8l::swiglu_workspace_bytes(rows, hidden, scaling);
}

int fp8_swiglu_fwd(const void *a, const void *b, int64_t rows, int64_t hidden, int scaling,
                   void *h, void *hq, void *hqt, float *scale, float *scale_t, float *amax_out,
                   void *workspace, size_t workspace_bytes, void *stream) {
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (bad_dim(rows) || bad_dim(hidden) || rows * hidden > kMaxElems) return FP8L_ESHAPE;
  if (!fp8l::quantize_fits(rows, hidden, scaling)) return FP8L_ESHAPE;
  const bool rw = scaling == FP8L_ROWWISE;
  if ((!scale && (!rw || rows > 0)) || (!scale_t && (!rw || hidden > 0))) return FP8L_EINVAL;
  if (rows * hidden > 0 && (!a || !b || !h || !hq || !hqt)) return FP8L_EINVAL;
  const size_t need = fp8l::swiglu_workspace_bytes(rows, hidden, scaling);
  if (!workspace) return FP8L_EINVAL;
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(a) || misaligned(b) || misaligned(h) || misaligned(hq) || misaligned(hqt) ||
      misaligned(workspace))
    return FP8L_EALIGN;
  if ((reinterpret_cast<uintptr_t>(scale) & 3u) || (reinterpret_cast<uintptr_t>(scale_t) & 3u) ||
      (reinterpret_cast<uintptr_t>(amax_out) & 3u))
    return FP8L_EALIGN;
  hipError_t e = fp8l::swiglu_fwd_launch(a, b, rows, hidden, scaling, h, hq, hqt, scale,
                                         scale_t, amax_out, workspace,
                                         static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_swiglu_bwd(const void *dh, const void *a, const void *b, int64_t rows, int64_t hidden,
                   int scaling, void *da, void *db, void *daq, void *daqt, float *da_scale,
                   float *da_scale_t, float *da_amax, void *dbq, void *dbqt, float *db_scale,
                   float *db_scale_t, float *db_amax, void *workspace, size_t workspace_bytes,
                   void *stream) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(rows) || bad_dim(hidden) || rows * hidden > kMaxElems) return FP8L_ESHAPE;
  if (!fp8l::quantize_fits(rows, hidden, scaling)) return FP8L_ESHAPE;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  if ((!da_scale || !db_scale) && (!rw || rows > 0)) return FP8L_EINVAL;
  if ((!da_scale_t || !db_scale_t) && (!rw || hidden > 0)) return FP8L_EINVAL;
  if (rows * hidden > 0 &&
      (!dh || !a || !b || !da || !db || !daq || !daqt || !dbq || !dbqt))
    return FP8L_EINVAL;
  const size_t need = fp8l::swiglu_workspace_bytes(rows, hidden, scaling);
  if (!workspace) return FP8L_EINVAL;
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(dh) || misaligned(a) || misaligned(b) || misaligned(da) || misaligned(db) ||
      misaligned(daq) || misaligned(daqt) || misaligned(dbq) || misaligned(dbqt) ||
      misaligned(workspace))
    return FP8L_EALIGN;
  for (const float *f : {da_scale, da_scale_t, da_amax, db_scale, db_scale_t, db_amax})
    if (reinterpret_cast<uintptr_t>(f) & 3u) return FP8L_EALIGN;
  const fp8l::Fp8Out qa = {daq, daqt, da_scale, da_scale_t, da_amax};
  const fp8l::Fp8Out qb = {dbq, dbqt, db_scale, db_scale_t, db_amax};
  hipError_t e = fp8l::swiglu_bwd_launch(dh, a, b, rows, hidden, scaling, da, db, qa, qb,
                                         workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

size_t fp8_gated_workspace_bytes(int64_t M, int64_t H, int scaling) {
  if (M < 0 || M > (int64_t)1 << 30 || bad_dim(H) || bad_scaling(scaling)) return 0;
  return fp8l::gated_workspace_bytes(M, H, scaling);
}

int fp8_gated_fwd(const void *xq, const float *sx, const void *w1q, const float *sw1,
                  const void *w3q, const float *sw3, int64_t M, int64_t H, int64_t K, int scaling,
                  void *a, void *b, void *h, void *hq, void *hqt, float *scale, float *scale_t,
                  float *amax_out, void *workspace, size_t workspace_bytes, void *stream) {
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (M < 0 || M > (int64_t)1 << 30 || bad_dim(H) || bad_dim(K)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, H, K)) return FP8L_ESHAPE;
  const bool quant = hq || hqt || scale || scale_t || amax_out;
  if (quant && M % 16 != 0) return FP8L_ESHAPE;
  int s = check_gemm_operands(xq, sx, w1q, sw1, h, M, H, K);
  if (s == FP8L_OK) s = check_gemm_operands(xq, sx, w3q, sw3, h, M, H, K);
  if (s != FP8L_OK) return s;
  if (M * H > 0 && !a != !b) return FP8L_EINVAL;
  if (misaligned(a) || misaligned(b)) return FP8L_EALIGN;
  size_t need = 0;
  if (quant) {
    s = check_quantize_args(h, M, H, scaling, hq, hqt, scale, scale_t, amax_out);
    if (s != FP8L_OK) return s;
    if (!workspace) return FP8L_EINVAL;
    need = fp8l::gated_workspace_bytes(M, H, scaling);
    if (workspace_bytes < need) return FP8L_EWORKSPACE;
    if (misaligned(workspace)) return FP8L_EALIGN;
  }
  const int64_t mh = M * H;
  const bool rw = scaling == FP8L_ROWWISE;
  const int64_t sm = rw ? 4 * M : 4, sh = rw ? 4 * H : 4;   // bytes of the scale vectors
  const Span spans[] = {{a, 2 * mh}, {b, 2 * mh}, {h, 2 * mh}, {hq, mh}, {hqt, mh}, {scale, sm},
                        {scale_t, sh}, {amax_out, rw ? sm + sh : 4}, {workspace, (int64_t)need},
                        {xq, M * K}, {w1q, H * K}, {w3q, H * K}, {sx, sm}, {sw1, sh}, {sw3, sh}};
  if (overlapping(spans, 9)) return FP8L_EINVAL;
  const fp8l::Fp8Out o = {hq, hqt, scale, scale_t, amax_out};
  hipError_t e = fp8l::gated_fwd_launch(
      static_cast<const uint8_t *>(xq), sx, static_cast<const uint8_t *>(w1q), sw1,
      static_cast<const uint8_t *>(w3q), sw3, M, H, K, scaling, static_cast<uint16_t *>(a),
      static_cast<uint16_t *>(b), static_cast<uint16_t *>(h), quant ? &o : nullptr, workspace,
      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_gated_bwd(const void *dyq, const float *sdy, const void *w2tq, const float *sw2t,
                  const void *a, const void *b, int64_t M, int64_t H, int64_t D, int scaling,
                  void *da, void *db, void *daq, void *daqt, float *da_scale, float *da_scale_t,
                  float *da_amax, void *dbq, void *dbqt, float *db_scale, float *db_scale_t,
                  float *db_amax, void *workspace, size_t workspace_bytes, void *stream) {
  if (bad_scaling(scaling)) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(H) || bad_dim(D)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, H, D)) return FP8L_ESHAPE;
  int s = check_gemm_operands(dyq, sdy, w2tq, sw2t, da, M, H, D);
  if (s == FP8L_OK)
    s = check_quantize_args(da, M, H, scaling, daq, daqt, da_scale, da_scale_t, da_amax);
  if (s == FP8L_OK)
    s = check_quantize_args(db, M, H, scaling, dbq, dbqt, db_scale, db_scale_t, db_amax);
  if (s != FP8L_OK) return s;
  if (M * H > 0 && (!a || !b)) return FP8L_EINVAL;
  if (!workspace) return FP8L_EINVAL;
  const size_t need = fp8l::gated_workspace_bytes(M, H, scaling);
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(a) || misaligned(b) || misaligned(workspace)) return FP8L_EALIGN;
  const int64_t mh = M * H;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  const int64_t sm = rw ? 4 * M : 4, sh = rw ? 4 * H : 4, am = rw ? sm + sh : 4;
  const Span spans[] = {{da, 2 * mh}, {db, 2 * mh}, {daq, mh}, {daqt, mh}, {dbq, mh}, {dbqt, mh},
                        {da_scale, sm}, {da_scale_t, sh}, {da_amax, am}, {db_scale, sm},
                        {db_scale_t, sh}, {db_amax, am}, {workspace, (int64_t)need},
                        {a, 2 * mh}, {b, 2 * mh}, {dyq, M * D}, {w2tq, H * D}, {sdy, sm},
                        {sw2t, sh}};
  if (overlapping(spans, 13)) return FP8L_EINVAL;
  const fp8l::Fp8Out qa = {daq, daqt, da_scale, da_scale_t, da_amax};
  const fp8l::Fp8Out qb = {dbq, dbqt, db_scale, db_scale_t, db_amax};
  hipError_t e = fp8l::gated_bwd_launch(
      static_cast<const uint8_t *>(dyq), sdy, static_cast<const uint8_t *>(w2tq), sw2t,
      static_cast<const uint16_t *>(a), static_cast<const uint16_t *>(b), M, H, D, scaling,
      static_cast<uint16_t *>(da), static_cast<uint16_t *>(db), qa, qb, workspace,
      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

size_t fp8_linear_act_workspace_bytes(int64_t M, int64_t N, int scaling) {
  if (M < 0 || M > (int64_t)1 << 30 || bad_dim(N) || bad_scaling(scaling)) return 0;
  return fp8l::linear_act_workspace_bytes(M, N, scaling);
}

int fp8_linear_act_fwd(const void *xq, const float *sx, const void *wq, const float *sw,
                       int64_t M, int64_t N, int64_t K, int scaling, const void *bias, int pdtype,
                       int act, const void *residual, void *z, void *y, void *q, void *qt,
                       float *scale, float *scale_t, float *amax_out, void *workspace,
                       size_t workspace_bytes, void *stream) {
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (bad_act(act, pdtype)) return FP8L_EINVAL;
  if (M < 0 || M > (int64_t)1 << 30 || bad_dim(N) || bad_dim(K)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, N, K)) return FP8L_ESHAPE;
  const bool rw = scaling == FP8L_ROWWISE;
  const bool quant = q || qt || scale || scale_t || amax_out;
  const bool rows_only = quant && rw && !qt && !scale_t;
  if (quant && !rows_only && M % 16 != 0) return FP8L_ESHAPE;
  // y may be left out where z and its codes are written
  if (M * N > 0 && !y && (!z || !quant || residual)) return FP8L_EINVAL;
  int s = check_gemm_operands(xq, sx, wq, sw, y ? y : z, M, N, K);
  if (s != FP8L_OK) return s;
  if (misaligned(bias) || misaligned(residual) || misaligned(z)) return FP8L_EALIGN;
  if (quant) {
    if (rows_only) {
      if (M * N > 0 && !q) return FP8L_EINVAL;
      if (M > 0 && !scale) return FP8L_EINVAL;
      if (misaligned(q)) return FP8L_EALIGN;
      if (misaligned4(scale) || misaligned4(amax_out)) return FP8L_EALIGN;
    } else {
      s = check_quantize_args(y ? y : z, M, N, scaling, q, qt, scale, scale_t, amax_out);
      if (s != FP8L_OK) return s;
    }
  }
  if (!workspace) return FP8L_EINVAL;
  const size_t need = fp8l::linear_act_workspace_bytes(M, N, scaling);
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(workspace)) return FP8L_EALIGN;
  const int64_t mn = M * N;
  const int64_t sm = rw ? 4 * M : 4, sn = rw ? 4 * N : 4, st = rows_only ? 0 : sn;
  const Span spans[] = {{z, 2 * mn}, {y, 2 * mn}, {q, mn}, {qt, mn}, {scale, sm}, {scale_t, st},
                        {amax_out, rw ? sm + st : 4}, {workspace, (int64_t)need}, {xq, M * K},
                        {wq, N * K}, {sx, sm}, {sw, sn},
                        {bias, N * (pdtype == FP8L_F32 ? 4 : 2)},
                        {residual == y ? nullptr : residual, 2 * mn}};
  if (overlapping(spans, 8)) return FP8L_EINVAL;
  const fp8l::LinearActIn in = {static_cast<const uint8_t *>(xq), static_cast<const uint8_t *>(wq),
                                sx, sw, M, N, K, bias, pdtype == FP8L_F32, act,
                                static_cast<const uint16_t *>(residual),
                                static_cast<uint16_t *>(z), static_cast<uint16_t *>(y)};
  const fp8l::Fp8Out o = {q, qt, scale, scale_t, amax_out};
  const hipError_t e = fp8l::linear_act_fwd_launch(in, scaling, quant ? &o : nullptr, workspace,
                                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_act_bwd(const void *dyq, const float *sdy, const void *wtq, const float *swt,
                       const void *z, int64_t M, int64_t H, int64_t D, int scaling, int act,
                       void *dz, void *q, void *qt, float *scale, float *scale_t, float *amax_out,
                       void *dbias, int pdtype, void *workspace, size_t workspace_bytes,
                       void *stream) {
  if (bad_scaling(scaling) || bad_act(act, pdtype)) return FP8L_EINVAL;
  if (bad_dim(M) || bad_dim(H) || bad_dim(D)) return FP8L_ESHAPE;
  if (bad_gemm_sizes(M, H, D)) return FP8L_ESHAPE;
  int s = check_gemm_operands(dyq, sdy, wtq, swt, dz, M, H, D);
  if (s == FP8L_OK) s = check_quantize_args(dz, M, H, scaling, q, qt, scale, scale_t, amax_out);
  if (s != FP8L_OK) return s;
  if (act == FP8L_ACT_NONE) z = nullptr;
  else if (M * H > 0 && !z) return FP8L_EINVAL;
  if (misaligned(z) || misaligned(dbias)) return FP8L_EALIGN;
  if (!workspace) return FP8L_EINVAL;
  const size_t need = fp8l::linear_act_workspace_bytes(M, H, scaling);
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(workspace)) return FP8L_EALIGN;
  const int64_t mh = M * H;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  const int64_t sm = rw ? 4 * M : 4, sh = rw ? 4 * H : 4;
  const Span spans[] = {{dz, 2 * mh}, {q, mh}, {qt, mh}, {scale, sm}, {scale_t, sh},
                        {amax_out, rw ? sm + sh : 4}, {dbias, H * (pdtype == FP8L_F32 ? 4 : 2)},
                        {workspace, (int64_t)need}, {dyq, M * D}, {wtq, H * D}, {sdy, sm},
                        {swt, sh}, {z, 2 * mh}};
  if (overlapping(spans, 8)) return FP8L_EINVAL;
  const hipError_t e = fp8l::linear_act_bwd_launch(
      static_cast<const uint8_t *>(dyq), sdy, static_cast<const uint8_t *>(wtq), swt,
      static_cast<const uint16_t *>(z), act, M, H, D, scaling, static_cast<uint16_t *>(dz), dbias,
      pdtype == FP8L_F32, {q, qt, scale, scale_t, amax_out}, workspace,
      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_bias_act_bwd(const void *dy, const void *z, int64_t M, int64_t N, int scaling, int act,
                     void *dz, void *q, void *qt, float *scale, float *scale_t, float *amax_out,
                     void *dbias, int pdtype, void *workspace, size_t workspace_bytes,
                     void *stream) {
  if (bad_scaling(scaling) || bad_act(act, pdtype)) return FP8L_EINVAL;
  int s = check_quantize_args(dy, M, N, scaling, q, qt, scale, scale_t, amax_out);
  if (s != FP8L_OK) return s;
  if (dbias && !fp8l::quantize_fits(M, N, scaling, (N + 63) / 64)) return FP8L_ESHAPE;
  if (act == FP8L_ACT_NONE) z = nullptr;
  else if (M * N > 0 && (!z || !dz)) return FP8L_EINVAL;
  if (misaligned(z) || misaligned(dz) || misaligned(dbias)) return FP8L_EALIGN;
  if (!workspace) return FP8L_EINVAL;
  const size_t need = fp8l::linear_act_workspace_bytes(M, N, scaling);
  if (workspace_bytes < need) return FP8L_EWORKSPACE;
  if (misaligned(workspace)) return FP8L_EALIGN;
  const int64_t mn = M * N;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  const int64_t sm = rw ? 4 * M : 4, sn = rw ? 4 * N : 4;
  const Span spans[] = {{dz, 2 * mn}, {q, mn}, {qt, mn}, {scale, sm}, {scale_t, sn},
                        {amax_out, rw ? sm + sn : 4}, {dbias, N * (pdtype == FP8L_F32 ? 4 : 2)},
                        {workspace, (int64_t)need}, {dy, 2 * mn}, {z, 2 * mn}};
  if (overlapping(spans, 8)) return FP8L_EINVAL;
  const size_t maxima = fp8l::linear_act_maxima_bytes(M, N, scaling);
  const hipError_t e = fp8l::bias_act_bwd_launch(
      dy, z, act, M, N, scaling, dz, dbias, pdtype == FP8L_F32, {q, qt, scale, scale_t, amax_out},
      workspace, reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + maxima),
      static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

size_t fp8_layernorm_workspace_bytes(int64_t rows, int64_t cols, int scaling) {
  if (check_norm(rows, cols, 0, 0, 0) != FP8L_OK || bad_scaling(scaling)) return 0;
  return fp8l::norm_workspace_bytes(rows, cols, scaling);
}

int fp8_layernorm_fwd(const void *x, int64_t rows, int64_t cols, int kind, int dtype,
                      const void *weight, const void *bias, int pdtype, float eps, void *y,
                      float *mean, float *rstd, void *stream) {
  const int s = check_norm(rows, cols, kind, dtype, pdtype);
  if (s != FP8L_OK) return s;
  if (bad_eps(eps) || (rows > 0 && (!x || !y))) return FP8L_EINVAL;
  if (misaligned(x) || misaligned(weight) || misaligned(bias) || misaligned(y) ||
      misaligned4(mean) || misaligned4(rstd))
    return FP8L_EALIGN;
  const int64_t bytes = rows * cols * (dtype == FP8L_F32 ? 4 : 2);
  const int64_t pb = cols * (pdtype == FP8L_F32 ? 4 : 2);
  const Span spans[] = {{y, bytes}, {mean, 4 * rows}, {rstd, 4 * rows}, {x, bytes}, {weight, pb},
                        {bias, pb}};
  if (overlapping(spans, 3)) return FP8L_EINVAL;
  const fp8l::NormIn in = {x, weight, bias, pdtype == FP8L_F32, kind == FP8L_RMSNORM, eps,
                           rows, cols};
  hipError_t e = fp8l::norm_fwd_launch(in, dtype == FP8L_F32, y, mean, rstd,
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_layernorm_quantize(const void *x, int64_t rows, int64_t cols, int kind,
                           const void *weight, const void *bias, int pdtype, float eps,
                           int scaling, void *y, float *mean, float *rstd, void *q, void *qt,
                           float *scale, float *scale_t, float *amax_out, void *workspace,
                           size_t workspace_bytes, void *stream) {
  const int s = check_norm(rows, cols, kind, FP8L_BF16, pdtype);
  if (s != FP8L_OK) return s;
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (bad_eps(eps)) return FP8L_EINVAL;
  const bool rw = scaling == FP8L_ROWWISE;
  const bool rows_only = rw && !qt && rows > 0;
  if (cols % 16 != 0 || (!rows_only && rows % 16 != 0)) return FP8L_ESHAPE;
  if (!rows_only && !fp8l::quantize_fits(rows, cols, scaling)) return FP8L_ESHAPE;
  if (rows > 0 && (!x || !q || (!qt && !rows_only))) return FP8L_EINVAL;
  // scale vectors may be NULL only where they have no entries
  if (!scale && (!rw || rows > 0)) return FP8L_EINVAL;
  if (!scale_t && qt) return FP8L_EINVAL;
  if (!scale_t && !rw) return FP8L_EINVAL;
  if (!rows_only && rows > 0 && !y && (!rstd || (kind == FP8L_LAYERNORM && !mean)))
    return FP8L_EINVAL;
  if (misaligned(x) || misaligned(weight) || misaligned(bias) || misaligned(y) ||
      misaligned(q) || misaligned(qt))
    return FP8L_EALIGN;
  for (const float *f : {(const float *)mean, (const float *)rstd, (const float *)scale,
                         (const float *)scale_t, (const float *)amax_out})
    if (misaligned4(f)) return FP8L_EALIGN;
  const fp8l::NormIn in = {x, weight, bias, pdtype == FP8L_F32, kind == FP8L_RMSNORM, eps,
                           rows, cols};
  hipStream_t st = static_cast<hipStream_t>(stream);
  size_t need = 0;
  if (!rows_only) {
    if (rw && !scale_t) return FP8L_OK;          // no rows, no column scales wanted
    if (!workspace) return FP8L_EINVAL;
    need = fp8l::norm_workspace_bytes(rows, cols, scaling);
    if (workspace_bytes < need) return FP8L_EWORKSPACE;
    if (misaligned(workspace)) return FP8L_EALIGN;
  }
  const int64_t n = rows * cols, pb = cols * (pdtype == FP8L_F32 ? 4 : 2);
  const int64_t sr = rw ? 4 * rows : 4, sc = rows_only ? 0 : rw ? 4 * cols : 4;
  const Span spans[] = {{y, 2 * n}, {q, n}, {qt, n}, {mean, 4 * rows}, {rstd, 4 * rows},
                        {scale, sr}, {scale_t, sc}, {amax_out, rw ? sr + sc : 4},
                        {workspace, (int64_t)need}, {x, 2 * n}, {weight, pb}, {bias, pb}};
  if (overlapping(spans, 9)) return FP8L_EINVAL;
  hipError_t e;
  if (rows_only) {
    e = fp8l::norm_rows_launch(in, y, mean, rstd, q, scale, amax_out, st);
  } else {
    e = fp8l::norm_quantize_launch(in, scaling, y, mean, rstd,
                                   {q, qt, scale, scale_t, amax_out}, workspace, st);
  }
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_layernorm_bwd(const void *dy, const void *x, const void *weight, const float *mean,
                      const float *rstd, int64_t rows, int64_t cols, int kind, int dtype,
                      int pdtype, void *dx, float *dweight, float *dbias, void *workspace,
                      size_t workspace_bytes, void *stream) {
  const int s = check_norm(rows, cols, kind, dtype, pdtype);
  if (s != FP8L_OK) return s;
  if (!dx && !dweight && !dbias) return FP8L_EINVAL;
  if (rows > 0 && (!dy || !x || !rstd || (kind == FP8L_LAYERNORM && !mean))) return FP8L_EINVAL;
  if (misaligned(dy) || misaligned(x) || misaligned(weight) || misaligned(dx))
    return FP8L_EALIGN;
  for (const float *f : {mean, rstd, (const float *)dweight, (const float *)dbias})
    if (misaligned4(f)) return FP8L_EALIGN;
  size_t need = 0;
  if (dweight || dbias) {
    if (!workspace) return FP8L_EINVAL;
    need = fp8l::norm_workspace_bytes(rows, cols, FP8L_TENSORWISE);
    if (workspace_bytes < need) return FP8L_EWORKSPACE;
    if (misaligned(workspace)) return FP8L_EALIGN;
  }
  const int64_t bytes = rows * cols * (dtype == FP8L_F32 ? 4 : 2);
  const Span spans[] = {{dx, bytes}, {dweight, 4 * cols}, {dbias, 4 * cols},
                        {workspace, (int64_t)need}, {dy, bytes}, {x, bytes},
                        {weight, cols * (pdtype == FP8L_F32 ? 4 : 2)}, {mean, 4 * rows},
                        {rstd, 4 * rows}};
  if (overlapping(spans, 4)) return FP8L_EINVAL;
  const fp8l::NormIn in = {x, weight, nullptr, pdtype == FP8L_F32, kind == FP8L_RMSNORM, 0.f,
                           rows, cols};
  hipError_t e = fp8l::norm_bwd_launch(dy, in, dtype == FP8L_F32, mean, rstd, dx, dweight, dbias,
                                       workspace, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

size_t fp8_resnorm_workspace_bytes(int64_t rows, int64_t cols, int scaling) {
  if (check_norm(rows, cols, 0, 0, 0) != FP8L_OK || bad_scaling(scaling)) return 0;
  return fp8l::resnorm_workspace_bytes(rows, cols, scaling);
}

int fp8_resnorm_fwd(const fp8l_resnorm *r, void *stream) {
  fp8l::ResIn in;
  const int s = check_resnorm(r, in);
  if (s != FP8L_OK) return s;
  if (bad_eps(r->eps) || (in.rows > 0 && (!in.x || (in.pre && !in.y)))) return FP8L_EINVAL;
  const int64_t n = in.rows * in.cols, e = in.f32 ? 4 : 2, pb = in.cols * (in.wf32 ? 4 : 2);
  const Span spans[] = {{in.s, e * n}, {in.y, 2 * n}, {in.mean_post, 4 * in.rows},
                        {in.rstd_post, 4 * in.rows}, {in.mean_pre, 4 * in.rows},
                        {in.rstd_pre, 4 * in.rows}, {in.b, 2 * n}, {in.x, e * n},
                        {in.post_w, pb}, {in.post_b, pb}, {in.pre_w, pb}, {in.pre_b, pb},
                        {in.gate, pb}};
  if (overlapping(spans, 6)) return FP8L_EINVAL;
  const hipError_t err = fp8l::resnorm_fwd_launch(in, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_resnorm_quantize(const fp8l_resnorm *r, int scaling, void *q, void *qt, float *scale,
                         float *scale_t, float *amax_out, void *workspace,
                         size_t workspace_bytes, void *stream) {
  fp8l::ResIn in;
  const int s = check_resnorm(r, in);
  if (s != FP8L_OK) return s;
  if (scaling != FP8L_TENSORWISE && scaling != FP8L_ROWWISE) return FP8L_EINVAL;
  if (bad_eps(r->eps) || !in.pre) return FP8L_EINVAL;
  const bool rw = scaling == FP8L_ROWWISE;
  const bool rows_only = rw && !qt && in.rows > 0;
  if (in.cols % 16 != 0 || (!rows_only && in.rows % 16 != 0)) return FP8L_ESHAPE;
  if (!rows_only && !fp8l::quantize_fits(in.rows, in.cols, scaling)) return FP8L_ESHAPE;
  if (in.rows > 0 && (!in.x || !q || (!qt && !rows_only))) return FP8L_EINVAL;
  // scale vectors may be NULL only where they have no entries
  if (!scale && (!rw || in.rows > 0)) return FP8L_EINVAL;
  if (!scale_t && (qt || !rw)) return FP8L_EINVAL;
  if (!rows_only && in.rows > 0 && !in.y &&
      (in.f32 || !in.rstd_pre || (!in.rms && !in.mean_pre)))
    return FP8L_EINVAL;
  if (misaligned(q) || misaligned(qt)) return FP8L_EALIGN;
  if (misaligned4(scale) || misaligned4(scale_t) || misaligned4(amax_out)) return FP8L_EALIGN;
  size_t need = 0;
  if (!rows_only) {
    if (rw && !scale_t) return FP8L_OK;          // no rows, no column scales wanted
    if (!workspace) return FP8L_EINVAL;
    need = fp8l::resnorm_workspace_bytes(in.rows, in.cols, scaling);
    if (workspace_bytes < need) return FP8L_EWORKSPACE;
    if (misaligned(workspace)) return FP8L_EALIGN;
  }
  const int64_t n = in.rows * in.cols, e = in.f32 ? 4 : 2, pb = in.cols * (in.wf32 ? 4 : 2);
  const int64_t sr = rw ? 4 * in.rows : 4, sc = rows_only ? 0 : rw ? 4 * in.cols : 4;
  const Span spans[] = {{in.s, e * n}, {in.y, 2 * n}, {q, n}, {qt, n}, {scale, sr},
                        {scale_t, sc}, {amax_out, rw ? sr + sc : 4}, {workspace, (int64_t)need},
                        {in.mean_post, 4 * in.rows}, {in.rstd_post, 4 * in.rows},
                        {in.mean_pre, 4 * in.rows}, {in.rstd_pre, 4 * in.rows},
                        {in.b, 2 * n}, {in.x, e * n}, {in.post_w, pb}, {in.post_b, pb},
                        {in.pre_w, pb}, {in.pre_b, pb}, {in.gate, pb}};
  if (overlapping(spans, 12)) return FP8L_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t err =
      rows_only ? fp8l::resnorm_rows_launch(in, q, scale, amax_out, st)
                : fp8l::resnorm_quantize_launch(in, scaling, {q, qt, scale, scale_t, amax_out},
                                                workspace, st);
  return err == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_resnorm_bwd(const fp8l_resnorm *r, const void *dy, const void *ds,
                    const fp8l_resnorm_grads *g, int scaling, void *q, void *qt, float *scale,
                    float *scale_t, float *amax_out, void *workspace, size_t workspace_bytes,
                    void *stream) {
  fp8l::ResIn in;
  const int s = check_resnorm(r, in);
  if (s != FP8L_OK) return s;
  if (!g || bad_scaling(scaling)) return FP8L_EINVAL;
  const bool quant = q || qt || scale || scale_t || amax_out;
  if (quant && (in.rows % 16 != 0 || in.cols % 16 != 0)) return FP8L_ESHAPE;
  if (in.rows > 0) {
    if (!g->db || !dy != !in.pre || (!ds && !in.pre)) return FP8L_EINVAL;
    if ((in.post && (!in.rstd_post || (!in.rms && !in.mean_post))) ||
        (in.pre && (!in.rstd_pre || (!in.rms && !in.mean_pre))))
      return FP8L_EINVAL;
  }
  if ((!in.post && (g->dpost_w || g->dpost_b)) || (!in.pre && (g->dpre_w || g->dpre_b)) ||
      (!in.gate && g->dgate))
    return FP8L_EINVAL;
  if (misaligned(dy) || misaligned(ds) || misaligned(g->dx) || misaligned(g->db))
    return FP8L_EALIGN;
  const bool wants = g->dgate || g->dpost_w || g->dpost_b || g->dpre_w || g->dpre_b;
  const int64_t beside = wants ? 2 * ((in.cols + 63) / 64) : 0;
  if (quant && !fp8l::quantize_fits(in.rows, in.cols, scaling, beside)) return FP8L_ESHAPE;
  for (const float *f : {g->dgate, g->dpost_w, g->dpost_b, g->dpre_w, g->dpre_b})
    if (misaligned4(f)) return FP8L_EALIGN;
  if (quant) {
    const int e = check_quantize_args(g->db, in.rows, in.cols, scaling, q, qt, scale, scale_t,
                                      amax_out);
    if (e != FP8L_OK) return e;
  }
  size_t need = 0;
  if (wants || quant) {
    if (!workspace) return FP8L_EINVAL;
    need = fp8l::resnorm_workspace_bytes(in.rows, in.cols, scaling);
    if (workspace_bytes < need) return FP8L_EWORKSPACE;
    if (misaligned(workspace)) return FP8L_EALIGN;
  }
  const int64_t n = in.rows * in.cols, e = in.f32 ? 4 : 2, pb = in.cols * (in.wf32 ? 4 : 2);
  const int64_t cb = 4 * in.cols, rb = 4 * in.rows;
  const bool rw = (scaling & FP8L_ROWWISE) != 0;
  const int64_t sr = rw ? rb : 4, sc = rw ? cb : 4;
  const Span spans[] = {{g->dx, e * n}, {g->db, 2 * n}, {g->dgate, cb}, {g->dpost_w, cb},
                        {g->dpost_b, cb}, {g->dpre_w, cb}, {g->dpre_b, cb}, {q, n}, {qt, n},
                        {scale, sr}, {scale_t, sc}, {amax_out, rw ? sr + sc : 4},
                        {workspace, (int64_t)need}, {dy, 2 * n}, {ds, e * n}, {in.b, 2 * n},
                        {in.s, e * n}, {in.post_w, pb}, {in.post_b, pb}, {in.pre_w, pb},
                        {in.pre_b, pb}, {in.gate, pb}, {in.mean_post, rb}, {in.rstd_post, rb},
                        {in.mean_pre, rb}, {in.rstd_pre, rb}};
  if (overlapping(spans, 13)) return FP8L_EINVAL;
  const fp8l::ResGrads gr = {g->dx, g->db, g->dgate, g->dpost_w, g->dpost_b, g->dpre_w,
                             g->dpre_b};
  const fp8l::Fp8Out o = {q, qt, scale, scale_t, amax_out};
  const hipError_t err = fp8l::resnorm_bwd_launch(in, dy, ds, gr, scaling, quant ? &o : nullptr,
                                                  workspace, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_encode_e4m3(const float *in, uint8_t *out, int64_t n, void *stream) {
  if (n < 0 || n > kMaxElems) return FP8L_ESHAPE;
  if (n == 0) return FP8L_OK;
  if (!in || !out) return FP8L_EINVAL;
  if (misaligned(in) || misaligned(out)) return FP8L_EALIGN;
  hipError_t e = fp8l::encode_launch(in, out, n, 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

int fp8_linear_encode_e5m2(const float *in, uint8_t *out, int64_t n, void *stream) {
  if (n < 0 || n > kMaxElems) return FP8L_ESHAPE;
  if (n == 0) return FP8L_OK;
  if (!in || !out) return FP8L_EINVAL;
  if (misaligned(in) || misaligned(out)) return FP8L_EALIGN;
  hipError_t e = fp8l::encode_launch(in, out, n, 1, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8L_OK : FP8L_EHIP;
}

const char *fp8_linear_status_string(int status) {
  switch (status) {
    case FP8L_OK: return "ok";
    case FP8L_EINVAL: return "invalid argument (null pointer or unknown enum)";
    case FP8L_ESHAPE: return "invalid shape (dimension < 0 or not a multiple of 16)";
    case FP8L_EALIGN: return "misaligned pointer (tensors need 16-byte alignment)";
    case FP8L_EWORKSPACE: return "workspace too small";
    case FP8L_EHIP: return "HIP launch or runtime error";
    default: return "unknown status";
  }
}

const char *fp8_linear_version(void) { return "fp8_linear 0.1 gfx950"; }

}  // extern "C"
