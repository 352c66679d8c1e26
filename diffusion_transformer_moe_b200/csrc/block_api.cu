// C entry points of the operators around the layer: argument checks, workspaces, launches.
// As in api.cu, every check runs on the host before anything is enqueued.
#include <math.h>

#include <atomic>

#include "block_ops.cuh"

namespace nmoe {
#ifdef NMOE_DEBUG
static std::atomic<uint64_t> g_block_wait_ns{kDefaultWaitNs};
uint64_t block_wait_ns() { return g_block_wait_ns.load(); }
// Debug build only: the budget of the block operators' waits from now on; with 0 the first
// wait of every kernel runs out.
extern "C" __attribute__((visibility("default"))) void nmoe_debug_block_wait_ns(uint64_t ns) {
  g_block_wait_ns.store(ns);
}
#else
uint64_t block_wait_ns() { return kDefaultWaitNs; }
#endif
}  // namespace nmoe

namespace {

using nmoe::current_device;

constexpr int kMaxSms = 160;                    // more than any sm_100 part has
constexpr int64_t kMaxNormDim = 16384;          // a row stays in one block's registers
constexpr int64_t kMaxLinearDim = int64_t(1) << 30;  // tile coordinates are 32-bit

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
size_t esize(nmoe_dtype dt) { return dt == NMOE_F32 ? 4 : 2; }
bool is_dtype(nmoe_dtype dt) { return dt == NMOE_BF16 || dt == NMOE_F32; }
bool is_act(nmoe_act a) { return a >= NMOE_ACT_NONE && a <= NMOE_ACT_GELU_TANH; }

// The arrays of one call. Absent ones (NULL) are skipped; every other must be 16-byte
// aligned, and no output may share a byte with an input or with another output.
struct Arrays {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  } r[16];
  int n = 0;
  bool ok = true;
  void add(const void* p, int64_t bytes, bool out) {
    if (!p) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (!aligned16(p)) ok = false;
    for (int i = 0; i < n; ++i)
      if ((out || r[i].out) && lo < r[i].hi && r[i].lo < lo + (uintptr_t)bytes) ok = false;
    r[n++] = {lo, lo + (uintptr_t)bytes, out};
  }
  void in(const void* p, int64_t bytes) { add(p, bytes, false); }
  void out(const void* p, int64_t bytes) { add(p, bytes, true); }
};

// A caller's workspace, or a stream-ordered allocation for the call.
struct Workspace {
  char* p = nullptr;
  bool own = false;
  nmoe_status take(void* given, size_t given_bytes, size_t need, cudaStream_t st) {
    if (need == 0) return NMOE_OK;
    if (given) {
      if (given_bytes < need) return NMOE_ERR_WORKSPACE;
      p = static_cast<char*>(given);
      return NMOE_OK;
    }
    if (cudaMallocAsync(reinterpret_cast<void**>(&p), need, st) != cudaSuccess) {
      cudaGetLastError();
      return NMOE_ERR_WORKSPACE;
    }
    own = true;
    return NMOE_OK;
  }
  nmoe_status finish(cudaError_t e, cudaStream_t st) {
    if (own) {
      const cudaError_t f = cudaFreeAsync(p, st);
      if (e == cudaSuccess) e = f;
    }
    if (e == cudaSuccess) return NMOE_OK;
    cudaGetLastError();
    return NMOE_ERR_CUDA;
  }
};

bool workspace_ok(const void* workspace) {
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0;
}

nmoe_status check_rows(int64_t T, int64_t d, nmoe_dtype dt) {
  if (!is_dtype(dt) || T < 1 || T >= (int64_t(1) << 31) || d < 1) return NMOE_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > kMaxNormDim) return NMOE_ERR_UNSUPPORTED;
  return NMOE_OK;
}

nmoe_status check_linear(int64_t M, int64_t K, int64_t N, nmoe_act act, int k_multiple) {
  if (M < 1 || K < 1 || N < 1 || !is_act(act)) return NMOE_ERR_INVALID_ARG;
  if (M > kMaxLinearDim || K > kMaxLinearDim || N > kMaxLinearDim) return NMOE_ERR_UNSUPPORTED;
  if (K % k_multiple != 0 || N % 8 != 0) return NMOE_ERR_UNSUPPORTED;
  return NMOE_OK;
}

nmoe_status check_balance(int64_t T, int64_t E, int64_t k, int64_t n_seg, float coef) {
  if (T < 1 || T >= (int64_t(1) << 31) || E < 1 || E > 256) return NMOE_ERR_INVALID_ARG;
  if (n_seg < 1 || n_seg > 65535 || T % n_seg != 0) return NMOE_ERR_INVALID_ARG;
  if (k < 1 || k > E || !isfinite(coef)) return NMOE_ERR_INVALID_ARG;
  return NMOE_OK;
}

nmoe_status linear(nmoe::Linear& a, nmoe_dtype out_dtype, int k_multiple, cudaStream_t st) {
  nmoe_status v = check_linear(a.M, a.K, a.N, a.act, k_multiple);
  if (v != NMOE_OK) return v;
  if (!is_dtype(out_dtype) || !a.x || !a.w || !a.out) return NMOE_ERR_INVALID_ARG;
  a.out_f32 = out_dtype == NMOE_F32;
  const int64_t es = a.x_scale ? 1 : 2;
  Arrays r;
  r.in(a.x, a.M * a.K * es);
  r.in(a.w, a.K * a.N * es);
  r.in(a.x_scale, 4 * a.M);
  r.in(a.w_scale, 4 * a.N);
  r.in(a.bias, 2 * a.N);
  r.in(a.residual, 2 * a.M * a.N);
  r.out(a.preact, 2 * a.M * a.N);
  r.out(a.out, (int64_t)esize(out_dtype) * a.M * a.N);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  if (nmoe::launch_linear(a, err, sms, st) != cudaSuccess) {
    cudaGetLastError();
    return NMOE_ERR_CUDA;
  }
  return NMOE_OK;
}

// Parts of the gradient's workspace: dz (with an activation) and dbias's partial rows.
struct BackwardLayout {
  size_t dz, partial, total;
};
BackwardLayout backward_layout(int64_t M, int64_t N, nmoe_act act) {
  BackwardLayout l;
  l.dz = 0;
  l.partial = act == NMOE_ACT_NONE ? 0 : align256((size_t)2 * M * N);
  l.total = l.partial + align256((size_t)4 * nmoe::linear_dz_partial_rows(M, (int)N) * N);
  return l;
}

}  // namespace

extern "C" {

nmoe_status nmoe_rms_norm(const void* x, const void* residual, const void* weight, int64_t T,
                          int64_t d, float eps, nmoe_dtype dtype, void* h, void* y, void* q,
                          float* scale, float* rstd, nmoe_stream_t stream) {
  nmoe_status v = check_rows(T, d, dtype);
  if (v != NMOE_OK) return v;
  if (!(eps >= 0.f) || !isfinite(eps)) return NMOE_ERR_INVALID_ARG;
  if (!x || (!y && !q) || (q == nullptr) != (scale == nullptr) ||
      (residual == nullptr) != (h == nullptr))
    return NMOE_ERR_INVALID_ARG;
  const int64_t bytes = T * d * (int64_t)esize(dtype);
  Arrays r;
  r.in(x, bytes);
  r.in(residual, bytes);
  r.in(weight, d * (int64_t)esize(dtype));
  r.out(h, bytes);
  r.out(y, bytes);
  r.out(q, T * d);
  r.out(scale, 4 * T);
  r.out(rstd, 4 * T);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  if (nmoe::launch_rms_norm(x, residual, weight, T, (int)d, eps, dtype, h, y, q, scale, rstd, sms,
                            static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return NMOE_ERR_CUDA;
  }
  return NMOE_OK;
}

size_t nmoe_rms_norm_backward_workspace(int64_t T, int64_t d) {
  if (check_rows(T, d, NMOE_F32) != NMOE_OK) return 0;
  // a partial row a block, for either type and any device; one block or cluster needs none
  int parts = 1;
  for (nmoe_dtype dt : {NMOE_BF16, NMOE_F32}) {
    const int n = nmoe::rms_norm_backward_parts(T, (int)d, dt, kMaxSms);
    if (n > parts) parts = n;
  }
  return parts > 1 ? align256((size_t)4 * parts * d) : 0;
}

nmoe_status nmoe_rms_norm_backward(const void* dy, const void* h, const float* rstd,
                                   const void* weight, const void* dh, int64_t T, int64_t d,
                                   nmoe_dtype dtype, void* dx, float* dweight, void* workspace,
                                   size_t workspace_bytes, nmoe_stream_t stream) {
  nmoe_status v = check_rows(T, d, dtype);
  if (v != NMOE_OK) return v;
  if (!dy || !h || !rstd || !dx || !workspace_ok(workspace)) return NMOE_ERR_INVALID_ARG;
  const int64_t bytes = T * d * (int64_t)esize(dtype);
  const size_t need = dweight ? nmoe_rms_norm_backward_workspace(T, d) : 0;
  Arrays r;
  r.in(dy, bytes);
  r.in(h, bytes);
  r.in(rstd, 4 * T);
  r.in(weight, d * (int64_t)esize(dtype));
  r.in(dh, bytes);
  r.out(dx, bytes);
  r.out(dweight, 4 * d);
  // (with dweight, one inside another array is refused also where these sizes write none of it)
  r.out(workspace, dweight && need == 0 ? 1 : (int64_t)need);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Workspace ws;
  if ((v = ws.take(workspace, workspace_bytes, need, st)) != NMOE_OK) return v;
  return ws.finish(nmoe::launch_rms_norm_backward(dy, h, rstd, weight, dh, T, (int)d, dtype, dx,
                                                  dweight, reinterpret_cast<float*>(ws.p), err,
                                                  sms < kMaxSms ? sms : kMaxSms, st),
                   st);
}

nmoe_status nmoe_quantize_rows(const void* x, int64_t T, int64_t d, nmoe_dtype dtype, void* q,
                               float* scale, nmoe_stream_t stream) {
  nmoe_status v = check_rows(T, d, dtype);
  if (v != NMOE_OK) return v;
  if (!x || !q || !scale) return NMOE_ERR_INVALID_ARG;
  Arrays r;
  r.in(x, T * d * (int64_t)esize(dtype));
  r.out(q, T * d);
  r.out(scale, 4 * T);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  if (nmoe::launch_quantize_rows(x, T, (int)d, dtype, q, scale, sms,
                                 static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return NMOE_ERR_CUDA;
  }
  return NMOE_OK;
}

nmoe_status nmoe_linear(const void* x, const void* W, const void* bias, const void* residual,
                        int64_t M, int64_t K, int64_t N, nmoe_act act, nmoe_dtype out_dtype,
                        void* preact, void* out, nmoe_stream_t stream) {
  nmoe::Linear a = {x, W, nullptr, nullptr, bias, residual, preact, out, M, K, N, act, false};
  return linear(a, out_dtype, 8, static_cast<cudaStream_t>(stream));
}

nmoe_status nmoe_linear_fp8(const void* q_x, const float* x_scale, const void* q_w,
                            const float* w_scale, const void* bias, const void* residual,
                            int64_t M, int64_t K, int64_t N, nmoe_act act, nmoe_dtype out_dtype,
                            void* out, nmoe_stream_t stream) {
  if (!x_scale || !w_scale) return NMOE_ERR_INVALID_ARG;
  nmoe::Linear a = {q_x, q_w, x_scale, w_scale, bias, residual, nullptr, out, M, K, N, act,
                    false};
  return linear(a, out_dtype, 16, static_cast<cudaStream_t>(stream));
}

size_t nmoe_linear_backward_workspace(int64_t M, int64_t K, int64_t N, nmoe_act act) {
  if (check_linear(M, K, N, act, 8) != NMOE_OK) return 0;
  return backward_layout(M, N, act).total;
}

nmoe_status nmoe_linear_backward(const void* dy, const void* x, const void* W,
                                 const void* preact, int64_t M, int64_t K, int64_t N,
                                 nmoe_act act, void* dx, void* dW, float* dbias,
                                 void* workspace, size_t workspace_bytes,
                                 nmoe_stream_t stream) {
  nmoe_status v = check_linear(M, K, N, act, 8);
  if (v != NMOE_OK) return v;
  if (!dy || (!dx && !dW && !dbias) || (dW && !x) || (dx && !W) || !workspace_ok(workspace))
    return NMOE_ERR_INVALID_ARG;
  if ((act != NMOE_ACT_NONE) != (preact != nullptr)) return NMOE_ERR_INVALID_ARG;
  const BackwardLayout l = backward_layout(M, N, act);
  const bool products = dx || dW;
  // without an activation dz is dy itself
  const size_t need = dbias ? l.total : products && preact ? l.partial : 0;
  Arrays r;
  r.in(dy, 2 * M * N);
  r.in(dW ? x : nullptr, 2 * M * K);
  r.in(dx ? W : nullptr, 2 * K * N);
  r.in(preact, 2 * M * N);
  r.out(dx, 2 * M * K);
  r.out(dW, 2 * K * N);
  r.out(dbias, 4 * N);
  r.out(workspace, (int64_t)need);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Workspace ws;
  if ((v = ws.take(workspace, workspace_bytes, need, st)) != NMOE_OK) return v;
  void* dz = products && preact ? ws.p + l.dz : nullptr;
  float* partial = reinterpret_cast<float*>(ws.p + l.partial);
  cudaError_t e = cudaSuccess;
  // dbias is of the unrounded dz: without an activation of dy itself, whatever computes it
  const bool first = dz || !products;
  if (first) e = nmoe::launch_linear_dz(dy, preact, M, (int)N, act, dz, dbias, partial, st);
  if (e == cudaSuccess && products)
    e = nmoe::launch_linear_grads(dz ? dz : dy, x, W, M, K, N, dx, dW, first ? nullptr : dbias,
                                  partial, err, sms, st);
  return ws.finish(e, st);
}

size_t nmoe_balance_loss_workspace(int64_t T, int64_t E, int64_t n_segments) {
  if (check_balance(T, E, 1, n_segments, 0.f) != NMOE_OK) return 0;
  return align256(nmoe::balance_workspace(T / n_segments, (int)E, (int)n_segments));
}

nmoe_status nmoe_balance_loss(const float* scores, const uint8_t* mask, int64_t T, int64_t E,
                              int64_t k, int64_t n_segments, float coef, int32_t* counts,
                              float* loss, void* workspace, size_t workspace_bytes,
                              nmoe_stream_t stream) {
  nmoe_status v = check_balance(T, E, k, n_segments, coef);
  if (v != NMOE_OK) return v;
  if (!scores || !counts || !loss || !workspace_ok(workspace)) return NMOE_ERR_INVALID_ARG;
  const size_t need = nmoe_balance_loss_workspace(T, E, n_segments);
  Arrays r;
  r.in(scores, 4 * T * E);
  r.in(mask, T);
  r.out(counts, 4 * n_segments * E);
  r.out(loss, 4 * n_segments);
  r.out(workspace, (int64_t)need);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Workspace ws;
  if ((v = ws.take(workspace, workspace_bytes, need, st)) != NMOE_OK) return v;
  return ws.finish(nmoe::launch_balance_loss(scores, mask, T, (int)E, (int)k, (int)n_segments,
                                             coef, counts, loss, ws.p, st),
                   st);
}

nmoe_status nmoe_balance_loss_backward(const float* scores, const uint8_t* mask,
                                       const int32_t* counts, const float* dloss, int64_t T,
                                       int64_t E, int64_t k, int64_t n_segments, float coef,
                                       nmoe_score_fn score_fn, nmoe_dtype dtype, void* dlogits,
                                       nmoe_stream_t stream) {
  nmoe_status v = check_balance(T, E, k, n_segments, coef);
  if (v != NMOE_OK) return v;
  if (score_fn != NMOE_SCORE_SOFTMAX && score_fn != NMOE_SCORE_SIGMOID)
    return NMOE_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || !scores || !counts || !dlogits) return NMOE_ERR_INVALID_ARG;
  Arrays r;
  r.in(scores, 4 * T * E);
  r.in(mask, T);
  r.in(counts, 4 * n_segments * E);
  r.in(dloss, 4 * n_segments);
  r.out(dlogits, (int64_t)esize(dtype) * T * E);
  if (!r.ok) return NMOE_ERR_INVALID_ARG;
  unsigned* err;
  int sms;
  if ((v = current_device(&err, &sms)) != NMOE_OK) return v;
  if (nmoe::launch_balance_backward(scores, mask, counts, dloss, T, (int)E, (int)k,
                                    (int)n_segments, coef, score_fn, dtype, dlogits, sms,
                                    static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return NMOE_ERR_CUDA;
  }
  return NMOE_OK;
}

}  // extern "C"
