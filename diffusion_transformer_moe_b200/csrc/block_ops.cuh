// Declarations of the operators around the layer (norm.cu, linear.cu, balance.cu) and what
// their C entry points share. Sizes arrive here validated.
#pragma once

#include "nmoe_internal.cuh"

namespace nmoe {

// 16 bytes that this kernel reads once. Volatile, so that the load stays behind the wait
// for the previous kernel (the compiler may move the plain load intrinsics across it).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The budget of each bounded wait of these operators; the debug build may set another.
uint64_t block_wait_ns();

// Column sums that more than one CTA or cluster computes are left as partial rows
// [parts, d] fp32 and added up in a fixed order by a second launch (launch_sum_parts), so a
// result never depends on which CTA ran first.

cudaError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int64_t T,
                            int d, float eps, nmoe_dtype dt, void* h, void* y, void* q,
                            float* scale, float* rstd, int sm_count, cudaStream_t st);
// normalise = false: the rows themselves are quantised
cudaError_t launch_quantize_rows(const void* x, int64_t T, int d, nmoe_dtype dt, void* q,
                                 float* scale, int sm_count, cudaStream_t st);
int rms_norm_backward_parts(int64_t T, int d, nmoe_dtype dt, int sm_count);
cudaError_t launch_rms_norm_backward(const void* dy, const void* h, const float* rstd,
                                     const void* weight, const void* dh, int64_t T, int d,
                                     nmoe_dtype dt, void* dx, float* dweight, float* partial,
                                     unsigned* err, int sm_count, cudaStream_t st);
// out[c] = sum over i < parts of partial[i, c], in a fixed order
cudaError_t launch_sum_parts(const float* partial, int parts, int d, float* out,
                             cudaStream_t st);

struct Linear {
  const void* x;          // [M, K] bf16, or e4m3
  const void* w;          // [K, N] bf16, or [N, K] e4m3
  const float* x_scale;   // [M], e4m3 only
  const float* w_scale;   // [N], e4m3 only
  const void* bias;       // [N] bf16 or NULL
  const void* residual;   // [M, N] bf16 or NULL
  void* preact;           // [M, N] bf16 or NULL
  void* out;              // [M, N]
  int64_t M, K, N;
  nmoe_act act;
  bool out_f32;
};
cudaError_t launch_linear(const Linear& a, unsigned* err, int sm_count, cudaStream_t st);
// dz = dy * act'(preact) in bf16 (dz NULL: not written) and its column sums (dbias NULL: not
// wanted); partial: linear_dz_partial_rows() rows [N] of scratch for them
int linear_dz_partial_rows(int64_t M, int N);
cudaError_t launch_linear_dz(const void* dy, const void* preact, int64_t M, int N, nmoe_act act,
                             void* dz, float* dbias, float* partial, cudaStream_t st);
// dx [M, K] = dz [M, N] W^T and dW [K, N] = x^T dz, all bf16, either may be NULL; dbias
// [N] (NULL: not wanted), the column sums of dz, with partial as above
cudaError_t launch_linear_grads(const void* dz, const void* x, const void* W, int64_t M,
                                int64_t K, int64_t N, void* dx, void* dW, float* dbias,
                                float* partial, unsigned* err, int sm_count, cudaStream_t st);

size_t balance_workspace(int64_t S, int E, int n_seg);  // bytes
cudaError_t launch_balance_loss(const float* scores, const uint8_t* mask, int64_t T, int E,
                                int k, int n_seg, float coef, int32_t* counts, float* loss,
                                void* workspace, cudaStream_t st);
cudaError_t launch_balance_backward(const float* scores, const uint8_t* mask,
                                    const int32_t* counts, const float* dloss, int64_t T, int E,
                                    int k, int n_seg, float coef, nmoe_score_fn fn,
                                    nmoe_dtype dt, void* dlogits, int sm_count,
                                    cudaStream_t st);

}  // namespace nmoe
