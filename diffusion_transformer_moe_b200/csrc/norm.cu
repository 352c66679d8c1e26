// Residual RMS norm of token rows, its 8-bit output, its gradient, and the 8-bit rows alone.
//
// Every row is read once: its values stay in registers (fp32) between the sum of squares,
// the norm, the row's largest magnitude and the 8-bit rounding, so the forward moves the
// bytes of its inputs and outputs and nothing else, and HBM bounds it. 16-byte loads and
// stores; one warp holds a row of up to 64 values a lane (shuffles only, no block
// barrier), a block the longer rows.
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "sm100_ptx.cuh"

namespace nmoe {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: its reciprocal is still finite
constexpr float kLowMean = 0x1p-100f, kHighMean = 3.4028235e38f;

// maximum that keeps a NaN of either side (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(pack_e4m3(f[0], f[1], f[2], f[3]), pack_e4m3(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[4]) {
  *reinterpret_cast<uint32_t*>(p) = pack_e4m3(f[0], f[1], f[2], f[3]);
}

struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct MaxNan {
  __device__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// The result over a row's TPR threads, in every one of them. A row of more than one warp
// is its whole block; `sh` then holds one value a warp and is used for one reduction only.
template <int TPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, float* sh, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = op(v, sh[i]);
  }
  return v;
}

// TPR threads a row, VPT 16-byte vectors a thread. NORM false: the rows are quantised as
// they are (x to q and scale), five blocks an SM (8192 x 8192 bf16: 31.8 us, with four 34).
template <typename T, int TPR, int VPT, bool NORM>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, !NORM && TPR == 256 && VPT <= 4 ? 5 : 0)
rms_norm_kernel(const T* x, const T* residual, const T* weight, int64_t rows, int d, float eps,
                T* h, T* y, uint8_t* q, float* scale, float* rstd_out) {
  constexpr int N = Vec<T>::kN;
  constexpr int kRows = TPR == 32 ? 4 : 1;
  __shared__ float sh_sum[32], sh_again[32], sh_max[32];
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= rows) return;  // a whole warp (TPR == 32); never part of a block that waits
  const int nv = d / N;
  const int64_t at = row * d;
  uint4 raw[VPT], rres[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * TPR;
    raw[i] = rres[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      raw[i] = load_once(reinterpret_cast<const uint4*>(x + at) + v);
      if (NORM && residual) rres[i] = load_once(reinterpret_cast<const uint4*>(residual + at) + v);
    }
  }
  float f[VPT][N];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * TPR;
    unpack(raw[i], f[i]);
    if (NORM && residual) {
      float r[N];
      unpack(rres[i], r);
#pragma unroll
      for (int j = 0; j < N; ++j) f[i][j] += r[j];
      // the norm is taken of the sum as it is stored, which is what the gradient reads
      const uint4 hv = pack(f[i]);
      unpack(hv, f[i]);
      if (v < nv) reinterpret_cast<uint4*>(h + at)[v] = hv;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) ss = fmaf(f[i][j], f[i][j], ss);
  }
  if constexpr (NORM) {
    ss = row_reduce<TPR>(ss, sh_sum, Add());
    const float mean = ss / (float)d + eps;
    // y = h a r weight, and rstd = a r: of the smallest rows it is beyond fp32, and y is not
    float a = 1.f, r = 1.f / sqrtf(mean), rstd = r;
    if (mean < kLowMean || mean > kHighMean) {
      // the squares underflow (each is off by up to 2^-150, half of fp32's smallest step: not
      // seen in a mean of 2^-100) or sum beyond fp32: the whole row once more, scaled by a
      // power of two. A true infinity stays one
      const float up = mean < kLowMean ? 0x1p100f : 0x1p-80f;
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float s = f[i][j] * up;
          ss = fmaf(s, s, ss);
        }
      ss = row_reduce<TPR>(ss, sh_again, Add());
      r = 1.f / sqrtf(ss / (float)d + eps * up * up);
      rstd = r * up;
      if (up > 1.f) a = up; else r = rstd;
    }
    if (t == 0 && rstd_out) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + i * TPR;
      float w[N];
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = 1.f;
      if (weight && v < nv) unpack(reinterpret_cast<const uint4*>(weight)[v], w);
#pragma unroll
      for (int j = 0; j < N; ++j) f[i][j] = f[i][j] * a * r * w[j];
      if (y && v < nv) reinterpret_cast<uint4*>(y + at)[v] = pack(f[i]);
    }
  }
  if (!q) return;  // the same for every thread
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (t + i * TPR < nv) {
#pragma unroll
      for (int j = 0; j < N; ++j) m = max_nan(m, fabsf(f[i][j]));
    }
  m = row_reduce<TPR>(m, sh_max, MaxNan());
  const float sc = max_nan(m / kE4m3Max, kTinyScale);
  // The codes are those of the quotient y / scale. y * (1 / scale) alone is rounded twice and
  // gives 50 codes in a million a neighbour's value; a division a value took 8192 x 2048 bf16
  // rows from 9.3 to 15.6 us. One division a row and the remainder's correction of each
  // product give the rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990).
  float by = sc;
  if (sc < 0x1p-64f) {  // the remainders of such rows would be subnormal
    by = sc * 0x1p64f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) f[i][j] *= 0x1p64f;
  }
  const float inv = 1.f / by;
  if (by > 3.4028235e38f) by = 0.f;  // a row with an infinity: finite values' codes are 0
  if (t == 0) scale[row] = sc;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * TPR;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float c = f[i][j] * inv;
      f[i][j] = fmaf(-fmaf(c, by, -f[i][j]), inv, c);
    }
    if (v < nv) store_e4m3(q + at + (int64_t)v * N, f[i]);
  }
}

template <typename T, int TPR, int VPT, bool NORM>
cudaError_t launch_rows(const void* x, const void* residual, const void* weight, int64_t rows,
                        int d, float eps, void* h, void* y, void* q, float* scale, float* rstd,
                        cudaStream_t st) {
  constexpr int kRows = TPR == 32 ? 4 : 1;
  return launch_kernel(rms_norm_kernel<T, TPR, VPT, NORM>,
                       dim3((unsigned)ceil_div(rows, kRows)), dim3(TPR == 32 ? 128 : TPR), 0, st,
                       true, 1, static_cast<const T*>(x), static_cast<const T*>(residual),
                       static_cast<const T*>(weight), rows, d, eps, static_cast<T*>(h),
                       static_cast<T*>(y), static_cast<uint8_t*>(q), scale, rstd);
}

// Rows of up to 256 vectors (2048 bf16, 1024 fp32 values) go to one warp each once there
// are rows enough for every SM's warps, else to a block of 256 threads: with 512 bf16
// values, residual and 8-bit output, 1 row takes 1.7 us on a block and 1.95 on a warp, 592
// rows 2.5 and 2.25, 8192 rows 19 and 7.3. From 129 vectors on the warp's longer rows pay only
// with the second reduction of an 8-bit output (8192 x 2048 bf16 with a residual: 22.8 and
// 21.1 us; without an 8-bit output 22.3 and 24.6), and where h and y go out too up to 192 (8192
// x 1344 22.2 and 17.7 us, 8192 x 2048 26.7 and 27.9, 4000 x 2048 12.7 and 13.5).
template <typename T, bool NORM>
cudaError_t launch_rows_of(const void* x, const void* residual, const void* weight, int64_t rows,
                           int d, float eps, void* h, void* y, void* q, float* scale,
                           float* rstd, int sm_count, cudaStream_t st) {
  const int nv = d / Vec<T>::kN;
  auto go = [&](auto fn) {
    return fn(x, residual, weight, rows, d, eps, h, y, q, scale, rstd, st);
  };
  if (nv <= 32) return go(launch_rows<T, 32, 1, NORM>);
  const int longest = !q ? 128 : residual && y ? 192 : 256;
  if (nv <= longest && 16 * rows >= (int64_t)nv * sm_count) {
    if (nv <= 64) return go(launch_rows<T, 32, 2, NORM>);
    if (nv <= 128) return go(launch_rows<T, 32, 4, NORM>);
    return go(launch_rows<T, 32, 8, NORM>);
  }
  if (nv <= 256) return go(launch_rows<T, 256, 1, NORM>);
  if (nv <= 512) return go(launch_rows<T, 256, 2, NORM>);
  if (nv <= 1024) return go(launch_rows<T, 256, 4, NORM>);
  if (nv <= 2048) return go(launch_rows<T, 256, 8, NORM>);
  if constexpr (sizeof(T) == 4) return go(launch_rows<T, 512, 8, NORM>);
  return cudaErrorInvalidValue;  // d <= 16384 was checked
}

// ---- gradient -----------------------------------------------------------------------------
//
// Persistent, one block an SM. A group of WPR warps takes a row at a time from its own ring
// of slots, which bulk copies keep full (dy, h and dh of a row are contiguous), so the
// reductions of one group run under the copies of all. A thread owns the same columns of
// every row, so dweight accumulates in its registers, and a block leaves one partial row.
// Bound by HBM: three rows in and one out for each row. With the rows in registers instead
// (four of them a block and barrier, four blocks an SM) the loads stopped at each reduction
// and 8192 x 2048 bf16 took 30 us; clusters of four blocks to add the partial rows made
// that 46 us.
constexpr int kBwdWarps = 16;
constexpr int kBwdThreads = 32 * kBwdWarps;
constexpr int kBwdMaxSlots = 4;
constexpr int kBwdRing = 196608;

__device__ __forceinline__ void group_sync(int grp, int threads) {
  if (threads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(threads) : "memory");
}

template <typename T, int WPR, int VPT>
__global__ void __launch_bounds__(kBwdThreads, 1)
rms_norm_backward_kernel(const T* dy, const T* h, const float* rstd, const T* weight,
                         const T* dh, int64_t rows, int d, T* dx, float* partial, int slots,
                         int cluster, unsigned* err, uint64_t wait_ns) {
  constexpr int N = Vec<T>::kN;
  constexpr int kGroups = kBwdWarps / WPR, kGroupThreads = 32 * WPR;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kGroups][kBwdMaxSlots];
  __shared__ float sh_dot[kBwdWarps];
  __shared__ int abort_flag;
  const int grp = threadIdx.x / kGroupThreads, t = threadIdx.x % kGroupThreads;
  const int nv = d / N;
  const uint32_t row_bytes = (uint32_t)d * sizeof(T);
  const int arrays = dh ? 3 : 2;
  uint8_t* const ring = smem + (size_t)grp * slots * arrays * row_bytes;
  if (threadIdx.x == 0) abort_flag = 0;
  if (t < slots) ptx::mbar_init(&full_bar[grp][t], 1);
  ptx::fence_mbar_init();
  __syncthreads();
  volatile int* abort_v = &abort_flag;
  pdl_wait();
  pdl_launch_dependents();

  const int64_t first = (int64_t)blockIdx.x * kGroups + grp;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  auto fetch = [&](int64_t row, int slot) {  // the group's first thread
    uint8_t* to = ring + (size_t)slot * arrays * row_bytes;
    uint64_t* bar = &full_bar[grp][slot];
    ptx::mbar_arrive_expect_tx(bar, arrays * row_bytes);
    ptx::bulk_load(to, dy + row * d, row_bytes, bar);
    ptx::bulk_load(to + row_bytes, h + row * d, row_bytes, bar);
    if (dh) ptx::bulk_load(to + 2 * row_bytes, dh + row * d, row_bytes, bar);
  };
  if (t == 0)
    for (int s = 0; s < slots; ++s)
      if (first + s * step < rows) fetch(first + s * step, s);

  uint4 w[VPT];
  float acc[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * kGroupThreads;
    w[i] = make_uint4(0, 0, 0, 0);
    if (weight && v < nv) w[i] = reinterpret_cast<const uint4*>(weight)[v];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
  }
  int slot = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < rows; row += step) {
    const float rs = rstd[row];
    // (after a timeout the rows that follow are not fetched, and the call's outputs undefined)
    ptx::ring_wait(&full_bar[grp][slot], phase, abort_v, wait_ns);
    const uint4* sdy = reinterpret_cast<const uint4*>(ring + (size_t)slot * arrays * row_bytes);
    const uint4* sh = sdy + nv;
    const uint4* sdh = sh + nv;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + i * kGroupThreads;
      if (v < nv) {
        float g[N], x[N], wf[N];
        unpack(sdy[v], g);
        unpack(sh[v], x);
        unpack(w[i], wf);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float xh = x[j] * rs;
          acc[i][j] = fmaf(g[j], xh, acc[i][j]);
          dot = fmaf(weight ? g[j] * wf[j] : g[j], xh, dot);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 31) == 0) sh_dot[threadIdx.x >> 5] = dot;
      group_sync(grp, kGroupThreads);
      dot = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) dot += sh_dot[grp * WPR + i];
    }
    const float c = -dot / (float)d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = t + i * kGroupThreads;
      if (v < nv) {
        float g[N], x[N], wf[N], o[N];
        unpack(sdy[v], g);
        unpack(sh[v], x);
        unpack(w[i], wf);
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = 0.f;
        if (dh) unpack(sdh[v], o);
#pragma unroll
        for (int j = 0; j < N; ++j)
          o[j] = fmaf(rs, fmaf(x[j] * rs, c, weight ? g[j] * wf[j] : g[j]), o[j]);
        __stcs(reinterpret_cast<uint4*>(dx + row * d) + v, pack(o));
      }
    }
    group_sync(grp, kGroupThreads);  // the slot is read, and sh_dot
    if (t == 0 && row + slots * step < rows && *abort_v == 0) fetch(row + slots * step, slot);
    if (++slot == slots) { slot = 0; phase ^= 1; }
  }
  __syncthreads();  // every slot of the block has been read
  if (*abort_v) {
    // a copy did not arrive in time: report it, and give the others time to land before the
    // shared memory is released
    if (threadIdx.x == 0) atomicOr(err, kErrTimeout);
    const uint64_t t0 = ptx::globaltimer_ns();
    while ((int64_t)(ptx::globaltimer_ns() - t0) < 1000000) {
    }
  }
  if (!partial) return;  // the same for every thread of the grid
  // (after a timeout the sums are as undefined as dx, and every thread still meets the others)
  float* const sums = reinterpret_cast<float*>(smem);
  float* const dw = sums + grp * kGroupThreads * VPT * N;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; j += 4)
      *reinterpret_cast<float4*>(dw + (t + i * kGroupThreads) * N + j) =
          make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
  __syncthreads();
  // the block's groups in order
  for (int c = 4 * threadIdx.x; c < d; c += 4 * kBwdThreads) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float4 v = *reinterpret_cast<const float4*>(sums + g * kGroupThreads * VPT * N + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    // (this thread alone reads these columns of the block's)
    if (cluster > 1) *reinterpret_cast<float4*>(sums + c) = s;
    else *reinterpret_cast<float4*>(partial + (int64_t)blockIdx.x * d + c) = s;
  }
  if (cluster > 1) {
    // the grid is one cluster: its blocks' sums in rank order, each block its share of columns
    __syncwarp();
    ptx::cluster_sync_all();
    for (int c = 4 * (threadIdx.x + kBwdThreads * blockIdx.x); c < d;
         c += 4 * kBwdThreads * cluster) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int o = 0; o < cluster; ++o) {
        const float4 v = ptx::ld_cluster_f4(ptx::mapa_shared(sums + c, (uint32_t)o));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      *reinterpret_cast<float4*>(partial + c) = s;
    }
    __syncwarp();
    ptx::cluster_sync_all();  // no block still reads this one's sums
  }
}

// Warps a row: four vectors a lane at most (eight beyond 2048 a row). 8192 x 2048 bf16 with
// four takes 28 us, with two 33, with eight (a warp a row) 48.
template <typename T>
int warps_per_row(int d) {
  const int nv = d / Vec<T>::kN;
  int w = 1;
  while (w < kBwdWarps && nv > 128 * w) w *= 2;
  return w;
}

template <typename T, int WPR, int VPT>
cudaError_t launch_bwd(const void* dy, const void* h, const float* rstd, const void* weight,
                       const void* dh, int64_t rows, int d, void* dx, float* partial, int parts,
                       int cluster, unsigned* err, cudaStream_t st) {
  const size_t slot = (size_t)(kBwdWarps / WPR) * (dh ? 3 : 2) * d * sizeof(T);
  int slots = (int)(kBwdRing / slot);
  slots = slots < 1 ? 1 : slots > kBwdMaxSlots ? kBwdMaxSlots : slots;
  const size_t sums = sizeof(float) * kBwdThreads * VPT * Vec<T>::kN;
  const size_t smem = slots * slot > sums ? slots * slot : sums;
  return launch_kernel(rms_norm_backward_kernel<T, WPR, VPT>, dim3((unsigned)parts),
                       dim3(kBwdThreads), smem, st, true, (unsigned)cluster,
                       static_cast<const T*>(dy), static_cast<const T*>(h), rstd,
                       static_cast<const T*>(weight), static_cast<const T*>(dh), rows, d,
                       static_cast<T*>(dx), partial, slots, cluster, err, block_wait_ns());
}

template <typename T>
cudaError_t launch_bwd_of(const void* dy, const void* h, const float* rstd, const void* weight,
                          const void* dh, int64_t rows, int d, void* dx, float* partial,
                          int parts, int cluster, unsigned* err, cudaStream_t st) {
  const int nv = d / Vec<T>::kN;
  auto go = [&](auto fn) {
    return fn(dy, h, rstd, weight, dh, rows, d, dx, partial, parts, cluster, err, st);
  };
  switch (warps_per_row<T>(d)) {
    case 1:
      return nv <= 32   ? go(launch_bwd<T, 1, 1>)
             : nv <= 64 ? go(launch_bwd<T, 1, 2>)
                        : go(launch_bwd<T, 1, 4>);
    case 2: return go(launch_bwd<T, 2, 4>);
    case 4: return go(launch_bwd<T, 4, 4>);
    case 8: return go(launch_bwd<T, 8, 4>);
    default: break;
  }
  if constexpr (sizeof(T) == 4)
    if (nv > 2048) return go(launch_bwd<T, 16, 8>);
  return go(launch_bwd<T, 16, 4>);
}

// 32 columns x 32 row slices a block; a slice adds its rows in ascending order, the slices
// are added in ascending order.
__global__ void __launch_bounds__(1024)
sum_parts_kernel(const float* partial, int parts, int d, float* out) {
  __shared__ float sh[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), s = threadIdx.x >> 5;
  float v = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int i = s; i < parts; i += 32) v += partial[(int64_t)i * d + c];
  }
  sh[s][threadIdx.x & 31] = v;
  __syncthreads();
  if (s == 0 && c < d) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sh[i][threadIdx.x];
    out[c] = sum;
  }
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, const void* residual, const void* weight, int64_t T,
                            int d, float eps, nmoe_dtype dt, void* h, void* y, void* q,
                            float* scale, float* rstd, int sm_count, cudaStream_t st) {
  return dt == NMOE_F32
             ? launch_rows_of<float, true>(x, residual, weight, T, d, eps, h, y, q, scale, rstd,
                                           sm_count, st)
             : launch_rows_of<__nv_bfloat16, true>(x, residual, weight, T, d, eps, h, y, q,
                                                   scale, rstd, sm_count, st);
}

cudaError_t launch_quantize_rows(const void* x, int64_t T, int d, nmoe_dtype dt, void* q,
                                 float* scale, int sm_count, cudaStream_t st) {
  return dt == NMOE_F32
             ? launch_rows_of<float, false>(x, nullptr, nullptr, T, d, 0.f, nullptr, nullptr, q,
                                            scale, nullptr, sm_count, st)
             : launch_rows_of<__nv_bfloat16, false>(x, nullptr, nullptr, T, d, 0.f, nullptr,
                                                    nullptr, q, scale, nullptr, sm_count, st);
}

namespace {
// A row a group, then rows in turn on one block an SM. Up to eight blocks are one cluster,
// which finishes dweight in this launch. On the device that takes as long as two launches
// (bf16: 8 x 1024 3.8 against 3.5 us, 128 x 1024 5.6 both, 32 x 4096 6.4 against 5.8), but the
// call is a launch and mostly a workspace shorter: 64 x 1024 10.1 against 14.2 us, 128 x 1024
// 12.1. Of more rows a cluster's groups would take several in turn (192 x 1024 on the device:
// 7.7 against 5.6 us).
struct BackwardGrid {
  int blocks, cluster;
};
BackwardGrid backward_grid(int64_t T, int d, nmoe_dtype dt, int sm_count) {
  const int groups =
      kBwdWarps / (dt == NMOE_F32 ? warps_per_row<float>(d) : warps_per_row<__nv_bfloat16>(d));
  const int64_t blocks = ceil_div(T, groups);
  if (blocks <= 8) return {(int)blocks, (int)blocks};
  return {(int)(blocks < sm_count ? blocks : sm_count), 1};
}
}  // namespace

int rms_norm_backward_parts(int64_t T, int d, nmoe_dtype dt, int sm_count) {
  const BackwardGrid g = backward_grid(T, d, dt, sm_count);
  return g.cluster > 1 ? 1 : g.blocks;
}

cudaError_t launch_rms_norm_backward(const void* dy, const void* h, const float* rstd,
                                     const void* weight, const void* dh, int64_t T, int d,
                                     nmoe_dtype dt, void* dx, float* dweight, float* partial,
                                     unsigned* err, int sm_count, cudaStream_t st) {
  const BackwardGrid g = backward_grid(T, d, dt, sm_count);
  const bool direct = g.cluster > 1 || g.blocks == 1;
  float* to = !dweight ? nullptr : direct ? dweight : partial;
  const int cluster = dweight ? g.cluster : 1;
  cudaError_t e = dt == NMOE_F32
                      ? launch_bwd_of<float>(dy, h, rstd, weight, dh, T, d, dx, to, g.blocks,
                                             cluster, err, st)
                      : launch_bwd_of<__nv_bfloat16>(dy, h, rstd, weight, dh, T, d, dx, to,
                                                     g.blocks, cluster, err, st);
  if (e == cudaSuccess && dweight && !direct)
    e = launch_sum_parts(partial, g.blocks, d, dweight, st);
  return e;
}

cudaError_t launch_sum_parts(const float* partial, int parts, int d, float* out,
                             cudaStream_t st) {
  return launch_kernel(sum_parts_kernel, dim3((unsigned)ceil_div(d, 32)), dim3(1024), 0, st, true,
                       1, partial, parts, d, out);
}

}  // namespace nmoe
