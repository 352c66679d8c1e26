// Dense matrix products with their epilogue: out = act(x W + bias) + residual in bf16 and
// e4m3, and the two products of the gradient, on the fifth-generation tensor cores.
//
// One operand pair (P: `rows` of the output, Q: `cols` of it, contracted over k) covers all
// of them: each operand is stored either with k innermost (K-major) or with its rows or
// columns innermost (MN-major), and TMA boxes and MMA descriptors take both, so no operand
// is ever transposed in memory:
//   x W         P = x [M, K] K-major         Q = W [K, N] MN-major
//   x8 w8^T     P = x8 [M, K] K-major        Q = w8 [N, K] K-major
//   dz W^T      P = dz [M, N] K-major        Q = W [K, N] K-major
//   x^T dz      P = x [M, K] MN-major        Q = dz [M, N] MN-major
// Every k-block is 128 bytes of k (64 bf16, 128 e4m3) in the 128-byte swizzle; partial
// tiles are zero-filled by TMA and not stored.
//
// Two kernels share the epilogue's arithmetic:
//   linear_pair_kernel  256 x 256 tiles on 2-CTA clusters, persistent, two accumulators:
//                       the tensor-bound sizes;
//   linear_tile_kernel  128 x 16..128 tiles of one CTA with the contraction split over a
//                       cluster: the sizes with too few 256 x 256 tiles to fill the SMs.
//                       With few output rows the operands change places (the 128 rows of
//                       the MMA are output columns, the rows its N), so a one-row product
//                       streams W at full tile height.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>

#include "block_ops.cuh"
#include "sm100_ptx.cuh"

namespace nmoe {

namespace {

using namespace ptx;

constexpr int kRowBytes = 128;             // bytes of k in a k-block
constexpr int kTile128 = 128 * kRowBytes;  // 128 rows (or columns) of a k-block: 16 KB
constexpr int kBox64 = 64 * kRowBytes;     // 64 of them: 8 KB
constexpr uint64_t kDrainNs = 20000000ull; // 20 ms for the issued MMAs after an abort
constexpr size_t kMaxSmem = 232448;

// ---- epilogue -----------------------------------------------------------------------------

struct Epi {
  const float* row_scale;            // e4m3: [rows]
  const float* col_scale;            // e4m3: [cols]
  const __nv_bfloat16* bias;         // [cols] or NULL
  const __nv_bfloat16* residual;     // [rows, cols] or NULL
  __nv_bfloat16* preact;             // [rows, cols] or NULL
  void* out;                         // [rows, cols]
  int64_t rows;
  int cols;
  int act;
  int out_f32;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The activations of n values at a time, one step of all of them after the other: an
// epilogue has two warps a scheduler, so the steps of one value alone would leave most
// issue slots waiting for the step before. Exponentials and reciprocals are the fast ones, off
// by 2 and 1 ulp. An exponential's argument is rounded like any product, which moves a value
// far out on a tail as much as a step or two of z would: SiLU is off by up to (2 |z| + 8) 2^-24
// of its value, the tanh form by 8 (|2u| + 1) 2^-24, the erf form by 9 (z^2 / 2 + 6) 2^-24 and
// its fit's 1.2e-7. bf16 outputs are rounded by up to 2^-8; fp32 outputs show it. An exponential or
// logistic function below 2^-126 counts as 0.

// s = 1 / (1 + e^-t), the logistic function; with z (1 + tanh u) / 2 = z / (1 + e^-2u) it
// serves both smooth activations
template <int kN>
__device__ __forceinline__ void logistic(const float (&t)[kN], float (&s)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) s[i] = ptx::ex2_approx(-kLog2e * t[i]);
#pragma unroll
  for (int i = 0; i < kN; ++i) s[i] = ptx::rcp_approx(1.f + s[i]);
}

// 2u of the tanh form
__device__ __forceinline__ float gelu_argument(float z) {
  return z * fmaf(2.f * kSqrt2OverPi * kGeluCubic * z, z, 2.f * kSqrt2OverPi);
}

// The normal distribution function, erfc(-z / sqrt 2) / 2, by the Chebyshev fit of erfc in
// Press et al., Numerical Recipes (2nd ed., section 6.2): relative error below 1.2e-7
// before fp32's own roundings, on both tails, in half of erfcf's instructions.
template <int kN>
__device__ __forceinline__ void normal_cdfs(const float* z, float (&cdf)[kN]) {
  constexpr float c[9] = {-0.82215223f, 1.48851587f, -1.13520398f, 0.27886807f, -0.18628806f,
                          0.09678418f,  0.37409196f, 1.00002368f,  -1.26551223f};
  float x[kN], t[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = kSqrtHalf * fabsf(z[i]);
#pragma unroll
  for (int i = 0; i < kN; ++i) t[i] = ptx::rcp_approx(fmaf(0.5f, x[i], 1.f));
#pragma unroll
  for (int i = 0; i < kN; ++i) cdf[i] = 0.17087277f;
#pragma unroll
  for (int k = 0; k < 9; ++k)
#pragma unroll
    for (int i = 0; i < kN; ++i) cdf[i] = fmaf(t[i], cdf[i], c[k]);
#pragma unroll
  for (int i = 0; i < kN; ++i) cdf[i] = ptx::ex2_approx(kLog2e * fmaf(-x[i], x[i], cdf[i]));
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float tail = 0.5f * t[i] * cdf[i];
    cdf[i] = z[i] < 0.f ? tail : 1.f - tail;
  }
}

// act of n values (a multiple of 4)
template <int kN>
__device__ __forceinline__ void activate(float (&v)[kN], int act) {
  constexpr int kG = kN < 8 ? kN : 8;
  float t[kG], s[kG];
  switch (act) {
    case NMOE_ACT_SILU:
#pragma unroll
      for (int g = 0; g < kN; g += kG) {
#pragma unroll
        for (int i = 0; i < kG; ++i) t[i] = v[g + i];
        logistic(t, s);
#pragma unroll
        for (int i = 0; i < kG; ++i) v[g + i] *= s[i];
      }
      break;
    case NMOE_ACT_GELU:
#pragma unroll
      for (int g = 0; g < kN; g += kG) {
        normal_cdfs(v + g, s);
#pragma unroll
        for (int i = 0; i < kG; ++i) v[g + i] *= s[i];
      }
      break;
    case NMOE_ACT_GELU_TANH:
#pragma unroll
      for (int g = 0; g < kN; g += kG) {
#pragma unroll
        for (int i = 0; i < kG; ++i) t[i] = gelu_argument(v[g + i]);
        logistic(t, s);
#pragma unroll
        for (int i = 0; i < kG; ++i) v[g + i] *= s[i];
      }
      break;
    default: break;
  }
}

// d[i] *= act'(z[i]) of n values. |z| is held to 100, where every slope is 0 or 1 to fp32 and
// the formulas' factors are still finite (a NaN stays one).
template <int kN>
__device__ __forceinline__ void scale_by_slopes(float (&d)[kN], float (&z)[kN], int act) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
    asm("max.NaN.f32 %0, %0, 0fC2C80000;\n min.NaN.f32 %0, %0, 0f42C80000;" : "+f"(z[i]));
  float s[kN], t[kN];
  switch (act) {
    case NMOE_ACT_SILU:
      logistic(z, s);
#pragma unroll
      for (int i = 0; i < kN; ++i) d[i] *= s[i] * fmaf(z[i], 1.f - s[i], 1.f);
      break;
    case NMOE_ACT_GELU:
      normal_cdfs(z, s);
#pragma unroll
      for (int i = 0; i < kN; ++i) t[i] = ptx::ex2_approx(-0.5f * kLog2e * z[i] * z[i]);
#pragma unroll
      for (int i = 0; i < kN; ++i) d[i] *= fmaf(kInvSqrt2Pi * z[i], t[i], s[i]);
      break;
    case NMOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < kN; ++i) t[i] = gelu_argument(z[i]);
      logistic(t, s);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float du = fmaf(6.f * kSqrt2OverPi * kGeluCubic * z[i], z[i], 2.f * kSqrt2OverPi);
        d[i] *= fmaf(z[i] * s[i] * (1.f - s[i]), du, s[i]);
      }
      break;
    default: break;
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void unpack4(uint2 v, float* f) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The residual's values at (row, col .. col+3), or zeros.
__device__ __forceinline__ uint2 residual4(const Epi& e, int64_t row, int col) {
  if (!e.residual || row >= e.rows || col >= e.cols) return make_uint2(0, 0);
  return *reinterpret_cast<const uint2*>(e.residual + row * e.cols + col);
}

__device__ __forceinline__ float4 abs4(float4 v) {
  return make_float4(fabsf(v.x), fabsf(v.y), fabsf(v.z), fabsf(v.w));
}
__device__ __forceinline__ float min4(float4 v) {
  return fminf(fminf(v.x, v.y), fminf(v.z, v.w));
}
__device__ __forceinline__ float max4(float4 v) {
  return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
}

// What the epilogue adds or multiplies in columns col .. col+3 (inside the output), as
// loaded and as used.
struct RawTerms {
  uint2 bias;
  float4 scale;
};
struct ColTerms {
  float bias[4], scale[4];
  float lo, hi;  // the scales' least and largest magnitude
};
template <bool F8>
__device__ __forceinline__ RawTerms raw_terms(const Epi& e, int col) {
  RawTerms t;
  if (col >= e.cols) col = 0;  // a lane outside the output: its terms are not used
  t.bias = e.bias ? *reinterpret_cast<const uint2*>(e.bias + col) : make_uint2(0, 0);
  t.scale = F8 ? *reinterpret_cast<const float4*>(e.col_scale + col) : make_float4(1, 1, 1, 1);
  return t;
}
template <bool F8>
__device__ __forceinline__ ColTerms column_terms(const RawTerms& r) {
  ColTerms t;
  unpack4(r.bias, t.bias);
  t.scale[0] = r.scale.x; t.scale[1] = r.scale.y; t.scale[2] = r.scale.z; t.scale[3] = r.scale.w;
  t.lo = min4(abs4(r.scale));
  t.hi = max4(abs4(r.scale));
  return t;
}

// What an epilogue has to do. The code of what it has not is left out: it cost small products
// 0.4 us of 3.1 (4 x 1032 x 56), most of it registers that kept the next launch off the SM.
enum EpiKind {
  kPlain,   // bf16 out, nothing added
  kAffine,  // scales, bias, residual, either type
  kAny      // activations and pre-activations too
};

// An accumulator times x_scale w_scale. One product of the scales serves as long as all of a
// thread's or warp's are normal numbers. Where both are small or both large, their product may
// leave fp32 though the result does not: they are then applied one after the other (the first
// step is no further out than the result; of a small and a large one the product lies between).
// That test is one a row and four columns, or one a tile and warp: one a value made pairs of
// 8192 x 256 x 2048 28 us, not 18.
__device__ __forceinline__ bool scales_fit(float row_lo, float row_hi, float col_lo,
                                           float col_hi) {
  return row_lo * col_lo >= 1.17549435e-38f && row_hi * col_hi <= 3.4028235e38f;
}
// The same over a warp's rows (one a lane) and columns (four a lane); the order of positive
// floats is that of their bits.
__device__ __forceinline__ bool warp_scales_fit(float row, float4 cols) {
  constexpr uint32_t kAll = 0xffffffffu;
  const float4 c = abs4(cols);
  const uint32_t r = __float_as_uint(fabsf(row));
  return scales_fit(__uint_as_float(__reduce_min_sync(kAll, r)),
                    __uint_as_float(__reduce_max_sync(kAll, r)),
                    __uint_as_float(__reduce_min_sync(kAll, __float_as_uint(min4(c)))),
                    __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(max4(c)))));
}

// Finishes the fp32 accumulators of R rows row0, row0 + step, ... and columns col .. col+3,
// and stores those below `rows` and inside the output. Everything read is passed in: a load
// behind the store of the row before would wait for its own round trip.
template <bool F8, EpiKind KIND, int R>
__device__ __forceinline__ void finish(const Epi& e, float (&v)[4 * R], const uint2 (&res)[R],
                                       const float (&row_scale)[R], const ColTerms& t,
                                       int64_t row0, int step, int64_t rows, int col) {
  const bool inside = col < e.cols;
  if constexpr (KIND != kPlain) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float rs = row_scale[i];
      if (F8 && !scales_fit(fabsf(rs), fabsf(rs), t.lo, t.hi)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = v[4 * i + j] * rs * t.scale[j] + t.bias[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[4 * i + j] = F8 ? fmaf(v[4 * i + j], rs * t.scale[j], t.bias[j])
                            : v[4 * i + j] + t.bias[j];
      }
    }
    if (KIND == kAny && e.preact) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (inside && row0 + step * i < rows)
          *reinterpret_cast<uint2*>(e.preact + (row0 + step * i) * e.cols + col) = make_uint2(
              pack2(v[4 * i], v[4 * i + 1]), pack2(v[4 * i + 2], v[4 * i + 3]));
    }
    if constexpr (KIND == kAny) activate(v, e.act);
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float r[4];
        unpack4(res[i], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] += r[j];
      }
    }
  }
  if (KIND != kPlain && e.out_f32) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (inside && row0 + step * i < rows)
        *reinterpret_cast<float4*>(static_cast<float*>(e.out) + (row0 + step * i) * e.cols + col) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (inside && row0 + step * i < rows)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(e.out) +
                                  (row0 + step * i) * e.cols + col) =
            make_uint2(pack2(v[4 * i], v[4 * i + 1]), pack2(v[4 * i + 2], v[4 * i + 3]));
  }
}

// The residual's 32 values at (row, col ..), zeros outside the output (its width is a
// multiple of 8, so a 16-byte piece is inside or outside as a whole).
__device__ __forceinline__ void load_residual32(const Epi& e, int64_t row, int col,
                                                uint4 (&r)[4]) {
  const uint4* at = reinterpret_cast<const uint4*>(e.residual + row * e.cols + col);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = e.residual && row < e.rows && col + 8 * i < e.cols ? at[i] : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void add_residual32(float (&v)[32], const uint4 (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    unpack4(make_uint2(r[i].x, r[i].y), f);
    unpack4(make_uint2(r[i].z, r[i].w), f + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * i + j] += f[j];
  }
}

// Scales (e4m3) and bias for a round's 32 columns from col on. The bias comes from the lanes
// that hold it: lane l has columns 4 l .. 4 l + 3 of the warp's 128, loaded before the
// accumulator was ready (from memory it would cost each round a trip to L2: the ring leaves
// no L1; 8192 x 64 x 2048 14.4 -> 13.6 us). The scales stay loads, the same addresses for
// the whole warp: as shuffles, four times as many, they cost more than the trip (8192 x 2048
// x 2048 with SiLU 30.4 -> 33.8 us).
template <bool F8>
__device__ __forceinline__ void add_bias32(const Epi& e, uint2 bias, float (&v)[32],
                                           float row_scale, bool fit, int col, int round) {
  if (F8 && !fit) {
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {
      float s = 1.f;
      if (col + j < e.cols) s = e.col_scale[col + j];
      // (a loop over registers would spill them: every value is scaled where it is the j-th)
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = i == j ? v[i] * row_scale * s : v[i];
    }
  } else if (F8) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float4 s = make_float4(1, 1, 1, 1);
      if (col + 4 * g < e.cols) s = *reinterpret_cast<const float4*>(e.col_scale + col + 4 * g);
      v[4 * g] *= row_scale * s.x;
      v[4 * g + 1] *= row_scale * s.y;
      v[4 * g + 2] *= row_scale * s.z;
      v[4 * g + 3] *= row_scale * s.w;
    }
  }
  if (e.bias) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int from = 8 * round + g;
      float b[4];
      unpack4(make_uint2(__shfl_sync(0xffffffffu, bias.x, from),
                         __shfl_sync(0xffffffffu, bias.y, from)), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * g + i] += b[i];
    }
  }
}

// A row's 32 values to (row, col ..), as far as they are inside the output.
__device__ __forceinline__ void store_row32(void* out, bool f32, const float (&v)[32],
                                            int64_t row, int64_t rows, int col, int cols) {
  if (row >= rows) return;
  if (f32) {
    float* const at = static_cast<float*>(out) + row * cols + col;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + 4 * k < cols)
        *reinterpret_cast<float4*>(at + 4 * k) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else {
    __nv_bfloat16* const at = static_cast<__nv_bfloat16*>(out) + row * cols + col;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + 8 * k < cols)
        *reinterpret_cast<uint4*>(at + 8 * k) = make_uint4(
            pack2(v[8 * k], v[8 * k + 1]), pack2(v[8 * k + 2], v[8 * k + 3]),
            pack2(v[8 * k + 4], v[8 * k + 5]), pack2(v[8 * k + 6], v[8 * k + 7]));
  }
}

// ---- copies -------------------------------------------------------------------------------

// How rows or columns of an operand are copied: in one box of k-innermost rows; in one box
// of 64-wide pieces, through a map with the pieces as a third dimension (its extent a
// multiple of 64); or piece by piece.
enum Layout { kKMajor = 0, kMnPieces = 1, kMnOneBox = 2 };

// One k-block of an operand from `at` on (in 1 or 2 pieces of 64 if MN-major), counted on
// this CTA's barrier, or with PAIR on the leader's at the same offset.
template <bool PAIR>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                             int mode, int at, int k0, int pieces) {
  const uint32_t leader = PAIR ? mapa_shared(bar, 0) : 0u;
  auto load2 = [&](uint8_t* to, int c0, int c1) {
    if (PAIR) tma_load_2d_pair(to, map, leader, c0, c1);
    else tma_load_2d(to, map, bar, c0, c1);
  };
  if (mode == kKMajor) {
    load2(dst, k0, at);
  } else if (mode == kMnOneBox) {
    if (PAIR) tma_load_3d_pair(dst, map, leader, 0, k0, at >> 6);
    else tma_load_3d(dst, map, bar, 0, k0, at >> 6);
  } else {
    load2(dst, at, k0);
    if (pieces == 2) load2(dst + kBox64, at + 64, k0);
  }
}

// ---- gradient of the epilogue ---------------------------------------------------------------
//
// dz = dy act'(z) and its column sums, bound by HBM (two arrays in, one out). A block takes
// 64 columns, a whole 128-byte line a row, and a share of the rows; a thread owns eight
// columns, so the sums stay in registers (fp32) until the block's partial row. Up to
// kDzClusterRows rows the shares of 64 columns are one cluster, whose first block adds the
// partial rows (2001 x 64: 4 us less than with a second launch for it).
constexpr int kDzThreads = 256;
constexpr int kDzCols = 8;                          // columns a thread
constexpr int kDzWide = 8;                          // threads across
constexpr int kDzRows = kDzThreads / kDzWide;       // rows a pass of the block
constexpr int kDzBatch = 4;                         // rows a thread has in flight: two arrays'
constexpr int kDzSumBatch = 8;                      // or one's, for the sums alone
constexpr int kDzClusterRows = 4096;

// cta = 64-column block * parts + part; FINAL: the parts are a cluster, `sums` is [N], else
// [parts, N].
struct DzShared {
  float sum[kDzThreads / 32][kDzWide * kDzCols];
};
template <bool FINAL, int BATCH>
__device__ __forceinline__ void dz_rows(const __nv_bfloat16* dy, const __nv_bfloat16* pre,
                                        int64_t M, int N, int act, int cta, int parts,
                                        __nv_bfloat16* dz, float* sums, DzShared& shared) {
  auto& sh = shared.sum;
  const int part = cta % parts, block = cta / parts;
  const int tx = threadIdx.x % kDzWide, ty = threadIdx.x / kDzWide;
  const int col = (block * kDzWide + tx) * kDzCols;
  float sum[kDzCols];
#pragma unroll
  for (int j = 0; j < kDzCols; ++j) sum[j] = 0.f;
  if (col < N) {
    const int64_t step = (int64_t)parts * kDzRows;
    for (int64_t r0 = (int64_t)part * kDzRows + ty; r0 < M; r0 += BATCH * step) {
      // a batch's loads are all in flight before the first of its stores
      uint4 v[BATCH], w[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int64_t at = (r0 + b * step) * N + col;
        v[b] = w[b] = make_uint4(0, 0, 0, 0);
        if (r0 + b * step < M) {
          v[b] = load_once(reinterpret_cast<const uint4*>(dy + at));
          if (pre) w[b] = load_once(reinterpret_cast<const uint4*>(pre + at));
        }
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (r0 + b * step >= M) continue;
        float d[kDzCols];
        unpack4(make_uint2(v[b].x, v[b].y), d);
        unpack4(make_uint2(v[b].z, v[b].w), d + 4);
        if (pre) {
          float z[kDzCols];
          unpack4(make_uint2(w[b].x, w[b].y), z);
          unpack4(make_uint2(w[b].z, w[b].w), z + 4);
          scale_by_slopes(d, z, act);
          if (dz)
            *reinterpret_cast<uint4*>(dz + (r0 + b * step) * N + col) =
                make_uint4(pack2(d[0], d[1]), pack2(d[2], d[3]), pack2(d[4], d[5]),
                           pack2(d[6], d[7]));
        }
#pragma unroll
        for (int j = 0; j < kDzCols; ++j) sum[j] += d[j];
      }
    }
  }
  if (!sums) return;  // the same for every thread of the grid
  // the four rows of a warp, then the warps in order, then the cluster's blocks in order
#pragma unroll
  for (int j = 0; j < kDzCols; ++j) {
    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
  }
  if ((threadIdx.x & 31) < kDzWide) {
#pragma unroll
    for (int j = 0; j < kDzCols; ++j) sh[threadIdx.x >> 5][tx * kDzCols + j] = sum[j];
  }
  __syncthreads();
  const int c = block * kDzWide * kDzCols + threadIdx.x;
  const bool mine = threadIdx.x < kDzWide * kDzCols && c < N;
  float s = 0.f;
  if (mine) {
#pragma unroll
    for (int i = 0; i < kDzThreads / 32; ++i) s += sh[i][threadIdx.x];
    if (FINAL) sh[0][threadIdx.x] = s;  // (read by this thread only until the cluster's barrier)
    else sums[(int64_t)part * N + c] = s;
  }
  if constexpr (FINAL) {
    __syncwarp();  // (the cluster barrier wants converged warps)
    if (parts > 1) cluster_sync_all();
    if (part == 0 && mine) {
      for (int o = 1; o < parts; ++o)
        s += ld_cluster_f(mapa_shared(&sh[0][threadIdx.x], (uint32_t)o));
      sums[c] = s;
    }
    __syncwarp();
    if (parts > 1) cluster_sync_all();  // no block still reads this one's sums
  }
}

// Three blocks an SM (80 registers): 8192 x 2048 with SiLU takes 20.3 us, with two 26.7.
template <bool FINAL>
__global__ void __launch_bounds__(kDzThreads, 3)
linear_dz_kernel(const __nv_bfloat16* dy, const __nv_bfloat16* pre, int64_t M, int N, int act,
                 int parts, __nv_bfloat16* dz, float* sums) {
  __shared__ DzShared shared;
  pdl_wait();
  pdl_launch_dependents();
  dz_rows<FINAL, kDzBatch>(dy, pre, M, N, act, blockIdx.x, parts, dz, sums, shared);
}

// ---- one-CTA tiles, split contraction -------------------------------------------------------

constexpr int kTileThreads = 256;
constexpr int kMaxStages = 8;
// 96 KB of stages: two CTAs share an SM, so that one's epilogue runs under the other's MMAs
// and clusters of eight find room. Over 182 timed products, the fastest variant with 96 KB
// took 0.2% more than the fastest of all (3% at most), with 192 KB 2.3% (30% at most).
constexpr int kTileRing = 98304;
// Where there are no more CTAs than SMs, alone or in twos, and each has several turns of that
// ring to go, the copies' latency paces it: 384 x 2816 x 1536 in 72 tiles 14.6 us, with twice
// the ring 13.4; as pairs of 128 columns 12.7 and 11.9. Clusters of four lose by it (25 to 17
// us: they wait for four empty SMs of a group).
constexpr int kTileLongRing = 196608;
constexpr int kLongRingTurns = 3;
int tile_stages(int bn, bool long_ring) {
  const int n = (long_ring ? kTileLongRing : kTileRing) / (kTile128 + bn * kRowBytes);
  return n < kMaxStages ? n : kMaxStages;
}
bool takes_long_ring(int64_t tiles, int64_t nk, int bn, int split, int sm_count) {
  return split <= 2 && tiles * split <= sm_count - 8 &&
         nk >= (int64_t)split * kLongRingTurns * tile_stages(bn, false);
}

struct TileParams {
  Epi epi;
  int nk;        // k-blocks
  int k_elems;   // k elements of a k-block
  int bn;        // the MMA's N: 16, 32, 64 or 128
  int a_mode;    // Layout of the 128-row operand's copies, and of the other's
  int b_mode;
  int tiles_a;   // tiles along the 128-row side
  int tiles;
  int split;     // CTAs of a cluster, each a part of the k-blocks: 2^split_log2
  int split_log2;
  int stages;
};
// One product, or two in one launch (a gradient's): a product's CTAs start at `begin`. Their
// clusters are of one size, and a product whose `split` is 1 takes one for that many tiles.
// dx and dW of 2001 x 1032 x 64 take 8.9 us so, 11.1 behind one another. Beside two products
// sum_ctas CTAs, a cluster 64 columns, may add up the columns of dz (8.9 us with dbias too;
// behind a launch for it 14.2).
template <int NP>
struct TileArgs {
  CUtensorMap a[NP], b[NP];
  TileParams prob[NP];
  int begin[NP];
  int sum_begin, sum_ctas;  // (before or behind the products' CTAs)
  int cluster;
  const __nv_bfloat16* dz;  // [dz_rows, dz_cols]
  float* sums;
  int64_t dz_rows;
  int dz_cols;
  unsigned* err;
  uint64_t wait_ns;
};

// The two producer warps' barrier.
__device__ __forceinline__ void producers_meet() { asm volatile("bar.sync 1, 64;" ::: "memory"); }

// SWAP: the MMA's 128 rows are output columns and its bn columns output rows.
template <bool F8, bool SWAP, int NP, EpiKind KIND>
__global__ void __launch_bounds__(kTileThreads, 2)
linear_tile_kernel(const __grid_constant__ TileArgs<NP> args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (NP > 1) {
    const int at = (int)blockIdx.x - args.sum_begin;
    if (at >= 0 && at < args.sum_ctas) {
      __shared__ DzShared shared;
      pdl_wait();
      pdl_launch_dependents();
      dz_rows<true, kDzSumBatch>(args.dz, nullptr, args.dz_rows, args.dz_cols, NMOE_ACT_NONE,
                                 at, args.cluster, nullptr, args.sums, shared);
      return;
    }
  }
  const int which = NP > 1 && (int)blockIdx.x >= args.begin[NP - 1] ? NP - 1 : 0;
  const TileParams& p = args.prob[which];
  const CUtensorMap& map_a = args.a[which];
  const CUtensorMap& map_b = args.b[which];
  const uint64_t wait_ns = args.wait_ns;
  const int block = (int)blockIdx.x - (NP > 1 ? args.begin[which] : 0);
  const int tile = block >> p.split_log2, rank = block & (p.split - 1);
  if (NP > 1 && tile >= p.tiles) return;  // fills up a cluster of single tiles
  const int ta = tile % p.tiles_a, tb = tile / p.tiles_a;
  const int kb0 = (p.nk * rank) >> p.split_log2;  // (nk <= 2^24)
  const int kb1 = (p.nk * (rank + 1)) >> p.split_log2;
  const int b_bytes = p.bn * kRowBytes;
  const int stage_bytes = kTile128 + b_bytes;
  const uint32_t tmem_cols = p.bn < 32 ? 32u : (uint32_t)p.bn;  // 128 at most (tmem_alone)

  // One k-block's copies, each operand's by one thread (the first one's announces both).
  auto fetch_a = [&](int kb, int stage) {
    mbar_arrive_expect_tx(&full_bar[stage], (uint32_t)stage_bytes);
    load_operand<false>(smem + stage * stage_bytes, &map_a, &full_bar[stage], p.a_mode, ta * 128,
                        kb * p.k_elems, 2);
  };
  auto fetch_b = [&](int kb, int stage) {
    load_operand<false>(smem + stage * stage_bytes + kTile128, &map_b, &full_bar[stage],
                        p.b_mode, tb * p.bn, kb * p.k_elems, p.bn / 64);
  };
  const int ahead = kb1 - kb0 < p.stages ? kb1 - kb0 : p.stages;  // the first turn of the ring
  if (warp == 0) {
    // The barriers and the first turn's copies, here and in warp 2, need nothing of the other
    // warps: they go out while TMEM is allocated (1000 cycles).
    const bool issue = elect_one();
    if (issue) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(&full_bar[i], 1);
        mbar_init(&empty_bar[i], 1);
      }
      mbar_init(&done_bar, 1);
      abort_flag = 0;
      fence_mbar_init();
    }
    producers_meet();
    pdl_wait();
    if (issue)
      for (int i = 0; i < ahead; ++i) fetch_a(kb0 + i, i);
    __syncwarp();
  } else if (warp == 2) {
    const bool issue = elect_one();
    producers_meet();
    pdl_wait();
    if (issue)
      for (int i = 0; i < ahead; ++i) fetch_b(kb0 + i, i);
    __syncwarp();
  } else {
    if (warp == 1) tmem_alloc(&tmem_base_sh, tmem_cols);
    pdl_wait();
  }

  // What the epilogue reads first is asked for now: after the MMAs it would cost two round
  // trips to L2. A whole tile is finished from TMEM: a lane has a row, a warp half of the
  // columns, 32 at a time. Parts of one, and swapped tiles, go through shared memory.
  const bool whole = !SWAP && p.split == 1;
  const int q = warp & 3;
  const int64_t lane_row = (int64_t)ta * 128 + q * 32 + lane;
  const int rounds = p.bn / 64, col0 = tb * p.bn + (warp >> 2) * 32 * rounds;
  uint4 res32[4];
  float rs32 = 1.f;
  constexpr int kRows = SWAP ? 2 : 4;               // rows a thread finishes at a time
  const int64_t row0 = SWAP ? (int64_t)tb * p.bn : (int64_t)ta * 128;
  const int per_row = (SWAP ? 128 : p.bn) / 4;      // threads across: 16 or 32
  const int mine = (SWAP ? p.bn : 128) >> p.split_log2;   // this CTA's rows of the tile
  const int down = kTileThreads / per_row;          // rows a pass of the block: 16 or 8
  const int c = (threadIdx.x % per_row) * 4, col = (SWAP ? ta * 128 : tb * p.bn) + c;
  const int64_t first = row0 + rank * mine;
  const int64_t rows = first + mine < p.epi.rows ? first + mine : p.epi.rows;
  uint2 res[kRows];
  float rs[kRows];
  auto ask = [&](int r) {  // rows first + r, + down, ...
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = first + r + i * down;
      res[i] = row < rows ? residual4(p.epi, row, col) : make_uint2(0, 0);
      rs[i] = F8 && row < rows ? p.epi.row_scale[row] : 1.f;
    }
  };
  RawTerms raw;
  if (KIND == kPlain) {
    raw = RawTerms();
    for (int i = 0; i < kRows; ++i) {
      res[i] = make_uint2(0, 0);
      rs[i] = 1.f;
    }
  } else if (whole) {
    raw = raw_terms<F8>(p.epi, col0 + 4 * lane);
    if (F8 && lane_row < p.epi.rows) rs32 = p.epi.row_scale[lane_row];
    load_residual32(p.epi, lane_row, col0, res32);
  } else {
    raw = raw_terms<F8>(p.epi, col);
    ask(threadIdx.x / per_row);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  volatile int* abort_v = &abort_flag;
  pdl_launch_dependents();  // after the TMEM allocation: a dependent's CTA may want its own

  // The producers' and the issuer's warps stay converged and one elected lane of each
  // issues: their operands are then in uniform registers. A k-block costs each warp a fixed
  // number of cycles, whatever the tile's width, and that paces small tiles: one producer an
  // operand, and the next stage's barrier is asked before this one's work goes out.
  if (warp == 0 || warp == 2) {
    // ---------------- TMA producers: from the second turn on ----------------
    const bool issue = elect_one();
    int stage = 0;
    uint32_t phase = 0;  // of the empty barriers' first flip
    bool ready = false;
    for (int kb = kb0 + ahead; kb < kb1; ++kb) {
      if (!__all_sync(0xffffffffu,
                      ready || ring_wait(&empty_bar[stage], phase, abort_v, wait_ns)))
        break;
      const int at = stage;
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
      ready = mbar_test_wait(&empty_bar[stage], phase);
      if (issue) {
        if (warp == 0) fetch_a(kb, at); else fetch_b(kb, at);
      }
      __syncwarp();
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const bool issue = elect_one();
    const int a_mn = p.a_mode != kKMajor, b_mn = p.b_mode != kKMajor;
    const uint32_t idesc = idesc_of(F8, 128, p.bn, a_mn, b_mn);
    // a 32-byte step of k: 32 bytes along a K-major row, 16 rows (2 KB) of an MN-major box
    const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
    const uint32_t a0 = sdesc_lo(smem_u32(smem), a_mn ? kBox64 : 16);
    const uint32_t b0 = sdesc_lo(smem_u32(smem) + kTile128, b_mn ? kBox64 : 16);
    int stage = 0;
    uint32_t phase = 0;
    bool ready = false;
    for (int kb = kb0; kb < kb1; ++kb) {
      // every lane has seen this phase before the commit below can start the next one
      if (!__all_sync(0xffffffffu,
                      ready || ring_wait(&full_bar[stage], phase, abort_v, wait_ns)))
        break;
      tc_fence_after();
      const uint32_t a = a0 + stage * (stage_bytes >> 4), b = b0 + stage * (stage_bytes >> 4);
      uint64_t* const done = &empty_bar[stage];
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
      ready = mbar_test_wait(&full_bar[stage], phase);
      if (issue) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = sdesc_words(a + kk * a_step), bd = sdesc_words(b + kk * b_step);
          if (F8)
            mma_e4m3(tmem_base, ad, bd, idesc, kb != kb0 || kk != 0);
          else
            mma_bf16(tmem_base, ad, bd, idesc, kb != kb0 || kk != 0);
        }
        mma_commit(done);
      }
      __syncwarp();
    }
    if (issue) mma_commit(&done_bar);
    __syncwarp();
  }

  // ---------------- every warp: accumulators to shared memory, in output order ----------
  // After an abort the MMAs issued so far still complete, in far less than kDrainNs.
  {
    int ok = 1;
    if (lane == 0) {
      ok = ring_wait(&done_bar, 0, abort_v, wait_ns);
      if (!ok) {
        int dummy = 0;
        mbar_wait(&done_bar, 0, &dummy, kDrainNs);
      }
    }
    __syncwarp();
  }
  tc_fence_after();
  __syncthreads();  // no wait is left that could still set the flag
  const bool aborted = *abort_v != 0;
  float* const acc = reinterpret_cast<float*>(smem);
  // + 4 floats a row: the 16-byte writes of a warp's 32 rows then meet every bank evenly
  const int ld = (SWAP ? 128 : p.bn) + 4;
  if (whole) {
    if (!aborted) {
      // (every copy was consumed by an MMA that has completed)
      const bool fit = !F8 || warp_scales_fit(rs32, raw.scale);
#pragma unroll 1
      for (int r = 0; r < rounds; ++r) {
        const int c32 = col0 + 32 * r;
        uint32_t y[32];
        tmem_ld32(tmem_base + ((uint32_t)(q * 32) << 16) + (warp >> 2) * 32 * rounds + 32 * r, y);
        tmem_ld_wait();
        if (c32 >= p.epi.cols || lane_row - lane >= p.epi.rows) continue;  // the whole warp
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(y[i]);
        if constexpr (KIND != kPlain) add_bias32<F8>(p.epi, raw.bias, v, rs32, fit, c32, r);
        if constexpr (KIND == kAny) {
          if (p.epi.preact)
            store_row32(p.epi.preact, false, v, lane_row, p.epi.rows, c32, p.epi.cols);
          activate(v, p.epi.act);
        }
        if (KIND != kPlain && p.epi.residual) {
          add_residual32(v, res32);
          if (r + 1 < rounds) load_residual32(p.epi, lane_row, c32 + 32, res32);
        }
        store_row32(p.epi.out, KIND != kPlain && p.epi.out_f32 != 0, v, lane_row, p.epi.rows, c32,
                    p.epi.cols);
      }
      tc_fence_before();
    }
  } else if (!aborted) {
    // the ring is free: every copy was consumed by an MMA that has completed
    for (int c = (warp >> 2) * 16; c < p.bn; c += 32) {
      uint32_t v[16];
      tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + c, v);
      tmem_ld_wait();
      if (SWAP) {
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[(c + j) * ld + q * 32 + lane] = __uint_as_float(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(acc + (q * 32 + lane) * ld + c + j) =
              make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                          __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
      }
    }
    tc_fence_before();
  }
  __syncwarp();  // (the cluster barrier wants converged warps)
  if (p.split > 1) cluster_sync_all(); else __syncthreads();
  if (!aborted && !whole) {
    // this CTA's rows of the tile: the partial sums of the cluster's CTAs added in rank
    // order, so the result does not depend on which finished first
    const ColTerms terms = column_terms<F8>(raw);
    for (int r = threadIdx.x / per_row; first + r < rows; r += kRows * down) {
      float v[4 * kRows];
      for (int o = 0; o < p.split; ++o) {
        float4 f[kRows];  // in flight together: another CTA's memory is 250 cycles away
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          f[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          const float* const at = acc + (rank * mine + r + i * down) * ld + c;
          if (first + r + i * down < rows)
            f[i] = SWAP && p.split == 1 ? *reinterpret_cast<const float4*>(at)
                                        : ld_cluster_f4(mapa_shared(at, (uint32_t)o));
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          v[4 * i] = o == 0 ? f[i].x : v[4 * i] + f[i].x;
          v[4 * i + 1] = o == 0 ? f[i].y : v[4 * i + 1] + f[i].y;
          v[4 * i + 2] = o == 0 ? f[i].z : v[4 * i + 2] + f[i].z;
          v[4 * i + 3] = o == 0 ? f[i].w : v[4 * i + 3] + f[i].w;
        }
      }
      uint2 mine_res[kRows];
      float mine_rs[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        mine_res[i] = res[i];
        mine_rs[i] = rs[i];
      }
      if (KIND != kPlain && first + r + kRows * down < rows) ask(r + kRows * down);  // ahead of the stores
      finish<F8, KIND, kRows>(p.epi, v, mine_res, mine_rs, terms, first + r, down, rows, col);
    }
  }
  if (aborted) {
    if (threadIdx.x == 0) atomicOr(args.err, kErrTimeout);
    // give the copies in flight time to land before the shared memory is released
    const uint64_t t0 = globaltimer_ns();
    while ((int64_t)(globaltimer_ns() - t0) < 1000000) {
    }
  }
  __syncwarp();
  if (p.split > 1) cluster_sync_all(); else __syncthreads();  // no CTA still reads this one's
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ---- 2-CTA clusters, 256 x 256 tiles --------------------------------------------------------
//
// A pair's two CTAs each stage 128 rows of P and half of the tile's columns of Q; the
// leader's one thread issues tcgen05.mma.cta_group::2 with M = 256. Six stages of 32 KB
// are in flight a CTA, and two 256-column accumulators let the epilogue of one tile run
// under the next tile's MMAs. A last wave that fills at most half of the pairs is cut
// into half-width tiles.
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 32 * (2 + kPairEpiWarps);
constexpr int kPairStageBytes = 2 * kTile128;
constexpr int kPairStages = 6;
constexpr int kPairEpiStage = 32 * 128;        // a warp's staging: 32 rows of 32 fp32 values,
constexpr int kPairEpiHalf = kPairEpiStage / 2;  // or two blocks of as many bf16
constexpr int kAccCols = 256;
constexpr size_t kPairSmem =
    (size_t)kPairStages * kPairStageBytes + kPairEpiWarps * kPairEpiStage + 1024;
static_assert(kPairSmem <= kMaxSmem, "dynamic shared memory beyond the 227 KB a CTA may use");
static_assert(tmem_alone(kPairSmem), "all TMEM columns beside another kernel's");

constexpr int kMaxPairs = 80;

struct PairProblem {
  Epi epi;
  int nk;
  int k_elems;
  int a_mode, b_mode;  // Layout of the copies
  int tiles_m, tiles_n;
  int num_full;    // tiles of 256 columns; the rest are two items of 128 each
  int num_items;
};
struct PairMaps {
  CUtensorMap a, b, b_half, out, pre;
};
// One product, or two in one launch (a gradient's): the pairs then share the first one's
// items in turn and take contiguous runs of the second's, pair i from first[i] on, that even
// out their work.
template <int NP>
struct PairArgs {
  PairMaps map[NP];
  PairProblem prob[NP];
  int first[NP > 1 ? kMaxPairs + 1 : 1];
  unsigned* err;
  uint64_t wait_ns;
};

// The i-th item of a pair: false behind its last.
struct Work {
  int prob, item;
};
template <int NP>
__device__ __forceinline__ bool work_at(const PairArgs<NP>& p, int pair, int npairs, int i,
                                        Work* w) {
  const int n0 = p.prob[0].num_items;
  w->prob = 0;
  w->item = pair + i * npairs;
  if (NP == 1 || w->item < n0) return w->item < n0;
  const int own = pair < n0 ? (n0 - pair + npairs - 1) / npairs : 0;
  w->prob = NP - 1;
  w->item = p.first[NP > 1 ? pair : 0] + i - own;
  return w->item < p.first[NP > 1 ? pair + 1 : 0];
}

// A warp's 32 rows of 32 values to the output behind `map`: rows of 64 bytes (bf16) in
// 64-byte swizzle, or of 128 bytes (fp32) in 128-byte swizzle, then one tiled store. The
// store that last used this block, the one before last or (alone) the last, has been read
// before it is written over.
__device__ __forceinline__ void store_rows32(const float (&v)[32], const CUtensorMap* map,
                                             uint8_t* block, bool f32, bool alone, int col,
                                             int row, int lane) {
  if (lane == 0) {
    if (alone) bulk_wait_read<0>(); else bulk_wait_read<1>();
  }
  __syncwarp();
  if (f32) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4*>(block + lane * 128 + ((k ^ (lane & 7)) << 4)) =
          make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(block + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = make_uint4(
          pack2(v[8 * k], v[8 * k + 1]), pack2(v[8 * k + 2], v[8 * k + 3]),
          pack2(v[8 * k + 4], v[8 * k + 5]), pack2(v[8 * k + 6], v[8 * k + 7]));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, block, col, row);
    bulk_commit();
  }
}

struct Item {
  int m, n0, half;  // row tile, first column, half width
};

// Eight row tiles a group, columns outermost in it: the pairs that run at one time share
// their rows and columns in L2.
__device__ __forceinline__ Item item_of(int item, const PairProblem& p) {
  int tile = item, sub = 0;
  Item it;
  it.half = item >= p.num_full;
  if (it.half) {
    sub = (item - p.num_full) & 1;
    tile = p.num_full + ((item - p.num_full) >> 1);
  }
  constexpr int kGroup = 8;
  const int per_group = kGroup * p.tiles_n;
  const int g = tile / per_group, in = tile % per_group;
  const int left = p.tiles_m - g * kGroup;
  const int height = left < kGroup ? left : kGroup;
  it.m = g * kGroup + in % height;
  it.n0 = (in / height) * 256 + sub * 128;
  return it;
}

template <bool F8, int NP, EpiKind KIND>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ PairArgs<NP> p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kPairStages], empty_bar[kPairStages];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the leader, which issues the MMAs
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  uint8_t* const epi_smem = smem + (size_t)kPairStages * kPairStageBytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full_bar[i], 1);  // the leader's producer, with both CTAs' bytes
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * kPairEpiWarps);
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < NP; ++i) {
      prefetch_tensormap(&p.map[i].a);
      prefetch_tensormap(&p.map[i].b);
      prefetch_tensormap(&p.map[i].b_half);
      prefetch_tensormap(&p.map[i].out);
    }
  }
  if (warp == 1) tmem_alloc_pair(&tmem_base_sh, 2 * kAccCols);
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers are initialised and the TMEM is allocated
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  volatile int* abort_v = &abort_flag;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    // The warp stays converged and one elected lane issues (uniform operands): a stage's
    // copies go out as one or two boxes an operand.
    const bool issue = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Work w;
    for (int i = 0; ok && work_at(p, pair, npairs, i, &w); ++i) {
      const PairProblem& g = p.prob[w.prob];
      const PairMaps& m = p.map[w.prob];
      const Item it = item_of(w.item, g);
      const int nbox = it.half ? 1 : 2;  // 64-column pieces of this CTA's half of Q
      const uint32_t bytes = 2u * (uint32_t)(kTile128 + nbox * kBox64);
      const int row = it.m * 256 + (int)rank * 128;
      const int col = it.n0 + (int)rank * nbox * 64;
      for (int kb = 0; kb < g.nk; ++kb) {
        ok = __all_sync(0xffffffffu,
                        ring_wait(&empty_bar[stage], phase ^ 1, abort_v, p.wait_ns));
        if (!ok) break;
        if (issue) {
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], bytes);
          uint8_t* a = smem + stage * kPairStageBytes;
          uint8_t* b = a + kTile128;
          const int k0 = kb * g.k_elems;
          load_operand<true>(a, &m.a, &full_bar[stage], g.a_mode, row, k0, 2);
          load_operand<true>(b, it.half ? &m.b_half : &m.b, &full_bar[stage], g.b_mode, col, k0,
                             nbox);
        }
        __syncwarp();
        if (++stage == kPairStages) { stage = 0; phase ^= 1; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (the leader's one warp) ----------------
    // The warp stays converged and one elected lane issues: the operands then live in
    // uniform registers, and a k-block's four MMAs go out faster than they run.
    if (rank == 0) {
      const bool issue = elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      Work w;
      for (int i = 0; ok && work_at(p, pair, npairs, i, &w); ++i) {
        const PairProblem& g = p.prob[w.prob];
        const int a_mn = g.a_mode != kKMajor, b_mn = g.b_mode != kKMajor;
        const uint32_t idesc = idesc_of(F8, 256, w.item >= g.num_full ? 128 : 256, a_mn, b_mn);
        const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        const uint32_t a0 = sdesc_lo(smem_u32(smem), a_mn ? kBox64 : 16);
        const uint32_t b0 = sdesc_lo(smem_u32(smem) + kTile128, b_mn ? kBox64 : 16);
        ok = __all_sync(0xffffffffu,
                        ring_wait(&tempty_bar[acc], acc_phase ^ 1, abort_v, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kAccCols;
        for (int kb = 0; kb < g.nk; ++kb) {
          ok = __all_sync(0xffffffffu, ring_wait(&full_bar[stage], phase, abort_v, p.wait_ns));
          // every lane has seen this phase before the commit below can start the next one
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = a0 + stage * (kPairStageBytes >> 4);
          const uint32_t b = b0 + stage * (kPairStageBytes >> 4);
          if (issue) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = sdesc_words(a + kk * a_step), bd = sdesc_words(b + kk * b_step);
              if (F8)
                mma_e4m3_pair(d_tmem, ad, bd, idesc, (kb | kk) != 0);
              else
                mma_bf16_pair(d_tmem, ad, bd, idesc, (kb | kk) != 0);
            }
            mma_commit_both(&empty_bar[stage]);
          }
          __syncwarp();
          if (++stage == kPairStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (issue) mma_commit_both(&tfull_bar[acc]);
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      // every MMA issued above has completed once drain_bar flips
      if (issue) mma_commit_pair(mapa_shared(&drain_bar, 0));
      __syncwarp();
      int dummy = 0;
      mbar_wait(&drain_bar, 0, &dummy, kDrainNs);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: eight warps a CTA, two a TMEM lane quarter ----------------
    // A lane takes one row, 32 columns a round; the finished values go through the warp's
    // two staging blocks (16-byte pieces rotated by the row, the copies' swizzle) and out by
    // tiled stores, which clip the tile to the output. The residual's pieces are asked for a
    // round ahead, the first round's before the accumulator is ready. (Staging the fp32
    // accumulators to store whole row pieces from registers moved four times these bytes
    // through the shared memory that feeds the MMAs: 1400 cycles a round without any
    // activation, where this takes 500.)
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;
    uint8_t* const stage0 = epi_smem + (warp - 2) * kPairEpiStage;
    int acc = 0, buf = 0;
    uint32_t acc_phase = 0;
    Work wk;
    for (int i = 0; work_at(p, pair, npairs, i, &wk); ++i) {
      const Epi& epi = p.prob[wk.prob].epi;
      const PairMaps& m = p.map[wk.prob];
      const Item it = item_of(wk.item, p.prob[wk.prob]);
      const bool one_block = epi.out_f32 != 0;  // an fp32 block takes both staging blocks
      const int rounds = it.half ? 2 : 4;
      const int col0 = it.n0 + part * rounds * 32;
      const int row_base = it.m * 256 + (int)rank * 128 + q * 32;
      const int64_t row = (int64_t)row_base + lane;
      const float rs = F8 && row < epi.rows ? epi.row_scale[row] : 1.f;
      const RawTerms raw = KIND != kPlain ? raw_terms<F8>(epi, col0 + 4 * lane) : RawTerms();
      uint4 res[4];
      if (KIND != kPlain) load_residual32(epi, row, col0, res);
      int w = 1;
      if (lane == 0) w = ring_wait(&tfull_bar[acc], acc_phase, abort_v, p.wait_ns);
      if (__shfl_sync(0xffffffffu, w, 0) == 0) break;
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + ((uint32_t)(q * 32) << 16) + acc * kAccCols + part * rounds * 32;
      const bool fit = !F8 || warp_scales_fit(rs, raw.scale);
#pragma unroll 1
      for (int r = 0; r < rounds; ++r) {
        const int col = col0 + 32 * r;
        uint32_t y[32];
        tmem_ld32(taddr + 32 * r, y);
        tmem_ld_wait();
        if (r + 1 == rounds) {  // the accumulator is read: the next tile's MMAs may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(&tempty_bar[acc], 0));
        }
        if (col >= epi.cols || row_base >= epi.rows) continue;  // the whole warp
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(y[i]);
        if constexpr (KIND != kPlain) add_bias32<F8>(epi, raw.bias, v, rs, fit, col, r);
        if constexpr (KIND == kAny) {
          if (epi.preact) {
            store_rows32(v, &m.pre, stage0 + buf * kPairEpiHalf, false, one_block, col, row_base,
                         lane);
            if (!one_block) buf ^= 1;
          }
          activate(v, epi.act);
        }
        if (KIND != kPlain && epi.residual) {
          add_residual32(v, res);
          if (r + 1 < rounds) load_residual32(epi, row, col + 32, res);
        }
        store_rows32(v, &m.out, stage0 + buf * kPairEpiHalf, one_block, one_block, col,
                     row_base, lane);
        if (!one_block) buf ^= 1;
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  __syncthreads();
  if (*abort_v) {
    // a wait ran out: give the copies this CTA issued (which complete on the leader's
    // barriers, out of this CTA's sight) time to land before the pair's final barrier
    const uint64_t t0 = globaltimer_ns();
    while ((int64_t)(globaltimer_ns() - t0) < 1000000) {
    }
  }
  cluster_sync_all();  // the other CTA no longer touches this CTA's barriers or TMEM
  if (threadIdx.x == 0 && abort_flag) atomicOr(p.err, kErrTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kAccCols);
  }
}

// ---- host side ----------------------------------------------------------------------------

// One operand: `extent` rows (or columns) of the output, k elements deep.
struct Operand {
  const void* base;
  int64_t extent;
  bool mn;  // extent innermost
};

struct Product {
  Operand p, q;  // output rows, output columns
  int64_t k;
  bool f8;
  Epi epi;
};

EpiKind epi_kind(const Product& g) {
  if (g.epi.act != NMOE_ACT_NONE || g.epi.preact) return kAny;
  return g.f8 || g.epi.bias || g.epi.residual || g.epi.out_f32 ? kAffine : kPlain;
}

// A tensor map; dims and box innermost first.
bool encode_map(CUtensorMap* m, const void* base, uint32_t rank, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box, CUtensorMapDataType type,
                CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  const uint32_t elem[3] = {1, 1, 1};
  return fn(m, type, rank, const_cast<void*>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
CUtensorMapDataType operand_type(bool f8) {
  return f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// The output's map for the pair kernel's stores: boxes of 32 x 32.
bool output_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, bool f32) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * (f32 ? 4 : 2)};
  const uint32_t box[2] = {32, 32};
  return encode_map(m, base, 2, dims, strides, box,
                    f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// An operand's map: boxes of 64 extent x 64 k (MN-major), or box_rows extent x 128 bytes
// of k (K-major).
bool operand_map(CUtensorMap* m, const Operand& o, int64_t k, bool f8, uint32_t box_rows) {
  const uint64_t es = f8 ? 1 : 2;
  uint64_t dims[2] = {(uint64_t)k, (uint64_t)o.extent};
  uint64_t strides[1] = {(uint64_t)k * es};
  uint32_t box[2] = {(uint32_t)(kRowBytes / es), box_rows};
  if (o.mn) {
    dims[0] = (uint64_t)o.extent;
    dims[1] = (uint64_t)k;
    strides[0] = (uint64_t)o.extent * es;
    box[0] = box[1] = 64;
  }
  return encode_map(m, o.base, 2, dims, strides, box, operand_type(f8));
}

// Pairs of SMs that can hold one pair CTA each at the same time, on the current device.
int pair_slots(int sm_count) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  constexpr int kDevices = 64;
  static std::mutex mu;
  static int slots[kDevices];  // + 1; 0: not asked yet
  if (dev >= kDevices) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (slots[dev] != 0) return slots[dev] - 1;
  int n = 0;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(linear_pair_kernel<false, 1, kAny>),
                                 kPairSmem);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count & ~1));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel<false, 1, kAny>, &cfg);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    n = 0;  // the one-CTA tiles run instead
  }
  if (n > kMaxPairs) n = kMaxPairs;
  slots[dev] = n + 1;
  return n;
}

// The map of an operand and the Layout that goes with it: box_rows rows or columns a copy, in
// one box where the operand allows it.
bool copy_map(CUtensorMap* m, int* mode, const Operand& o, int64_t k, bool f8,
              uint32_t box_rows) {
  if (!o.mn || o.extent % 64 != 0) {
    *mode = o.mn ? kMnPieces : kKMajor;
    return operand_map(m, o, k, f8, box_rows);
  }
  *mode = kMnOneBox;
  const uint64_t dims[3] = {64, (uint64_t)k, (uint64_t)o.extent / 64};
  const uint64_t strides[2] = {(uint64_t)o.extent * 2, 128};
  const uint32_t box[3] = {64, 64, box_rows / 64};
  return encode_map(m, o.base, 3, dims, strides, box, operand_type(f8));
}

// A product's part of a pair launch; `whole`: no half-width items.
bool pair_problem(const Product& g, int npairs, bool whole, PairProblem* p, PairMaps* m) {
  if (!copy_map(&m->a, &p->a_mode, g.p, g.k, g.f8, 128) ||
      !copy_map(&m->b, &p->b_mode, g.q, g.k, g.f8, 128) ||
      !output_map(&m->out, g.epi.out, g.epi.rows, g.epi.cols, g.epi.out_f32 != 0))
    return false;
  p->epi = g.epi;
  p->k_elems = g.f8 ? 128 : 64;
  p->nk = (int)ceil_div(g.k, p->k_elems);
  p->tiles_m = (int)ceil_div(g.p.extent, 256);
  p->tiles_n = (int)ceil_div(g.q.extent, 256);
  const int tiles = p->tiles_m * p->tiles_n;
  const int rest = tiles % npairs;
  p->num_full = !whole && rest > 0 && 2 * rest <= npairs ? tiles - rest : tiles;
  p->num_items = p->num_full + 2 * (tiles - p->num_full);
  m->pre = m->out;
  if (g.epi.preact && !output_map(&m->pre, g.epi.preact, g.epi.rows, g.epi.cols, false))
    return false;
  m->b_half = m->b;
  int mode;
  return p->num_items == tiles || copy_map(&m->b_half, &mode, g.q, g.k, g.f8, 64);
}

cudaError_t launch_pairs(const Product& g, int npairs, unsigned* err, cudaStream_t st) {
  PairArgs<1> a;
  if (!pair_problem(g, npairs, false, &a.prob[0], &a.map[0])) return cudaErrorInvalidValue;
  a.err = err;
  a.wait_ns = block_wait_ns();
  const int pairs = a.prob[0].num_items < npairs ? a.prob[0].num_items : npairs;
  const EpiKind kind = epi_kind(g);
  void (*kernel)(PairArgs<1>) = g.f8 ? (kind == kAny ? linear_pair_kernel<true, 1, kAny>
                                                     : linear_pair_kernel<true, 1, kAffine>)
                                : kind == kAny    ? linear_pair_kernel<false, 1, kAny>
                                : kind == kAffine ? linear_pair_kernel<false, 1, kAffine>
                                                  : linear_pair_kernel<false, 1, kPlain>;
  return launch_kernel(kernel, dim3((unsigned)(2 * pairs)), dim3(kPairThreads), kPairSmem, st,
                       true, 2, a);
}

// How a launch of two products shares its pairs: the first one's `tiles0` items of `nk0`
// k-blocks in turn, then the second's, filling up the pairs with the least work. first[i]
// (may be NULL) as in PairArgs; returns the most loaded pair's items and k-blocks.
struct PairLoad {
  int64_t items, k_blocks;
};
PairLoad share_pairs(int64_t tiles0, int64_t nk0, int64_t tiles1, int64_t nk1, int npairs,
                     int* first) {
  const int64_t base = tiles0 / npairs, more = tiles0 % npairs;  // `more` pairs have base + 1
  const int64_t low = npairs - more;
  // runs of the second: `fill` for a pair with less of the first, `even` for every pair, and
  // one each for the first `odd` pairs in the order low, high
  int64_t fill = more > 0 ? nk0 / nk1 : 0;
  if (fill * low > tiles1) fill = tiles1 / low;
  int64_t rest = tiles1 - fill * low;
  const int64_t even = rest / npairs, odd = rest % npairs;
  PairLoad most = {0, 0};
  int64_t at = 0;
  for (int i = 0; i < npairs; ++i) {
    const bool high = i < more;
    const int64_t order = high ? low + i : i - more;
    const int64_t mine = even + (high ? 0 : fill) + (order < odd ? 1 : 0);
    const int64_t own = base + (high ? 1 : 0);
    if (first) first[i] = (int)at;
    at += mine;
    if (own + mine > most.items) most.items = own + mine;
    if (own * nk0 + mine * nk1 > most.k_blocks) most.k_blocks = own * nk0 + mine * nk1;
  }
  if (first) first[npairs] = (int)at;
  return most;
}

// Two bf16 products in one launch, the one with more k-blocks first.
cudaError_t launch_two(const Product& g0, const Product& g1, int npairs, unsigned* err,
                       cudaStream_t st) {
  PairArgs<2> a;
  if (!pair_problem(g0, npairs, true, &a.prob[0], &a.map[0]) ||
      !pair_problem(g1, npairs, true, &a.prob[1], &a.map[1]))
    return cudaErrorInvalidValue;
  share_pairs(a.prob[0].num_items, a.prob[0].nk, a.prob[1].num_items, a.prob[1].nk, npairs,
              a.first);
  a.err = err;
  a.wait_ns = block_wait_ns();
  return launch_kernel(linear_pair_kernel<false, 2, kPlain>, dim3((unsigned)(2 * npairs)),
                       dim3(kPairThreads), kPairSmem, st, true, 2, a);
}

// A product's part of a tile launch. `swap`: the MMA's 128 rows are output columns (q), its
// bn columns output rows (p, K-major). *smem: what its stages and accumulators need.
bool tile_problem(const Product& g, bool swap, int bn, int split, int sm_count, TileParams* p,
                  CUtensorMap* ma, CUtensorMap* mb, size_t* smem) {
  const Operand& a = swap ? g.q : g.p;
  const Operand& b = swap ? g.p : g.q;
  if (!copy_map(ma, &p->a_mode, a, g.k, g.f8, 128) ||
      !copy_map(mb, &p->b_mode, b, g.k, g.f8, (uint32_t)bn))
    return false;
  p->epi = g.epi;
  p->k_elems = g.f8 ? 128 : 64;
  p->nk = (int)ceil_div(g.k, p->k_elems);
  p->bn = bn;
  const int64_t tiles_a = ceil_div(a.extent, 128), tiles_b = ceil_div(b.extent, bn);
  const int64_t tiles = tiles_a * tiles_b;
  if (tiles * 8 >= (int64_t(1) << 31)) return false;
  p->tiles_a = (int)tiles_a;
  p->tiles = (int)tiles;
  p->split = split;
  p->split_log2 = 0;
  while (1 << p->split_log2 < split) ++p->split_log2;
  const int stage_bytes = kTile128 + bn * kRowBytes;
  p->stages = tile_stages(bn, takes_long_ring(tiles, p->nk, bn, split, sm_count));
  const size_t acc = (size_t)4 * (swap ? (size_t)bn * 132 : (size_t)128 * (bn + 4));
  size_t need = (size_t)p->stages * stage_bytes;
  if (acc > need) need = acc;
  if (need < kTmemLeastSmem) need = kTmemLeastSmem;  // (rings of narrow tiles: 80 KB)
  *smem = need + 1024;
  return true;
}

cudaError_t launch_tiles(const Product& g, bool swap, int bn, int split, int sm_count,
                         unsigned* err, cudaStream_t st) {
  TileArgs<1> a;
  size_t smem;
  if (!tile_problem(g, swap, bn, split, sm_count, &a.prob[0], &a.a[0], &a.b[0], &smem))
    return cudaErrorInvalidValue;
  a.begin[0] = a.sum_begin = a.sum_ctas = a.dz_cols = 0;
  a.cluster = split;
  a.dz = nullptr;
  a.sums = nullptr;
  a.dz_rows = 0;
  a.err = err;
  a.wait_ns = block_wait_ns();
  const EpiKind kind = epi_kind(g);
  void (*kernel)(TileArgs<1>);
  if (g.f8)
    kernel = swap ? (kind == kAny ? linear_tile_kernel<true, true, 1, kAny>
                                  : linear_tile_kernel<true, true, 1, kAffine>)
                  : (kind == kAny ? linear_tile_kernel<true, false, 1, kAny>
                                  : linear_tile_kernel<true, false, 1, kAffine>);
  else if (swap)
    kernel = kind == kAny      ? linear_tile_kernel<false, true, 1, kAny>
             : kind == kAffine ? linear_tile_kernel<false, true, 1, kAffine>
                               : linear_tile_kernel<false, true, 1, kPlain>;
  else
    kernel = kind == kAny      ? linear_tile_kernel<false, false, 1, kAny>
             : kind == kAffine ? linear_tile_kernel<false, false, 1, kAffine>
                               : linear_tile_kernel<false, false, 1, kPlain>;
  return launch_kernel(kernel, dim3((unsigned)(a.prob[0].tiles * split)), dim3(kTileThreads),
                       smem, st, true, (unsigned)split, a);
}

// Two bf16 products in one launch of clusters of `cluster` CTAs, and with sums (NULL: none)
// [N] the column sums of dz [M, N].
struct TileChoice {
  double us;
  int cluster, bn[2], split[2];  // a split is 1 or the cluster
};
cudaError_t launch_two_tiled(const Product& g0, const Product& g1, const TileChoice& c,
                             const void* dz, int64_t M, int64_t N, float* sums, unsigned* err,
                             cudaStream_t st) {
  TileArgs<2> a;
  size_t smem[2];
  const Product* const g[2] = {&g0, &g1};
  int64_t ctas[2];
  for (int i = 0; i < 2; ++i) {
    if (!tile_problem(*g[i], false, c.bn[i], c.split[i], 0, &a.prob[i], &a.a[i], &a.b[i], &smem[i]))
      return cudaErrorInvalidValue;
    ctas[i] = ceil_div((int64_t)a.prob[i].tiles * c.split[i], c.cluster) * c.cluster;
  }
  const int64_t sum_ctas = sums ? ceil_div(N, kDzWide * kDzCols) * c.cluster : 0;
  const int64_t grid = sum_ctas + ctas[0] + ctas[1];
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  // sums over many rows take as long as the products and start with them; over a few they
  // only fill up behind them
  const bool ahead = M > kDzRows * kDzSumBatch;
  a.begin[0] = ahead ? (int)sum_ctas : 0;
  a.begin[1] = a.begin[0] + (int)ctas[0];
  a.sum_begin = ahead ? 0 : a.begin[1] + (int)ctas[1];
  a.sum_ctas = (int)sum_ctas;
  a.cluster = c.cluster;
  a.dz = static_cast<const __nv_bfloat16*>(dz);
  a.sums = sums;
  a.dz_rows = M;
  a.dz_cols = (int)N;
  a.err = err;
  a.wait_ns = block_wait_ns();
  return launch_kernel(linear_tile_kernel<false, false, 2, kPlain>, dim3((unsigned)grid),
                       dim3(kTileThreads), smem[0] > smem[1] ? smem[0] : smem[1], st, true,
                       (unsigned)c.cluster, a);
}

// Estimated times in microseconds: a launch, a k-block's time, an epilogue a wave, for a split
// the cluster's exchange, and the CTAs that run at one time (clusters of four and eight leave
// SMs of their group empty). Fits to timings of 170 products (1 to 8192 rows, 64 to 8192 terms,
// 64 to 6000 columns) on every variant; on 100 others the variant of the smallest estimate took
// 1.6% more than the fastest one in the mean and 40% at most (36 x 1192 x 3688: 9.3 us, 6.6 in
// swapped tiles over clusters of four). By comparison, pairs alone take up to 4.3 times as long
// (one row, 8192 x 2048: 38 against 8.8 us) and one-CTA tiles alone 2.4 times (2048 x 8192 from
// 333 terms: 35 against 14 us).
double pair_estimate(double items, double k_blocks) {
  return 3.9 + 0.4 * k_blocks + 0.5 * items;
}

// CTAs that run at one time, as clusters of 1, 2, 4 and 8.
double tile_ctas(int i, int sm_count) {
  constexpr double kCap[4] = {148, 143, 103, 97};
  return kCap[i] * sm_count / 148;
}
double tile_start(int cluster) { return 2.2 + (cluster > 1 ? 0.47 + 0.22 * cluster : 0.0); }
double tile_body(int64_t nk, bool swap, int bn, int split, bool long_ring) {
  return ceil_div(nk, split) * (long_ring ? 0.21 + 0.00018 * bn : 0.199 + 0.0007 * bn) +
         (split == 1 ? (swap ? 0.029 : 0.009) : (swap ? 0.026 : 0.022) / sqrt((double)split)) * bn;
}

struct Choice {
  double us;
  int bn, split;  // bn 0: pairs
  bool swap;
};
Choice choose(const Product& g, int npairs, int sm_count) {
  const int64_t rows = g.p.extent, cols = g.q.extent;
  const int64_t nk = ceil_div(g.k, g.f8 ? 128 : 64);
  Choice best = {1e30, 0, 0, false};
  const int64_t tiles256 = ceil_div(rows, 256) * ceil_div(cols, 256);
  if (npairs > 0 && tiles256 < (int64_t(1) << 29)) {
    const int64_t rest = tiles256 % npairs;
    const double waves =
        (double)(tiles256 / npairs) + (rest == 0 ? 0.0 : 2 * rest <= npairs ? 0.5 : 1.0);
    best.us = pair_estimate(waves, waves * nk);
  }
  auto consider = [&](bool swap, int bn) {
    const int64_t tiles = swap ? ceil_div(cols, 128) * ceil_div(rows, bn)
                               : ceil_div(rows, 128) * ceil_div(cols, bn);
    if (tiles >= (int64_t(1) << 28)) return;
    for (int split = 1, i = 0; split <= 8 && split <= nk; split *= 2, ++i) {
      // (an SM with one CTA more takes half as long again, or its full share longer)
      double waves = (double)(tiles * split) / tile_ctas(i, sm_count);
      if (waves > 1.0) waves += 0.5 * (ceil(waves) - waves);
      const double body =
          (waves > 1.0 ? waves : 1.0) *
          tile_body(nk, swap, bn, split, takes_long_ring(tiles, nk, bn, split, sm_count));
      // the tiles' operands, from L2 at 11 TB/s (11e6 bytes a microsecond)
      const double fed = (double)(tiles * split) * ceil_div(nk, split) *
                         (kTile128 + bn * kRowBytes) / 11e6;
      const double us = tile_start(split) + (body > fed ? body : fed);
      if (us < best.us) best = {us, bn, split, swap};
    }
  };
  // up to 64 rows, W may stream past them at the MMA's full height
  if (rows <= 64 && !g.p.mn) consider(true, rows <= 16 ? 16 : rows <= 32 ? 32 : 64);
  consider(false, 64);
  consider(false, 128);
  return best;
}

// The same for two products in one launch of tiles: the longer one's tile or the waves of
// both, whichever takes longer, and a third of the other, since the CTAs share SMs. A fit to
// 120 pairs of products, 9% off in the mean.
// With sum_rows, the column sums of a [sum_rows, sum_cols] operand beside them: a cluster 64
// columns, half a microsecond a batch of rows.
TileChoice choose_two(const Product& g0, const Product& g1, int64_t sum_rows, int64_t sum_cols,
                      int sm_count) {
  TileChoice best = {1e30, 0, {0, 0}, {0, 0}};
  const Product* const g[2] = {&g0, &g1};
  for (int cluster = 1, i = 0; cluster <= 8; cluster *= 2, ++i) {
    // each product's tile and waves: of 64 and 128 columns, whole and split
    double body[2][4], waves[2][4];
    for (int j = 0; j < 2; ++j) {
      const int64_t nk = ceil_div(g[j]->k, 64), rows = ceil_div(g[j]->p.extent, 128);
      for (int v = 0; v < 4; ++v) {
        const int bn = v & 1 ? 128 : 64, split = v & 2 ? cluster : 1;
        const int64_t tiles = rows * ceil_div(g[j]->q.extent, bn);
        const bool fits = tiles < (int64_t(1) << 26) && split <= nk && (v < 2 || cluster > 1);
        body[j][v] = fits ? tile_body(nk, false, bn, split, false) : 1e30;
        waves[j][v] = (double)(tiles * split) / tile_ctas(i, sm_count) * body[j][v];
      }
    }
    double sum_body = 0.0, sum_waves = 0.0;
    if (sum_rows > 0) {
      sum_body = 0.3 + 0.5 * ceil_div(sum_rows, (int64_t)kDzRows * kDzSumBatch * cluster);
      sum_waves = (double)(ceil_div(sum_cols, kDzWide * kDzCols) * cluster) /
                  tile_ctas(i, sm_count) * sum_body;
    }
    for (int v = 0; v < 4; ++v)
      for (int u = 0; u < 4; ++u) {
        double longest = body[0][v] > body[1][u] ? body[0][v] : body[1][u];
        if (sum_body > longest) longest = sum_body;
        double both = waves[0][v] + waves[1][u] + sum_waves;
        if (both > longest) both *= 1.15;  // (full SMs: 10 to 40% over the estimate)
        const double us = tile_start(cluster) + 0.55 + (both > longest ? both : longest) +
                          0.365 * (both > longest ? longest : both);
        if (us < best.us)
          best = {us, cluster, {v & 1 ? 128 : 64, u & 1 ? 128 : 64},
                  {v & 2 ? cluster : 1, u & 2 ? cluster : 1}};
      }
  }
  return best;
}

cudaError_t launch_chosen(const Product& g, const Choice& c, int npairs, int sm_count,
                          unsigned* err, cudaStream_t st) {
  if (c.us >= 1e30) return cudaErrorInvalidValue;
  return c.bn == 0 ? launch_pairs(g, npairs, err, st)
                   : launch_tiles(g, c.swap, c.bn, c.split, sm_count, err, st);
}

}  // namespace

cudaError_t launch_linear(const Linear& a, unsigned* err, int sm_count, cudaStream_t st) {
  Product g;
  g.f8 = a.x_scale != nullptr;
  g.p = {a.x, a.M, false};
  g.q = {a.w, a.N, !g.f8};
  g.k = a.K;
  g.epi = {a.x_scale, a.w_scale, static_cast<const __nv_bfloat16*>(a.bias),
           static_cast<const __nv_bfloat16*>(a.residual), static_cast<__nv_bfloat16*>(a.preact),
           a.out, a.M, (int)a.N, (int)a.act, a.out_f32 ? 1 : 0};
  const int npairs = pair_slots(sm_count);
  return launch_chosen(g, choose(g, npairs, sm_count), npairs, sm_count, err, st);
}

cudaError_t launch_linear_grads(const void* dz, const void* x, const void* W, int64_t M,
                                int64_t K, int64_t N, void* dx, void* dW, float* dbias,
                                float* partial, unsigned* err, int sm_count, cudaStream_t st) {
  const Product gx = {{dz, M, false}, {W, K, false}, N, false,
                      {nullptr, nullptr, nullptr, nullptr, nullptr, dx, M, (int)K, NMOE_ACT_NONE, 0}};
  const Product gw = {{x, K, true}, {dz, N, true}, M, false,
                      {nullptr, nullptr, nullptr, nullptr, nullptr, dW, K, (int)N, NMOE_ACT_NONE, 0}};
  const int npairs = pair_slots(sm_count);
  const Choice cx = choose(gx, npairs, sm_count), cw = choose(gw, npairs, sm_count);
  cudaError_t e = cudaSuccess;
  auto sum_columns = [&] {
    return dbias ? launch_linear_dz(dz, nullptr, M, (int)N, NMOE_ACT_NONE, nullptr, dbias,
                                    partial, st)
                 : cudaSuccess;
  };
  if (dx && dW) {
    const int64_t kx = ceil_div(N, 64), kw = ceil_div(M, 64);
    const Product& g0 = kw > kx ? gw : gx;  // the longer one's CTAs first
    const Product& g1 = kw > kx ? gx : gw;
    // (two launches behind one another take longer than each in its turn; over 97 gradients the
    // choice took 1.6% more than the best of the three in the mean and 38% at most: 6228 x 5456
    // x 152 63 us, as one launch of pairs 45)
    const double apart = 1.1 * (cx.us + cw.us) + 4.0;
    TileChoice tiles = choose_two(g0, g1, 0, 0, sm_count);
    bool beside = false;  // dbias beside the tiles, not 3 us in a launch before them
    if (dbias) {
      const TileChoice with = choose_two(g0, g1, M, N, sm_count);
      beside = with.us < tiles.us + 3.0;
      if (beside) {
        tiles = with;
        tiles.us -= 3.0;  // (which the others have to come)
      }
    }
    double pairs = 1e30;
    const int64_t tx = ceil_div(M, 256) * ceil_div(K, 256);
    const int64_t tw = ceil_div(K, 256) * ceil_div(N, 256);
    if (npairs > 0 && tx + tw < (int64_t(1) << 29)) {
      const PairLoad l = kw > kx ? share_pairs(tw, kw, tx, kx, npairs, nullptr)
                                 : share_pairs(tx, kx, tw, kw, npairs, nullptr);
      pairs = pair_estimate((double)l.items, (double)l.k_blocks);
    }
    if (tiles.us < apart && tiles.us < pairs) {
      if (!beside) e = sum_columns();
      return e != cudaSuccess ? e
                              : launch_two_tiled(g0, g1, tiles, dz, M, N,
                                                 beside ? dbias : nullptr, err, st);
    }
    if (pairs < apart) {
      e = sum_columns();
      return e != cudaSuccess ? e : launch_two(g0, g1, npairs, err, st);
    }
  }
  e = sum_columns();
  if (e == cudaSuccess && dx) e = launch_chosen(gx, cx, npairs, sm_count, err, st);
  if (e == cudaSuccess && dW) e = launch_chosen(gw, cw, npairs, sm_count, err, st);
  return e;
}

// The row shares of 64 columns, and whether they are a cluster.
static int dz_parts(int64_t M, int N, bool* cluster) {
  const int64_t want = ceil_div(M, kDzRows * kDzBatch);  // each a batch of rows or more
  *cluster = M <= kDzClusterRows;
  const int64_t across = ceil_div(N, kDzWide * kDzCols);
  // up to eight, or up to three blocks an SM over both directions
  const int64_t most = *cluster ? 8 : across < 444 ? 444 / across : 1;
  return (int)(want < most ? want : most);
}

int linear_dz_partial_rows(int64_t M, int N) {
  bool cluster;
  const int parts = dz_parts(M, N, &cluster);
  return cluster || parts == 1 ? 0 : parts;
}

cudaError_t launch_linear_dz(const void* dy, const void* preact, int64_t M, int N, nmoe_act act,
                             void* dz, float* dbias, float* partial, cudaStream_t st) {
  bool cluster;
  const int parts = dz_parts(M, N, &cluster);
  const bool direct = cluster || parts == 1;
  const dim3 grid((unsigned)(ceil_div(N, kDzWide * kDzCols) * parts));
  cudaError_t e = launch_kernel(
      direct ? linear_dz_kernel<true> : linear_dz_kernel<false>, grid, dim3(kDzThreads), 0, st,
      true, direct && dbias ? (unsigned)parts : 1u, static_cast<const __nv_bfloat16*>(dy),
      static_cast<const __nv_bfloat16*>(preact), M, N, (int)act, parts,
      static_cast<__nv_bfloat16*>(dz), !dbias ? nullptr : direct ? dbias : partial);
  if (e == cudaSuccess && dbias && !direct) e = launch_sum_parts(partial, parts, N, dbias, st);
  return e;
}

}  // namespace nmoe
