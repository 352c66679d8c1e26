// Balance loss of router scores, per-expert counts, and the loss's gradient.
//
// One warp takes a token: lane l holds experts l*NE .. l*NE + NE - 1. The k best experts
// come out one at a time, as the warp's largest key (one redux) and its lowest holder (one
// ballot), so ties go to the lower expert. Counts and score sums stay in the lanes'
// registers over the warp's tokens and leave the block as one partial row, without atomics;
// a second launch adds the partial rows in a fixed order. The scores are read once; what
// bounds the sizes of a router (2 to 8 MB) is the chain of latencies: a token's k rounds,
// and the two launches.
#include "block_ops.cuh"
#include "sm100_ptx.cuh"

namespace nmoe {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kLossWarps = 32;  // of a block of the second launch
constexpr int kLossThreads = 32 * kLossWarps;

// Tokens a warp works on at a time, so that one's reductions run under the others'.
template <int NE>
struct Batch {
  static constexpr int kTokens = NE <= 4 ? 4 : 2;
};

// Order-preserving key of a score: -0 counts as 0, a NaN as the highest score. 0 is no
// score's key (it marks experts that are taken or beyond E).
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The NE scores of this lane (0 beyond E); `vec`: E is a multiple of NE, so that a lane's
// scores are aligned to their size and all inside E or all outside.
template <int NE>
__device__ __forceinline__ void load_scores(const float* row, int e0, int E, bool vec,
                                            float (&p)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) p[i] = 0.f;
  if (NE > 1 && vec) {
    if (e0 >= E) return;
    if constexpr (NE == 2) {
      const float2 v = *reinterpret_cast<const float2*>(row + e0);
      p[0] = v.x; p[1] = v.y;
    } else if constexpr (NE >= 4) {
#pragma unroll
      for (int i = 0; i < NE; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(row + e0 + i);
        p[i] = v.x; p[i + 1] = v.y; p[i + 2] = v.z; p[i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (e0 + i < E) p[i] = row[e0 + i];
  }
}

__device__ __forceinline__ double shuffle_tree(double v) {  // lane 0: the warp's sum
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  return v;
}

// coef E sum_e (c_e / (k N)) (s_e / N) with cs = sum_e c_e s_e and kn = sum_e c_e = k N
__device__ __forceinline__ float loss_of(double cs, double kn, int E, int k, float coef) {
  const double n = kn / (double)k;
  return kn > 0.0 ? (float)((double)coef * (double)E * cs / (kn * n)) : 0.f;
}

// Block (b, s): of segment s the tokens b*kWarps + warp, + parts*kWarps, ... FINAL: the
// segment's blocks are one cluster, whose first block adds their sums in rank order and
// finishes counts and loss. Else they leave part_p and part_c [n_seg, parts, E].
template <int NE, bool FINAL>
__global__ void __launch_bounds__(kThreads)
balance_partial_kernel(const float* scores, const uint8_t* mask, int64_t S, int E, int k,
                       float coef, double* part_p, int32_t* part_c, int32_t* counts,
                       float* loss) {
  constexpr int kB = Batch<NE>::kTokens;
  __shared__ double sh_p[kWarps][32 * NE];
  __shared__ int32_t sh_c[kWarps][32 * NE];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = lane * NE;
  const bool vec = E % NE == 0;
  const int64_t first = (int64_t)blockIdx.y * S;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  double sum[NE];  // 64 bits: a warp may add the scores of 10^5 tokens
  int32_t cnt[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    sum[i] = 0.0;
    cnt[i] = 0;
  }
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < S; t += kB * step) {
    uint32_t key[kB][NE];  // all 0 for a token that is masked or behind the last
    bool live[kB];
    float p[kB][NE];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int64_t at = first + t + b * step;
      live[b] = t + b * step < S && (!mask || mask[at] != 0);
#pragma unroll
      for (int i = 0; i < NE; ++i) p[b][i] = 0.f;
      if (live[b]) load_scores<NE>(scores + at * E, e0, E, vec, p[b]);
    }
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        key[b][i] = live[b] && e0 + i < E ? score_key(p[b][i]) : 0u;
        sum[i] += (double)p[b][i];
      }
    for (int j = 0; j < k; ++j) {
      uint32_t top[kB], holders[kB];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        top[b] = key[b][0];
#pragma unroll
        for (int i = 1; i < NE; ++i) top[b] = key[b][i] > top[b] ? key[b][i] : top[b];
        holders[b] = top[b];
      }
#pragma unroll
      for (int b = 0; b < kB; ++b) top[b] = __reduce_max_sync(0xffffffffu, top[b]);
#pragma unroll
      for (int b = 0; b < kB; ++b) holders[b] = __ballot_sync(0xffffffffu, holders[b] == top[b]);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        bool open = top[b] != 0u && lane == __ffs((int)holders[b]) - 1;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const bool take = open && key[b][i] == top[b];
          key[b][i] = take ? 0u : key[b][i];
          cnt[i] += take ? 1 : 0;
          open = open && !take;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    sh_p[warp][e0 + i] = sum[i];
    sh_c[warp][e0 + i] = cnt[i];
  }
  __syncthreads();
  const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * E;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double s = 0.0;
    int32_t c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s += sh_p[w][e];
      c += sh_c[w][e];
    }
    if (FINAL) {
      sh_p[0][e] = s;
      sh_c[0][e] = c;
    } else {
      part_p[at + e] = s;
      part_c[at + e] = c;
    }
  }
  if constexpr (FINAL) {
    const int ranks = gridDim.x;
    __syncwarp();  // (the cluster barrier wants converged warps)
    if (ranks > 1) ptx::cluster_sync_all(); else __syncthreads();
    if (blockIdx.x == 0) {
      const int e = threadIdx.x;  // E <= 256 < kThreads
      double s = 0.0;
      int64_t c = 0;
      if (e < E) {
        for (int o = 0; o < ranks; ++o) {
          s += ranks > 1 ? ptx::ld_cluster_d(ptx::mapa_shared(&sh_p[0][e], (uint32_t)o))
                         : sh_p[0][e];
          c += ranks > 1 ? ptx::ld_cluster_s32(ptx::mapa_shared(&sh_c[0][e], (uint32_t)o))
                         : sh_c[0][e];
        }
        counts[(int64_t)blockIdx.y * E + e] = (int32_t)c;
      }
      const double cs = shuffle_tree((double)c * s), cc = shuffle_tree((double)c);
      if (lane == 0) {  // (the other blocks read this one's first rows only)
        sh_p[1][warp] = cs;
        sh_p[2][warp] = cc;
      }
      __syncthreads();
      if (warp == 0) {
        const double a = shuffle_tree(lane < kWarps ? sh_p[1][lane] : 0.0);
        const double kn = shuffle_tree(lane < kWarps ? sh_p[2][lane] : 0.0);
        if (lane == 0) loss[blockIdx.y] = loss_of(a, kn, E, k, coef);
      }
    }
    __syncwarp();
    if (ranks > 1) ptx::cluster_sync_all();  // no block still reads this one's sums
  }
}

// A cluster a segment: block r adds the parts of experts 32 r .. 32 r + 31, each warp every
// kLossWarps-th part in ascending order; then one warp an expert adds the warps' sums, and
// one the experts' products, by fixed trees of shuffles, and the blocks come in rank order.
// All in 64 bits.
__global__ void __launch_bounds__(kLossThreads)
balance_loss_kernel(const double* part_p, const int32_t* part_c, int parts, int E, int k,
                    float coef, int32_t* counts, float* loss) {
  __shared__ double sh_p[kLossWarps][33], sh_c[kLossWarps][33];  // counts are exact: < 2^53
  __shared__ double sh_cs[32], sh_cc[32];
  __shared__ __align__(16) double sh_total[2];  // sum_e c_e s_e, sum_e c_e
  pdl_wait();
  pdl_launch_dependents();
  const int ranks = (E + 31) / 32;
  const int rank = blockIdx.x % ranks, seg = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = rank * 32 + lane;
  const int64_t at = (int64_t)seg * parts * E;
  double s = 0.0;
  int64_t n_e = 0;
  if (e < E) {
#pragma unroll 4
    for (int i = warp; i < parts; i += kLossWarps) {
      s += part_p[at + (int64_t)i * E + e];
      n_e += part_c[at + (int64_t)i * E + e];
    }
  }
  sh_p[warp][lane] = s;
  sh_c[warp][lane] = (double)n_e;
  __syncthreads();
  s = shuffle_tree(sh_p[lane][warp]);
  const double c = shuffle_tree(sh_c[lane][warp]);
  if (lane == 0) {
    if (rank * 32 + warp < E) counts[(int64_t)seg * E + rank * 32 + warp] = (int32_t)c;
    sh_cs[warp] = c * s;
    sh_cc[warp] = c;
  }
  __syncthreads();
  if (warp == 0) {
    const double cs = shuffle_tree(sh_cs[lane]), cc = shuffle_tree(sh_cc[lane]);
    if (lane == 0) {
      sh_total[0] = cs;
      sh_total[1] = cc;
    }
  }
  __syncwarp();  // (the cluster barrier wants converged warps)
  if (ranks > 1) ptx::cluster_sync_all(); else __syncthreads();
  if (rank == 0 && threadIdx.x == 0) {
    double cs = 0.0, kn = 0.0;  // kn = sum_e c_e = k N
    for (int o = 0; o < ranks; ++o) {
      const double2 v = ranks > 1 ? ptx::ld_cluster_d2(ptx::mapa_shared(sh_total, (uint32_t)o))
                                  : make_double2(sh_total[0], sh_total[1]);
      cs += v.x;
      kn += v.y;
    }
    loss[seg] = loss_of(cs, kn, E, k, coef);
  }
  __syncwarp();
  if (ranks > 1) ptx::cluster_sync_all();  // no block still reads this one's totals
}

constexpr int kBackWarps = 8;

template <int NE, typename OutT>
__global__ void __launch_bounds__(32 * kBackWarps)
balance_backward_kernel(const float* scores, const uint8_t* mask, const int32_t* counts,
                        const float* dloss, int64_t S, int E, int k, float coef, int softmax,
                        OutT* dlogits) {
  constexpr int kB = Batch<NE>::kTokens;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = lane * NE;
  const bool vec = E % NE == 0;
  const int64_t first = (int64_t)blockIdx.y * S;
  int32_t c[NE];
  int64_t kn = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    c[i] = e0 + i < E ? counts[(int64_t)blockIdx.y * E + e0 + i] : 0;
    kn += c[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) kn += __shfl_xor_sync(0xffffffffu, kn, o);
  // g_e = dloss coef E c_e / (k N^2), kn = k N; no token left: every row is masked
  const double n = (double)kn / (double)k;
  const double f = kn > 0 ? (double)(dloss ? dloss[blockIdx.y] : 1.f) * (double)coef * (double)E /
                                ((double)kn * n)
                          : 0.0;
  double g[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) g[i] = f * (double)c[i];
  const int64_t step = (int64_t)gridDim.x * kBackWarps;
  for (int64_t t = (int64_t)blockIdx.x * kBackWarps + warp; t < S; t += kB * step) {
    float p[kB][NE], d[kB][NE];
    bool live[kB];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int64_t at = first + t + b * step;
      live[b] = t + b * step < S && (!mask || mask[at] != 0);
#pragma unroll
      for (int i = 0; i < NE; ++i) p[b][i] = 0.f;
      if (live[b]) load_scores<NE>(scores + at * E, e0, E, vec, p[b]);
    }
    if (softmax) {
      // in 64 bits: the g of a nearly balanced router are nearly equal, and the difference
      // with their mean loses most of an fp32's digits
      double dot[kB];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        dot[b] = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) dot[b] = fma((double)p[b][i], g[i], dot[b]);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int b = 0; b < kB; ++b) dot[b] += __shfl_xor_sync(0xffffffffu, dot[b], s);
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int i = 0; i < NE; ++i) d[b][i] = p[b][i] * (float)(g[i] - dot[b]);
    } else {
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int i = 0; i < NE; ++i) d[b][i] = p[b][i] * (1.f - p[b][i]) * (float)g[i];
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if (t + b * step >= S) continue;
#pragma unroll
      for (int i = 0; i < NE; ++i) d[b][i] = live[b] ? d[b][i] : 0.f;  // whatever dloss is
      OutT* o = dlogits + (first + t + b * step) * E + e0;
      if (vec && e0 >= E) continue;
      if (vec && NE == 2 && sizeof(OutT) == 4) {
        *reinterpret_cast<float2*>(o) = make_float2(d[b][0], d[b][1]);
      } else if (vec && NE >= 4 && sizeof(OutT) == 4) {
#pragma unroll
        for (int i = 0; i + 3 < NE; i += 4)
          *reinterpret_cast<float4*>(o + i) =
              make_float4(d[b][i], d[b][i + 1], d[b][i + 2], d[b][i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (e0 + i < E) o[i] = from_f32<OutT>(d[b][i]);
      }
    }
  }
}

template <int NE>
cudaError_t launch_partial(const float* scores, const uint8_t* mask, int64_t S, int E, int k,
                           float coef, int parts, int n_seg, bool final, double* part_p,
                           int32_t* part_c, int32_t* counts, float* loss, cudaStream_t st) {
  return launch_kernel(final ? balance_partial_kernel<NE, true> : balance_partial_kernel<NE, false>,
                       dim3((unsigned)parts, (unsigned)n_seg), dim3(kThreads), 0, st, true,
                       final ? (unsigned)parts : 1u, scores, mask, S, E, k, coef, part_p, part_c,
                       counts, loss);
}

template <int NE, typename OutT>
cudaError_t launch_back(const float* scores, const uint8_t* mask, const int32_t* counts,
                        const float* dloss, int64_t S, int E, int k, int blocks, int n_seg,
                        float coef, int softmax, void* dlogits, cudaStream_t st) {
  return launch_kernel(balance_backward_kernel<NE, OutT>,
                       dim3((unsigned)blocks, (unsigned)n_seg), dim3(32 * kBackWarps), 0, st, true, 1,
                       scores, mask, counts, dloss, S, E, k, coef, softmax,
                       static_cast<OutT*>(dlogits));
}

}  // namespace

// Blocks a segment: one for every batch of its warps, and up to kClusterTokens tokens a
// segment one cluster of at most eight, which finishes the segment in this launch (161
// tokens of 128 experts: 8.6 us with the gradient, 10.3 us with partial rows and a second
// launch; 4096 tokens of 64 experts: 25 us on eight SMs a segment, 14 us on all of them).
constexpr int kClusterTokens = 1024;

struct BalanceGrid {
  int parts;
  bool final;
};
BalanceGrid balance_grid(int64_t S, int E, int n_seg) {
  constexpr int kBlocks = 148;  // (not the device's SMs: the sums' order is the same on any)
  const int64_t want = ceil_div(S, kWarps * (E <= 128 ? Batch<4>::kTokens : Batch<8>::kTokens));
  const bool final = S <= kClusterTokens;
  const int64_t most = final ? 8 : kBlocks / n_seg > 1 ? kBlocks / n_seg : 1;
  return {(int)(want < most ? want : most), final};
}

size_t balance_workspace(int64_t S, int E, int n_seg) {
  const BalanceGrid g = balance_grid(S, E, n_seg);
  return g.final ? 0 : (size_t)12 * g.parts * n_seg * E;  // a double and an int32 an expert
}

cudaError_t launch_balance_loss(const float* scores, const uint8_t* mask, int64_t T, int E,
                                int k, int n_seg, float coef, int32_t* counts, float* loss,
                                void* workspace, cudaStream_t st) {
  const int64_t S = T / n_seg;
  const BalanceGrid g = balance_grid(S, E, n_seg);
  double* part_p = static_cast<double*>(workspace);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)g.parts * n_seg * E);
  auto go = [&](auto fn) {
    return fn(scores, mask, S, E, k, coef, g.parts, n_seg, g.final, part_p, part_c, counts, loss,
              st);
  };
  cudaError_t e = E <= 32    ? go(launch_partial<1>)
                  : E <= 64  ? go(launch_partial<2>)
                  : E <= 128 ? go(launch_partial<4>)
                             : go(launch_partial<8>);
  if (e != cudaSuccess || g.final) return e;
  const int ranks = (int)ceil_div(E, 32);
  return launch_kernel(balance_loss_kernel, dim3((unsigned)(n_seg * ranks)), dim3(kLossThreads),
                       0, st, true, (unsigned)ranks, part_p, part_c, g.parts, E, k, coef, counts,
                       loss);
}

cudaError_t launch_balance_backward(const float* scores, const uint8_t* mask,
                                    const int32_t* counts, const float* dloss, int64_t T, int E,
                                    int k, int n_seg, float coef, nmoe_score_fn fn,
                                    nmoe_dtype dt, void* dlogits, int sm_count,
                                    cudaStream_t st) {
  const int64_t S = T / n_seg;
  // up to four blocks an SM, each warp with a batch of tokens or more
  const int64_t most = ceil_div(4 * (int64_t)sm_count, n_seg);
  const int64_t want = ceil_div(S, kBackWarps * (E <= 128 ? Batch<4>::kTokens : Batch<8>::kTokens));
  const int blocks = (int)(want < most ? want : most);
  const int softmax = fn == NMOE_SCORE_SOFTMAX ? 1 : 0;
  auto go = [&](auto f32, auto bf16) {
    return dt == NMOE_F32 ? f32(scores, mask, counts, dloss, S, E, k, blocks, n_seg, coef,
                                softmax, dlogits, st)
                          : bf16(scores, mask, counts, dloss, S, E, k, blocks, n_seg, coef,
                                 softmax, dlogits, st);
  };
  if (E <= 32) return go(launch_back<1, float>, launch_back<1, __nv_bfloat16>);
  if (E <= 64) return go(launch_back<2, float>, launch_back<2, __nv_bfloat16>);
  if (E <= 128) return go(launch_back<4, float>, launch_back<4, __nv_bfloat16>);
  return go(launch_back<8, float>, launch_back<8, __nv_bfloat16>);
}

}  // namespace nmoe
