// kmip_ffn_rows.cu -- the gated feed-forward block's forward for a few rows
// (one node joining a stored graph).
//
// Bound: reading the weights, 3 C F elements, once.  Tensor-core tiles of 256
// rows would leave most SMs idle and most of each tile empty; here S warps
// share CT output columns (CT rows of Wg and of Wu, or CT rows of Wd) for up
// to NR rows of x, every weight of a step in flight at once, and every SM
// streams weights.  CT = 2 or 4, so that a loaded and widened element of x
// meets four or eight weights.  x and h are small and come
// out of L1.  Sums are fp32, over a warp's lanes and then over the S warps in
// order; h stays in fp32 between the two kernels.
#include "kmip_act.cuh"
#include "kmip_ffn.h"
#include "kmip_launch.cuh"

namespace kmip {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sums of n values (a power of two) over the lanes of a warp.  Each exchange
// halves what a lane still carries: 62 shuffles for 64 values, not 320.
// Afterwards lane l holds, in v[0 ..], values l n / 32 on (n >= 32), or lanes
// l, l + 1, ... of 32 / n the one value l n / 32.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int n = N;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const bool up = lane & o;
          const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

// Vec<X>::load by a plain load: the second kernel starts before the first has
// written h, and the read-only path wants memory that no one writes while a
// kernel lives.
template <typename X>
__device__ __forceinline__ void load_row(const X* p, float* f) {
  if constexpr (sizeof(X) == 4) {
    *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(p);
  } else {
    Vec<X>::load(p, f);  // x, an input
  }
}

// Dot products of M weight rows (w[m], length K) with `rows` rows of x (row
// stride K) over every S-th step from `part` on: acc[m][n], in every lane.
template <typename T, typename X, int M, int NR>
__device__ __forceinline__ void dots(const T* const (&w)[M], const X* x, int rows, int K, int part,
                                     int S, float (&acc)[M * NR]) {
  constexpr int V = Vec<T>::N;
  constexpr int B = M >= 4 ? 1 : 4 / M;  // steps in flight
  const int lane = threadIdx.x & 31, step = S * 32 * V;
#pragma unroll
  for (int i = 0; i < M * NR; ++i) acc[i] = 0.f;
  for (int k0 = (part * 32 + lane) * V; k0 < K; k0 += B * step) {
    float f[B][M][V];
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (k0 + b * step < K) {
#pragma unroll
        for (int m = 0; m < M; ++m) Vec<T>::load(w[m] + k0 + b * step, f[b][m]);
      }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (k0 + b * step >= K) break;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (n >= rows) break;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; e += Vec<X>::N)
          load_row(x + (int64_t)n * K + k0 + b * step + e, v + e);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int e = 0; e < V; ++e)
            acc[m * NR + n] = fmaf(f[b][m][e], v[e], acc[m * NR + n]);
      }
    }
  }
}

// The S warps' sums, in order; afterwards thread i of the column group holds
// the sum of (m, n) = (i / NR, i % NR), for i < M NR.
template <int M, int NR>
__device__ __forceinline__ float join_warps(float (&acc)[M * NR], int group, int S,
                                            float (*red)[M * NR]) {
  constexpr int n = M * NR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  warp_sums(acc);
  if constexpr (n >= 32) {
#pragma unroll
    for (int i = 0; i < n / 32; ++i) red[warp][lane * (n / 32) + i] = acc[i];
  } else {
    if (lane % (32 / n) == 0) red[warp][lane / (32 / n)] = acc[0];
  }
  __syncthreads();
  const int i = threadIdx.x - group * S * 32;
  float sum = 0.f;
  if (i < M * NR)
    for (int s = 0; s < S; ++s) sum += red[group * S + s][i];
  return sum;
}

// h[n][f] = act(x_n . Wg_f) (x_n . Wu_f).
template <typename T, int NR, int CT>
__global__ void __launch_bounds__(kThreads) ffn_rows_glu(const T* x, const T* wg, const T* wu,
                                                         float* h, int N, int C, int F, int act,
                                                         int S) {
  after_previous();
  __shared__ float red[kWarps][2 * CT * NR];
  const int warp = threadIdx.x >> 5, group = warp / S, part = warp % S;
  const int f0 = (blockIdx.x * (kWarps / S) + group) * CT, n0 = blockIdx.y * NR;
  const int rows = min(NR, N - n0);
  const T* w[2 * CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {  // columns behind the last repeat it
    const int64_t f = min(f0 + j, F - 1);
    w[2 * j] = wg + f * C;
    w[2 * j + 1] = wu + f * C;
  }
  float acc[2 * CT * NR];
  dots<T, T, 2 * CT, NR>(w, x + (int64_t)n0 * C, rows, C, part, S, acc);
  join_warps<2 * CT, NR>(acc, group, S, red);
  // gate and up of (j, n) are M-neighbours: one thread takes both
  const int i = threadIdx.x - group * S * 32, j = i / NR, n = i % NR;
  if (i < CT * NR && f0 + j < F && n < rows) {
    float g = 0.f, u = 0.f;
    for (int s = 0; s < S; ++s) {
      g += red[group * S + s][2 * j * NR + n];
      u += red[group * S + s][(2 * j + 1) * NR + n];
    }
    KMIP_ACT_SWITCH(act, h[(int64_t)(n0 + n) * F + f0 + j] = act_value<T, ACT>(g) * u)
  }
}

// y[n][c] = h_n . Wd_c.
template <typename T, int NR, int CT>
__global__ void __launch_bounds__(kThreads) ffn_rows_down(const float* h, const T* wd, T* y, int N,
                                                          int C, int F, int S) {
  after_previous();
  __shared__ float red[kWarps][CT * NR];
  const int warp = threadIdx.x >> 5, group = warp / S, part = warp % S;
  const int c0 = (blockIdx.x * (kWarps / S) + group) * CT, n0 = blockIdx.y * NR;
  const int rows = min(NR, N - n0);
  const T* w[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) w[j] = wd + (int64_t)min(c0 + j, C - 1) * F;
  float acc[CT * NR];
  dots<T, float, CT, NR>(w, h + (int64_t)n0 * F, rows, F, part, S, acc);
  const float sum = join_warps<CT, NR>(acc, group, S, red);
  const int i = threadIdx.x - group * S * 32, j = i / NR, n = i % NR;
  if (i < CT * NR && c0 + j < C && n < rows) y[(int64_t)(n0 + n) * C + c0 + j] = (T)sum;
}

// Warps per column group: more while the blocks do not fill the SMs twice and
// every lane still has a step.
template <typename T>
int share(int columns, int ct, int K) {
  const int groups = (columns + ct - 1) / ct;
  int S = 1;
  while (S < kWarps && groups * S / kWarps < 2 * device_sm_count() &&
         2 * S * 32 * Vec<T>::N <= K)
    S *= 2;
  return S;
}

template <typename T, int NR, int CT>
cudaError_t rows_fwd(const FfnArgs& a, float* h, void* y, cudaStream_t stream) {
  const int parts = (a.N + NR - 1) / NR;
  auto grid = [&](int columns, int S) {
    const int per = kWarps / S * CT;
    return dim3((columns + per - 1) / per, parts);
  };
  const int sg = share<T>(a.F, CT, a.C), sd = share<T>(a.C, CT, a.F);
  ffn_rows_glu<T, NR, CT><<<grid(a.F, sg), kThreads, 0, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.wg), static_cast<const T*>(a.wu), h, a.N,
      a.C, a.F, a.act, sg);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(ffn_rows_down<T, NR, CT>, grid(a.C, sd), kThreads, 0, stream,
                     (const float*)h, static_cast<const T*>(a.wd), static_cast<T*>(y), a.N, a.C,
                     a.F, sd);
}

template <typename T>
cudaError_t rows_fwd(const FfnArgs& a, float* h, void* y, cudaStream_t stream) {
  if (a.N <= 2) return rows_fwd<T, 2, 2>(a, h, y, stream);
  if (a.N <= 4) return rows_fwd<T, 4, 2>(a, h, y, stream);
  return rows_fwd<T, 8, 4>(a, h, y, stream);
}

}  // namespace

cudaError_t launch_ffn_rows_fwd(kmip_dtype_t dtype, const FfnArgs& a, float* h, void* y,
                                cudaStream_t stream) {
  return dtype == KMIP_BF16 ? rows_fwd<__nv_bfloat16>(a, h, y, stream)
                            : rows_fwd<float>(a, h, y, stream);
}

}  // namespace kmip
