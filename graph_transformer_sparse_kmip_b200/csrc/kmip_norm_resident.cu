// kmip_norm_resident.cu -- group norm for inputs that fit in L2: one block per
// (graph, slab of groups), one launch.
//
// Two shapes of block: 256 threads that hold up to eight rows each, and, when
// there are fewer blocks than SMs, 1,024 threads that hold up to two (one
// graph of 1,024 x 32 fp32: a quarter of the steps in a row).
#include "kmip_launch.cuh"
#include "kmip_norm.cuh"

namespace kmip {
namespace {

// Sum over all threads of this thread's group (one vector tile).  `vals` and
// `sums` are shared, [NT] and [kMaxSlabGroups]; two calls in a row take
// different ones.  Lanes of a warp add up first where the tile's layout is a
// power of two (or one group is all there is); other layouts go through
// shared memory thread by thread.
template <int V, int NT>
__device__ __forceinline__ float group_sum(const NormParams& p, const Slab& s, float mine,
                                           float* vals, float* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = p.cg / V;
  if (s.ngroups == 1) {
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) vals[warp] = mine;
    __syncthreads();
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) a += vals[i];
    return a;
  }
  if (s.W <= 32 && (s.W & (s.W - 1)) == 0 && (w & (w - 1)) == 0) {
    for (int o = 16; o >= s.W; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    for (int o = w >> 1; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    const int j = s.tx / w;
    if (lane < s.W && lane % w == 0) vals[warp * s.ngroups + j] = mine;
    __syncthreads();
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) a += vals[i * s.ngroups + j];
    return a;
  }
  vals[threadIdx.x] = mine;
  __syncthreads();
  for (int j = warp; j < s.ngroups; j += NT / 32) {
    float a = 0.f;
    for (int y = lane; y < s.TY; y += 32)
      for (int i = 0; i < w; ++i) a += vals[y * s.W + j * w + i];
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0) sums[j] = a;
  }
  __syncthreads();
  return sums[min(s.tx / w, s.ngroups - 1)];
}

template <typename T, int V, int ACT, int NT, int HOLD>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) norm_fwd_resident(const NormParams p) {
  after_previous();
  __shared__ StatSmem<NT> sm;
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  for (int g = blockIdx.x; g < p.G; g += gridDim.x) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) continue;
    const int rows = hi - lo;
    const int64_t at = (int64_t)g * p.groups + s.g0;
    if (s.vecs <= s.W && rows > 0 && rows <= HOLD * s.TY) {
      const int mine = s.ty < s.TY ? rows - s.ty : 0;  // rows from this thread's first on
      const int c = s.c0 + s.tx * V;
      // (32 bits do: resident inputs are small)
      const int first = (lo + s.ty) * p.C + c, step = s.TY * p.C;
      const T* src = static_cast<const T*>(p.x);
      Row<T, V> x[HOLD];
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) x[u].load(src + (first + u * step));
      float2 sum = splat2(0.f), dev = sum;
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) add_deviations<T, V>(x[u], 0.f, sum, dev);
      const float count = (float)rows * (float)p.cg;
      float* v0 = reinterpret_cast<float*>(sm.s0);
      float* v1 = reinterpret_cast<float*>(sm.q);
      const float m = group_sum<V, NT>(p, s, sum.x + sum.y, v0, sm.mean) / count;
      dev = sum = splat2(0.f);
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) add_deviations<T, V>(x[u], m, sum, dev);
      const float var = group_sum<V, NT>(p, s, dev.x + dev.y, v1, sm.rstd) / count;
      const float rs = 1.f / sqrtf(var + p.eps);
      if (s.ty == 0 && s.tx * V % p.cg == 0) {
        p.mean[at + s.tx * V / p.cg] = m;
        p.rstd[at + s.tx * V / p.cg] = rs;
      }
      Forward<T, V> fw;
      fw.set(p, c, m, rs);
      T* out = static_cast<T*>(p.y);
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          fw.template apply<ACT>(x[u]);
          x[u].store(out + (first + u * step), 0);
        }
      __syncthreads();
      continue;
    }
    slab_stats<T, V, NT, 2>(p, s, lo, hi, sm);
    if (threadIdx.x < s.ngroups) {
      float m, r;
      finish_stats(sm.gs0[threadIdx.x], sm.gq[threadIdx.x], (double)rows * p.cg, p.eps, m, r);
      sm.mean[threadIdx.x] = m;
      sm.rstd[threadIdx.x] = r;
      p.mean[at + threadIdx.x] = m;
      p.rstd[at + threadIdx.x] = r;
    }
    __syncthreads();
    slab_apply<T, V, ACT, 2>(p, s, lo, hi, sm.mean, sm.rstd);
    __syncthreads();
  }
}

template <typename T, int V, int ACT, int NT, int HOLD>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) norm_bwd_resident(const NormParams p) {
  after_previous();
  extern __shared__ float4 dyn[];
  BwdSmem<NT, V>& sm = *reinterpret_cast<BwdSmem<NT, V>*>(dyn);
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  float* dst = p.chan + (int64_t)blockIdx.x * 2 * p.C;
  bool first_graph = true;
  for (int g = blockIdx.x; g < p.G; g += gridDim.x) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) lo = hi = 0;
    const int rows = hi - lo;
    if (threadIdx.x < s.ngroups) sm.gm1[threadIdx.x] = sm.gm2[threadIdx.x] = 0.0;
    if (s.vecs <= s.W && rows <= HOLD * s.TY) {
      const int mine = s.ty < s.TY ? rows - s.ty : 0;
      const int c = s.c0 + s.tx * V, j = s.tx * V / p.cg;
      const int first = (lo + s.ty) * p.C + c, step = s.TY * p.C;
      const T* src = static_cast<const T*>(p.x);
      const T* gsrc = static_cast<const T*>(p.dy);
      Row<T, V> x[HOLD], dy[HOLD];
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          x[u].load(src + (first + u * step));
          dy[u].load(gsrc + (first + u * step));
        }
      Backward<T, V> bw;
      bw.set(p, c, p.mean[(int64_t)g * p.groups + s.g0 + j],
             p.rstd[(int64_t)g * p.groups + s.g0 + j]);
      {
        constexpr int P = Row<T, V>::P;
        float2 sdb[P], sdw[P];
#pragma unroll
        for (int e = 0; e < P; ++e) sdb[e] = sdw[e] = splat2(0.f);
#pragma unroll
        for (int u = 0; u < HOLD; ++u)
          if (u * s.TY < mine) {
            float2 xh[P], dz[P];
            bw.template rows<ACT>(x[u], dy[u], xh, dz);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              sdb[e] = vadd<V>(sdb[e], dz[e]);
              sdw[e] = vfma<V>(dz[e], xh[e], sdw[e]);
            }
          }
        join_channels<T, V, NT, true>(p, s, 0, sdb, sdw, dst, first_graph, sm);
      }
      first_graph = false;
      const float inv = rows ? 1.f / ((float)rows * (float)p.cg) : 0.f;
      const float a1 = (float)sm.gm1[j] * inv, a2 = (float)sm.gm2[j] * inv;
      T* out = static_cast<T*>(p.dx);
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          bw.template apply<ACT>(x[u], dy[u], a1, a2);
          dy[u].store(out + (first + u * step), 0);
        }
      __syncthreads();
      continue;
    }
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_bwd_sums<T, V, ACT, NT, true, 1>(p, s, lo, hi, mean, rstd, dst, first_graph, sm);
    first_graph = false;
    if (threadIdx.x < s.ngroups) {
      const double M = (double)rows * p.cg;
      sm.m1[threadIdx.x] = (float)(sm.gm1[threadIdx.x] / M);
      sm.m2[threadIdx.x] = (float)(sm.gm2[threadIdx.x] / M);
    }
    __syncthreads();
    slab_bwd_apply<T, V, ACT, 1>(p, s, lo, hi, mean, rstd, sm.m1, sm.m2);
    __syncthreads();
  }
}

// Blocks walk over the graphs; enough of them to fill the SMs twice over.
dim3 resident_grid(const NormParams& p, int slabs) {
  return dim3((unsigned)norm_resident_blocks(p, slabs), (unsigned)slabs);
}
bool few_blocks(const NormParams& p, int slabs) {
  return (int64_t)p.G * slabs < device_sm_count();
}

}  // namespace

int norm_resident_blocks(const NormParams& p, int slabs) {
  const int64_t most = ((int64_t)device_sm_count() * 16 + slabs - 1) / slabs;
  return (int)(p.G < most ? p.G : most);
}

cudaError_t launch_norm_fwd_resident(kmip_dtype_t dtype, int v, int act, const NormParams& p,
                                     int slabs, cudaStream_t stream) {
  return norm_dispatch(dtype, v, act, [&]<typename T, int V, int ACT>() {
    if (few_blocks(p, slabs))
      norm_fwd_resident<T, V, ACT, 1024, 2><<<resident_grid(p, slabs), 1024, 0, stream>>>(p);
    else
      norm_fwd_resident<T, V, ACT, 256, 8><<<resident_grid(p, slabs), 256, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_bwd_resident(kmip_dtype_t dtype, int v, int act, const NormParams& p,
                                     int slabs, cudaStream_t stream) {
  return norm_dispatch(dtype, v, act, [&]<typename T, int V, int ACT>() {
    if (few_blocks(p, slabs)) {
      auto kern = norm_bwd_resident<T, V, ACT, 1024, 2>;
      constexpr int smem = sizeof(BwdSmem<1024, V>);
      const cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      kern<<<resident_grid(p, slabs), 1024, smem, stream>>>(p);
    } else {
      norm_bwd_resident<T, V, ACT, 256, 8>
          <<<resident_grid(p, slabs), 256, sizeof(BwdSmem<256, V>), stream>>>(p);
    }
    return cudaGetLastError();
  });
}

}  // namespace kmip
