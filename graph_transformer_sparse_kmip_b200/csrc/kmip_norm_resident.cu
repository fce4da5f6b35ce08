// kmip_norm_resident.cu -- group norm for inputs that fit in L2: one block per
// (graph, slab of groups), one launch.
//
// Two shapes of block: 256 threads that hold up to eight rows each, and, when
// there are fewer blocks than SMs, 1,024 threads that hold up to two (one
// graph of 1,024 x 32 fp32: a quarter of the steps in a row; 5.4 us on the
// device, 6.5 with registers instead of shared memory to hold them).
#include "kmip_launch.cuh"
#include "kmip_norm.cuh"

namespace kmip {
namespace {

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) {
  return make_float2(a.x + b.x, a.y + b.y);
}
__device__ __forceinline__ float from_lane(float a, int o) {
  return __shfl_xor_sync(0xffffffffu, a, o);
}
__device__ __forceinline__ float2 from_lane(float2 a, int o) {
  return make_float2(from_lane(a.x, o), from_lane(a.y, o));
}

// Sum over all threads of this thread's group (one vector tile) of a number or
// a pair.  `vals` and `sums` are shared, [NT] and [kMaxSlabGroups]; two calls in
// a row take different ones.  Lanes of a warp add up first where the tile's
// layout is a power of two (or one group is all there is); other layouts go
// through shared memory thread by thread.
template <int V, int NT, typename S>
__device__ __forceinline__ S group_sum(const NormParams& p, const Slab& s, S mine, S* vals,
                                       S* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = p.cg / V;
  if (s.ngroups == 1) {
#pragma unroll
    for (int o = 16; o; o >>= 1) mine = plus(mine, from_lane(mine, o));
    if (lane == 0) vals[warp] = mine;
    __syncthreads();
    S a = vals[lane % (NT / 32)];
#pragma unroll
    for (int o = NT / 64; o; o >>= 1) a = plus(a, from_lane(a, o));
    return a;
  }
  if (s.W <= 32 && (s.W & (s.W - 1)) == 0 && (w & (w - 1)) == 0) {
    for (int o = 16; o >= s.W; o >>= 1) mine = plus(mine, from_lane(mine, o));
    for (int o = w >> 1; o; o >>= 1) mine = plus(mine, from_lane(mine, o));
    const int j = s.tx / w;
    if (lane < s.W && lane % w == 0) vals[warp * s.ngroups + j] = mine;
    __syncthreads();
    S a{};
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) a = plus(a, vals[i * s.ngroups + j]);
    return a;
  }
  vals[threadIdx.x] = mine;
  __syncthreads();
  for (int j = warp; j < s.ngroups; j += NT / 32) {
    S a{};
    for (int y = lane; y < s.TY; y += 32)
      for (int i = 0; i < w; ++i) a = plus(a, vals[y * s.W + j * w + i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) a = plus(a, from_lane(a, o));
    if (lane == 0) sums[j] = a;
  }
  __syncthreads();
  return sums[min(s.tx / w, s.ngroups - 1)];
}

// A thread's rows of IN inputs between the passes over them, in registers or
// (16-byte vectors only) in shared memory.  Registers start on the first row
// as soon as it is there, but every pass is unrolled over all rows, code that
// runs once a graph and comes from memory.  Shared memory leaves room for more
// blocks an SM.
template <typename T, int V, int IN, int NT, int HOLD, bool SHARED>
struct Held {
  Row<T, V> rows[HOLD][IN];
  __device__ explicit Held(void*) {}
  __device__ void fetch(int u, int i, const T* from) { rows[u][i].load(from); }
  __device__ void landed() {}
  __device__ Row<T, V> get(int u, int i) const { return rows[u][i]; }
};
template <typename T, int V, int IN, int NT, int HOLD>
struct Held<T, V, IN, NT, HOLD, true> {
  uint4* at;  // [HOLD][IN][NT], this thread's column
  __device__ explicit Held(void* shared) : at(static_cast<uint4*>(shared) + threadIdx.x) {}
  __device__ void fetch(int u, int i, const T* from) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at + (u * IN + i) * NT));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  }
  __device__ void landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }
  __device__ Row<T, V> get(int u, int i) const {
    Row<T, V> r;
    r.raw = at[(u * IN + i) * NT];
    return r;
  }
};
template <typename T, int V>
constexpr bool kWide = sizeof(T) * V == 16;

template <typename T, int V, int ACT, int NT, int HOLD, bool SHARED>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : SHARED ? 4 : 2)
norm_fwd_resident(const NormParams p) {
  after_previous();
  constexpr int kUnroll = SHARED ? 2 : HOLD;
  extern __shared__ float4 dyn[];
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
      Held<T, V, 1, NT, HOLD, SHARED> held(dyn);
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) held.fetch(u, 0, src + (first + u * step));
      float2 sum = splat2(0.f), dev = sum;
      held.landed();
#pragma unroll kUnroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) add_deviations<T, V>(held.get(u, 0), 0.f, sum, dev);
      const float count = (float)rows * (float)p.cg;
      float* v0 = reinterpret_cast<float*>(sm.s0);
      float2* v1 = reinterpret_cast<float2*>(sm.q);
      const float near = group_sum<V, NT>(p, s, sum.x + sum.y, v0, sm.mean) / count;
      dev = sum = splat2(0.f);
#pragma unroll kUnroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) add_deviations<T, V>(held.get(u, 0), near, sum, dev);
      // What the first sum lost is in the second: the mean of the differences to
      // it.  (Not where they overflow.)
      const float2 d = group_sum<V, NT>(p, s, make_float2(sum.x + sum.y, dev.x + dev.y), v1,
                                        reinterpret_cast<float2*>(sm.gs0));
      float by = d.x / count, less = by * d.x;
      if (!isfinite(less)) by = less = 0.f;
      const float m = near + by, var = (d.y - less) / count;
      const float rs = 1.f / sqrtf((var < 0.f ? 0.f : var) + p.eps);  // a NaN stays
      if (s.ty == 0 && s.tx * V % p.cg == 0) {
        p.mean[at + s.tx * V / p.cg] = m;
        p.rstd[at + s.tx * V / p.cg] = rs;
      }
      Forward<T, V> fw;
      fw.set(p, c, m, rs);
      T* out = static_cast<T*>(p.y);
#pragma unroll kUnroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          Row<T, V> x = held.get(u, 0);
          fw.template apply<ACT>(x);
          x.store(out + (first + u * step), 0);
        }
      __syncthreads();
      continue;
    }
    slab_stats<T, V, NT, 2>(p, s, lo, lo, hi, sm);
    if (threadIdx.x < s.ngroups) {
      float m, r;
      const float c = rows ? pivot_of(first_of<T>(p, lo, s.g0 + threadIdx.x)) : 0.f;
      finish_stats(sm.gs0[threadIdx.x], sm.gq[threadIdx.x], (double)rows * p.cg, c, p.eps, m, r);
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
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : 2) norm_bwd_resident(const NormParams p) {
  after_previous();
  extern __shared__ float4 dyn[];
  // Two inputs do not fit in registers beside the sums: 256 graphs of 450 x 128
  // bf16 took 55 us so, 38 with shared memory, 64 graphs 18.6 and 15.3.
  constexpr int kUnroll = kWide<T, V> ? 2 : HOLD;
  BwdSmem<NT, V>& sm =
      *reinterpret_cast<BwdSmem<NT, V>*>(dyn + (kWide<T, V> ? HOLD * 2 * NT : 0));
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
      Held<T, V, 2, NT, HOLD, kWide<T, V>> held(dyn);
#pragma unroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          held.fetch(u, 0, src + (first + u * step));
          held.fetch(u, 1, gsrc + (first + u * step));
        }
      Backward<T, V> bw;
      bw.set(p, c, p.mean[(int64_t)g * p.groups + s.g0 + j],
             p.rstd[(int64_t)g * p.groups + s.g0 + j]);
      {
        constexpr int P = Row<T, V>::P;
        float2 sdb[P], sdw[P];
#pragma unroll
        for (int e = 0; e < P; ++e) sdb[e] = sdw[e] = splat2(0.f);
        held.landed();
#pragma unroll kUnroll
        for (int u = 0; u < HOLD; ++u)
          if (u * s.TY < mine) {
            float2 xh[P], dz[P];
            bw.template rows<ACT>(held.get(u, 0), held.get(u, 1), xh, dz);
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
#pragma unroll kUnroll
      for (int u = 0; u < HOLD; ++u)
        if (u * s.TY < mine) {
          Row<T, V> dy = held.get(u, 1);
          bw.template apply<ACT>(held.get(u, 0), dy, a1, a2);
          dy.store(out + (first + u * step), 0);
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
    const auto run = [&]<int NT, int HOLD, bool SHARED>() {
      auto kern = norm_fwd_resident<T, V, ACT, NT, HOLD, SHARED>;
      constexpr int smem = SHARED ? HOLD * NT * 16 : 0;
      static_assert(smem + sizeof(StatSmem<NT>) <= 232448, "shared memory");
      const cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      kern<<<resident_grid(p, slabs), NT, smem, stream>>>(p);
      return cudaGetLastError();
    };
    // Shared memory where blocks wait for one another (48,660 x 128 bf16 in 2,000
    // graphs 18.7 us, with registers 21.5), registers where all run at once
    // (28,072 x 128 in 64 graphs 8.0 us, with shared memory 10.2).
    if (few_blocks(p, slabs)) return run.template operator()<1024, 2, kWide<T, V>>();
    if (kWide<T, V> && (int64_t)p.G * slabs > 2 * device_sm_count())
      return run.template operator()<256, 8, kWide<T, V>>();
    return run.template operator()<256, 8, false>();
  });
}

cudaError_t launch_norm_bwd_resident(kmip_dtype_t dtype, int v, int act, const NormParams& p,
                                     int slabs, cudaStream_t stream) {
  return norm_dispatch(dtype, v, act, [&]<typename T, int V, int ACT>() {
    const auto run = [&]<int NT, int HOLD>() {
      auto kern = norm_bwd_resident<T, V, ACT, NT, HOLD>;
      // up to 106 KB with 256 threads and 226 KB with 1,024, and the statistics
      constexpr int smem = (kWide<T, V> ? HOLD * 2 * NT * 16 : 0) + (int)sizeof(BwdSmem<NT, V>);
      static_assert(smem + 2 * kMaxSlabGroups * 4 <= 232448, "shared memory");
      const cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      kern<<<resident_grid(p, slabs), NT, smem, stream>>>(p);
      return cudaGetLastError();
    };
    return few_blocks(p, slabs) ? run.template operator()<1024, 2>()
                                : run.template operator()<256, 8>();
  });
}

}  // namespace kmip
