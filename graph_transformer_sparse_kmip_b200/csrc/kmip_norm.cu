// kmip_norm.cu -- group norm per graph with an activation, channels last
// (kmip_group_norm_fwd, kmip_group_norm_bwd).
//
// Forward: mean and variance over (nodes of a graph) x (channels of a group),
// then y = act((x - mean) rstd w + b).  Backward: with dz = dy act'(z),
//   db_c = sum dz,  dw_c = sum dz xhat          per channel,
//   m1 = sum_c w_c db_c / M,  m2 = sum_c w_c dw_c / M   per graph and group,
//   dx = rstd (dz w - m1 - xhat m2),
// so the backward's group sums come out of the channel sums of the graph and
// need no pass of their own.
//
// Bound: memory traffic.  Every pass over the rows is the same shape: a block
// owns a slab of whole groups and a range of rows, thread (ty, tx) the V
// channels of vector tx in every TY-th row, kRows rows in flight.
//
// Statistics: a thread takes kRows x V values at a time, forms their own mean
// and squared deviations (two passes over registers) and joins them to its
// running (n, mean, M2); no difference of large sums is formed in fp32.
// Threads, and blocks, join in fp64 sums of n mean and M2 + n mean^2, in a
// fixed order: no atomics, the same bits every run.
//
// Two ways over the graphs, chosen by size in plan():
//   resident  one block per (graph, slab): statistics, then the same rows
//             again while L2 (or L1) still holds them.  One launch.  For small
//             inputs, where launches are what costs.
//   split     rows of each graph cut into slots of R rows; one launch writes
//             each slot's sums, one joins them, one walks the slots again in
//             reverse order, so that what the first pass left in L2 is met
//             first.  Any graph size spreads over all SMs.
#include "kmip_act.cuh"
#include "kmip_internal.h"

namespace kmip {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlabGroups = 64;

struct NormParams {
  const void *x, *w, *b, *dy;
  void *y, *dx;
  const int32_t* offsets;
  float *mean, *rstd;            // [G, groups]
  int N, C, G, groups, cg;
  int gps;                       // groups per slab
  int act;
  float eps;
  int R;                         // split: rows per slot
  int slots;                     // split: N / R + G
  double2* part;                 // split forward: [slots][groups] sums
  float* chan;                   // backward: [blocks or slots][2][C] (db, dw)
  const float* gchan;            // split backward: [G][2][C], per graph
  int* status;
};

// ------------------------------------------------------------ element access
template <typename T, int V>
struct Row;  // V consecutive elements, widened to fp32

template <>
struct Row<__nv_bfloat16, 8> {
  uint4 u;
  __device__ void load(const void* p) { u = *static_cast<const uint4*>(p); }
  __device__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = __uint_as_float(w[t] << 16);
      f[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
    }
  }
  __device__ static void store(void* p, const float* f) {
    Vec<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p), f);
  }
};
template <>
struct Row<__nv_bfloat16, 2> {
  uint32_t u;
  __device__ void load(const void* p) { u = *static_cast<const uint32_t*>(p); }
  __device__ void get(float* f) const {
    f[0] = __uint_as_float(u << 16);
    f[1] = __uint_as_float(u & 0xffff0000u);
  }
  __device__ static void store(void* p, const float* f) {
    *static_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
  }
};
template <>
struct Row<__nv_bfloat16, 1> {
  __nv_bfloat16 u;
  __device__ void load(const void* p) { u = *static_cast<const __nv_bfloat16*>(p); }
  __device__ void get(float* f) const { f[0] = __bfloat162float(u); }
  __device__ static void store(void* p, const float* f) {
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct Row<float, 4> {
  float4 u;
  __device__ void load(const void* p) { u = *static_cast<const float4*>(p); }
  __device__ void get(float* f) const { f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; }
  __device__ static void store(void* p, const float* f) {
    *static_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Row<float, 1> {
  float u;
  __device__ void load(const void* p) { u = *static_cast<const float*>(p); }
  __device__ void get(float* f) const { f[0] = u; }
  __device__ static void store(void* p, const float* f) { *static_cast<float*>(p) = f[0]; }
};

// ---------------------------------------------------------------- row ranges
// Node range of graph g; false (and a status) when its offsets are malformed.
__device__ __forceinline__ bool graph_rows(const NormParams& p, int g, int& lo, int& hi) {
  lo = p.offsets ? p.offsets[g] : 0;
  hi = p.offsets ? p.offsets[g + 1] : p.N;
  const bool ok = lo >= 0 && lo <= hi && hi <= p.N && (g > 0 || lo == 0) &&
                  (g < p.G - 1 || hi == p.N);
  if (!ok && threadIdx.x == 0) record_status(p.status, KMIP_ERR_BAD_OFFSETS);
  return ok;
}

// Slots: graph g owns slots [lo / R + g, ...), one per R rows; no two graphs'
// slots meet because floor((lo + n) / R) + 1 >= floor(lo / R) + ceil(n / R).
__device__ __forceinline__ int first_slot(const NormParams& p, int g) {
  return (p.offsets ? p.offsets[g] : 0) / p.R + g;
}

// Graph and rows of a slot; false when the slot holds none.
__device__ __forceinline__ bool slot_rows(const NormParams& p, int slot, int& g, int& r0,
                                          int& r1) {
  int a = 0, b = p.G - 1;  // last graph whose first slot is <= slot
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (first_slot(p, m) <= slot) a = m; else b = m - 1;
  }
  g = a;
  int lo, hi;
  if (!graph_rows(p, g, lo, hi)) return false;
  const int64_t at = lo + (int64_t)(slot - first_slot(p, g)) * p.R;
  if (at < lo || at >= hi) return false;
  r0 = (int)at;
  r1 = (int)min(at + p.R, (int64_t)hi);
  return true;
}

// ------------------------------------------------------------- block's slab
// The slab's vectors go in tiles of at most kThreads; W = tile width, TY rows
// side by side.
struct Slab {
  int c0, vecs, W, TY, tx, ty, ngroups, g0;
};

template <int V>
__device__ __forceinline__ Slab make_slab(const NormParams& p, int slab) {
  Slab s;
  s.g0 = slab * p.gps;
  s.ngroups = min(p.gps, p.groups - s.g0);
  s.c0 = s.g0 * p.cg;
  s.vecs = s.ngroups * p.cg / V;
  s.W = min(s.vecs, kThreads);
  s.TY = kThreads / s.W;
  s.tx = threadIdx.x % s.W;
  s.ty = threadIdx.x / s.W;
  return s;
}

struct StatSmem {
  double s0[kThreads], q[kThreads];
  double gs0[kMaxSlabGroups], gq[kMaxSlabGroups];
  float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
};

// Adds sum(n mean) and sum(M2 + n mean^2) of rows [r0, r1) to sm.gs0, sm.gq.
template <typename T, int V>
__device__ void slab_stats(const NormParams& p, const Slab& s, int r0, int r1, StatSmem& sm) {
  constexpr int kRows = V >= 4 ? 4 : 8;
  if (threadIdx.x < s.ngroups) sm.gs0[threadIdx.x] = sm.gq[threadIdx.x] = 0.0;
  for (int vt = 0; vt < s.vecs; vt += s.W) {
    const int v = vt + s.tx;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    if (s.ty < s.TY && v < s.vecs) {
      const T* col = static_cast<const T*>(p.x) + s.c0 + v * V;
      for (int r = r0 + s.ty; r < r1; r += kRows * s.TY) {
        Row<T, V> raw[kRows];
        const int left = (r1 - r + s.TY - 1) / s.TY;
        const int cnt = min(left, kRows);
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (u < cnt) raw[u].load(col + (int64_t)(r + u * s.TY) * p.C);
        float f[kRows][V], sum = 0.f, dev = 0.f;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (u < cnt) {
            raw[u].get(f[u]);
#pragma unroll
            for (int e = 0; e < V; ++e) sum += f[u][e];
          }
        const float nb = (float)(cnt * V);
        const float mb = sum / nb;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (u < cnt) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float t = f[u][e] - mb;
              dev = fmaf(t, t, dev);
            }
          }
        const float all = n + nb, d = mb - mean, share = nb / all;
        mean = fmaf(d, share, mean);
        m2 += fmaf(d * d, n * share, dev);
        n = all;
      }
    }
    sm.s0[threadIdx.x] = (double)n * mean;
    sm.q[threadIdx.x] = (double)m2 + (double)n * mean * mean;
    __syncthreads();
    // one warp per group of this tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vpg = p.cg / V, tile = min(s.W, s.vecs - vt);
    for (int j = vt / vpg + warp; j < s.ngroups && j * vpg < vt + tile; j += kThreads / 32) {
      const int a = max(j * vpg - vt, 0), b = min((j + 1) * vpg - vt, tile);
      const int w = b - a;
      double s0 = 0.0, q = 0.0;
      for (int i = lane; i < w * s.TY; i += 32) {
        const int at = (i / w) * s.W + a + i % w;
        s0 += sm.s0[at];
        q += sm.q[at];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        q += __shfl_xor_sync(0xffffffffu, q, o);
      }
      if (lane == 0) {
        sm.gs0[j] += s0;
        sm.gq[j] += q;
      }
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void finish_stats(double s0, double q, double count, float eps,
                                             float& mean, float& rstd) {
  const double m = count > 0 ? s0 / count : 0.0;
  double var = count > 0 ? q / count - m * m : 0.0;
  var = var < 0.0 ? 0.0 : var;  // a NaN stays
  mean = (float)m;
  rstd = (float)rsqrt(var + (double)eps);
}

// Channel parameters of a vector.
template <typename T, int V>
__device__ __forceinline__ void load_affine(const NormParams& p, int c, float* w, float* b) {
  const T* pw = static_cast<const T*>(p.w);
  const T* pb = static_cast<const T*>(p.b);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    w[e] = pw ? (float)pw[c + e] : 1.f;
    b[e] = pb ? (float)pb[c + e] : 0.f;
  }
}

template <typename T, int V>
__device__ void slab_apply(const NormParams& p, const Slab& s, int r0, int r1, const float* mean,
                           const float* rstd) {
  constexpr int kRows = V >= 4 ? 4 : 8;
  if (s.ty >= s.TY) return;
  for (int v = s.tx; v < s.vecs; v += s.W) {
    const int c = s.c0 + v * V, j = v * V / p.cg;
    float w[V], b[V];
    load_affine<T, V>(p, c, w, b);
    const float m = mean[j], rs = rstd[j];
    const T* col = static_cast<const T*>(p.x) + c;
    T* out = static_cast<T*>(p.y) + c;
    for (int r = r0 + s.ty; r < r1; r += kRows * s.TY) {
      Row<T, V> raw[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (r + u * s.TY < r1) raw[u].load(col + (int64_t)(r + u * s.TY) * p.C);
      KMIP_ACT_SWITCH(p.act, {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (r + u * s.TY < r1) {
            float f[V];
            raw[u].get(f);
#pragma unroll
            for (int e = 0; e < V; ++e)
              f[e] = act_value<T, ACT>(fmaf((f[e] - m) * rs, w[e], b[e]));
            Row<T, V>::store(out + (int64_t)(r + u * s.TY) * p.C, f);
          }
        }
      })
    }
  }
}

// ---------------------------------------------------------------- backward
struct BwdSmem {
  float red[2 * 2048];        // [2][threads * V]: per-thread channel sums
  double gm1[kMaxSlabGroups], gm2[kMaxSlabGroups];
  float m1[kMaxSlabGroups], m2[kMaxSlabGroups];
};

// Channel sums (db, dw) of rows [r0, r1), to dst[0][c], dst[1][c] (added to
// what is there unless `first`); with GROUPS also sm.gm1, sm.gm2.
template <typename T, int V, bool GROUPS>
__device__ void slab_bwd_sums(const NormParams& p, const Slab& s, int r0, int r1,
                              const float* mean, const float* rstd, float* dst, bool first,
                              BwdSmem& sm) {
  constexpr int kRows = V >= 4 ? 2 : 4;
  if (GROUPS && threadIdx.x < s.ngroups) sm.gm1[threadIdx.x] = sm.gm2[threadIdx.x] = 0.0;
  for (int vt = 0; vt < s.vecs; vt += s.W) {
    const int v = vt + s.tx;
    const bool on = s.ty < s.TY && v < s.vecs;
    float sdb[V], sdw[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sdb[e] = sdw[e] = 0.f;
    if (on) {
      const int c = s.c0 + v * V, j = v * V / p.cg;
      float w[V], b[V];
      load_affine<T, V>(p, c, w, b);
      const float m = mean[j], rs = rstd[j];
      const T* col = static_cast<const T*>(p.x) + c;
      const T* gcol = static_cast<const T*>(p.dy) + c;
      for (int r = r0 + s.ty; r < r1; r += kRows * s.TY) {
        Row<T, V> rx[kRows], rg[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (r + u * s.TY < r1) {
            rx[u].load(col + (int64_t)(r + u * s.TY) * p.C);
            rg[u].load(gcol + (int64_t)(r + u * s.TY) * p.C);
          }
        KMIP_ACT_SWITCH(p.act, {
#pragma unroll
          for (int u = 0; u < kRows; ++u) {
            if (r + u * s.TY < r1) {
              float f[V], g[V];
              rx[u].get(f);
              rg[u].get(g);
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const float xh = (f[e] - m) * rs;
                float fa;
                float ga;
                act_both<T, ACT>(fmaf(xh, w[e], b[e]), fa, ga);
                const float dz = g[e] * ga;
                sdb[e] += dz;
                sdw[e] = fmaf(dz, xh, sdw[e]);
              }
            }
          }
        })
      }
    }
    float* rb = sm.red;
    float* rw = sm.red + kThreads * V;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      rb[threadIdx.x * V + e] = sdb[e];
      rw[threadIdx.x * V + e] = sdw[e];
    }
    __syncthreads();
    // rows of threads, in order, for each channel of the tile; the sums go
    // back into the first row of threads' places for the group sums
    const int tile = min(s.W, s.vecs - vt) * V;
    for (int c = threadIdx.x; c < tile; c += kThreads) {
      float a = 0.f, q = 0.f;
      for (int y = 0; y < s.TY; ++y) {
        a += rb[y * s.W * V + c];
        q += rw[y * s.W * V + c];
      }
      const int ch = s.c0 + vt * V + c;
      dst[ch] = first ? a : dst[ch] + a;
      dst[p.C + ch] = first ? q : dst[p.C + ch] + q;
      if (GROUPS) {
        const float w = p.w ? (float)static_cast<const T*>(p.w)[ch] : 1.f;
        rb[c] = a * w;
        rw[c] = q * w;
      }
    }
    __syncthreads();
    if (GROUPS) {
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      const int base = vt * V;
      for (int j = base / p.cg + warp; j < s.ngroups && j * p.cg < base + tile;
           j += kThreads / 32) {
        const int a = max(j * p.cg - base, 0), b = min((j + 1) * p.cg - base, tile);
        double s1 = 0.0, s2 = 0.0;
        for (int i = a + lane; i < b; i += 32) {
          s1 += rb[i];
          s2 += rw[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        if (lane == 0) {
          sm.gm1[j] += s1;
          sm.gm2[j] += s2;
        }
      }
      __syncthreads();
    }
  }
}

template <typename T, int V>
__device__ void slab_bwd_apply(const NormParams& p, const Slab& s, int r0, int r1,
                               const float* mean, const float* rstd, const float* m1,
                               const float* m2) {
  constexpr int kRows = V >= 4 ? 2 : 4;
  if (s.ty >= s.TY) return;
  for (int v = s.tx; v < s.vecs; v += s.W) {
    const int c = s.c0 + v * V, j = v * V / p.cg;
    float w[V], b[V];
    load_affine<T, V>(p, c, w, b);
    const float m = mean[j], rs = rstd[j], a1 = m1[j], a2 = m2[j];
    const T* col = static_cast<const T*>(p.x) + c;
    const T* gcol = static_cast<const T*>(p.dy) + c;
    T* out = static_cast<T*>(p.dx) + c;
    for (int r = r0 + s.ty; r < r1; r += kRows * s.TY) {
      Row<T, V> rx[kRows], rg[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (r + u * s.TY < r1) {
          rx[u].load(col + (int64_t)(r + u * s.TY) * p.C);
          rg[u].load(gcol + (int64_t)(r + u * s.TY) * p.C);
        }
      KMIP_ACT_SWITCH(p.act, {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (r + u * s.TY < r1) {
            float f[V], g[V];
            rx[u].get(f);
            rg[u].get(g);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float xh = (f[e] - m) * rs;
              float fa;
              float ga;
              act_both<T, ACT>(fmaf(xh, w[e], b[e]), fa, ga);
              f[e] = rs * (fmaf(g[e] * ga, w[e], -a1) - xh * a2);
            }
            Row<T, V>::store(out + (int64_t)(r + u * s.TY) * p.C, f);
          }
        }
      })
    }
  }
}

// Copies the statistics of graph g's slab to shared memory.
__device__ __forceinline__ void load_stats(const NormParams& p, const Slab& s, int g, float* mean,
                                           float* rstd) {
  if (threadIdx.x < s.ngroups) {
    mean[threadIdx.x] = p.mean[(int64_t)g * p.groups + s.g0 + threadIdx.x];
    rstd[threadIdx.x] = p.rstd[(int64_t)g * p.groups + s.g0 + threadIdx.x];
  }
}

// ----------------------------------------------------------------- resident
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_fwd_resident(const NormParams p) {
  __shared__ StatSmem sm;
  const Slab s = make_slab<V>(p, blockIdx.y);
  for (int g = blockIdx.x; g < p.G; g += gridDim.x) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) continue;
    slab_stats<T, V>(p, s, lo, hi, sm);
    if (threadIdx.x < s.ngroups) {
      float m, r;
      finish_stats(sm.gs0[threadIdx.x], sm.gq[threadIdx.x], (double)(hi - lo) * p.cg, p.eps, m, r);
      sm.mean[threadIdx.x] = m;
      sm.rstd[threadIdx.x] = r;
      p.mean[(int64_t)g * p.groups + s.g0 + threadIdx.x] = m;
      p.rstd[(int64_t)g * p.groups + s.g0 + threadIdx.x] = r;
    }
    __syncthreads();
    slab_apply<T, V>(p, s, lo, hi, sm.mean, sm.rstd);
    __syncthreads();
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_bwd_resident(const NormParams p) {
  __shared__ BwdSmem sm;
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<V>(p, blockIdx.y);
  float* dst = p.chan + (int64_t)blockIdx.x * 2 * p.C;
  bool first = true;
  for (int g = blockIdx.x; g < p.G; g += gridDim.x) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) lo = hi = 0;
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_bwd_sums<T, V, true>(p, s, lo, hi, mean, rstd, dst, first, sm);
    first = false;
    if (threadIdx.x < s.ngroups && hi > lo) {
      const double M = (double)(hi - lo) * p.cg;
      sm.m1[threadIdx.x] = (float)(sm.gm1[threadIdx.x] / M);
      sm.m2[threadIdx.x] = (float)(sm.gm2[threadIdx.x] / M);
    }
    __syncthreads();
    slab_bwd_apply<T, V>(p, s, lo, hi, mean, rstd, sm.m1, sm.m2);
    __syncthreads();
  }
}

// -------------------------------------------------------------------- split
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_stats_split(const NormParams p) {
  __shared__ StatSmem sm;
  const Slab s = make_slab<V>(p, blockIdx.y);
  for (int slot = blockIdx.x; slot < p.slots; slot += gridDim.x) {
    int g, r0, r1;
    if (!slot_rows(p, slot, g, r0, r1)) continue;
    slab_stats<T, V>(p, s, r0, r1, sm);
    if (threadIdx.x < s.ngroups)
      p.part[(int64_t)slot * p.groups + s.g0 + threadIdx.x] =
          make_double2(sm.gs0[threadIdx.x], sm.gq[threadIdx.x]);
    __syncthreads();
  }
}

// One block per (graph, group): joins the graph's slots in a fixed order.
__global__ void __launch_bounds__(128) norm_join_stats(const NormParams p) {
  __shared__ double s0[4], s1[4];
  for (int64_t i = blockIdx.x; i < (int64_t)p.G * p.groups; i += gridDim.x) {
    const int g = (int)(i / p.groups), j = (int)(i % p.groups);
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) continue;
    const int a = first_slot(p, g), n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    double x = 0.0, q = 0.0;
#pragma unroll 4
    for (int t = threadIdx.x; t < n; t += 128) {
      const double2 v = p.part[(int64_t)(a + t) * p.groups + j];
      x += v.x;
      q += v.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if ((threadIdx.x & 31) == 0) {
      s0[threadIdx.x >> 5] = x;
      s1[threadIdx.x >> 5] = q;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      float m, r;
      finish_stats(s0[0] + s0[1] + s0[2] + s0[3], s1[0] + s1[1] + s1[2] + s1[3],
                   (double)(hi - lo) * p.cg, p.eps, m, r);
      p.mean[i] = m;
      p.rstd[i] = r;
    }
    __syncthreads();
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_apply_split(const NormParams p) {
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<V>(p, blockIdx.y);
  for (int slot = p.slots - 1 - (int)blockIdx.x; slot >= 0; slot -= gridDim.x) {
    int g, r0, r1;
    if (!slot_rows(p, slot, g, r0, r1)) continue;
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_apply<T, V>(p, s, r0, r1, mean, rstd);
    __syncthreads();
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_bwd_sums_split(const NormParams p) {
  __shared__ BwdSmem sm;
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<V>(p, blockIdx.y);
  for (int slot = blockIdx.x; slot < p.slots; slot += gridDim.x) {
    int g, r0, r1;
    if (!slot_rows(p, slot, g, r0, r1)) continue;
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_bwd_sums<T, V, false>(p, s, r0, r1, mean, rstd, p.chan + (int64_t)slot * 2 * p.C, true,
                               sm);
  }
}

// Sums of 32 channel columns over the rows of `src` [rows][2][C]: a graph's
// slots (per graph, to fp32) or all rows (to the parameters' type).
__device__ __forceinline__ float join_column(const float* src, int64_t cols, int rows,
                                             int64_t col, float (*red)[33]) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float a = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int r = ty; r < rows; r += 16) a += src[(int64_t)r * cols + col];
  }
  red[ty][tx] = a;
  __syncthreads();
  float sum = 0.f;
  if (ty == 0)
    for (int y = 0; y < 16; ++y) sum += red[y][tx];
  __syncthreads();
  return sum;  // meaningful in the first warp
}

__global__ void __launch_bounds__(512) norm_join_graph(const NormParams p, float* gchan) {
  __shared__ float red[16][33];
  const int64_t cols = 2 * (int64_t)p.C, col = blockIdx.x * 32ll + (threadIdx.x & 31);
  for (int g = blockIdx.y; g < p.G; g += gridDim.y) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) lo = hi = 0;
    const int n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    const float* src = p.chan + (hi > lo ? (int64_t)first_slot(p, g) * cols : 0);
    const float sum = join_column(src, cols, n, col, red);
    if (threadIdx.x < 32 && col < cols) gchan[(int64_t)g * cols + col] = sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(512) norm_join_params(const float* src, int rows, int C, T* dw,
                                                        T* db) {
  __shared__ float red[16][33];
  const int64_t cols = 2 * (int64_t)C, col = blockIdx.x * 32ll + (threadIdx.x & 31);
  const float sum = join_column(src, cols, rows, col, red);
  if (threadIdx.x < 32 && col < cols) {
    if (col < C) db[col] = (T)sum;
    else dw[col - C] = (T)sum;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply_split(const NormParams p) {
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  __shared__ float m1[kMaxSlabGroups], m2[kMaxSlabGroups];
  const Slab s = make_slab<V>(p, blockIdx.y);
  int have = -1;
  for (int slot = p.slots - 1 - (int)blockIdx.x; slot >= 0; slot -= gridDim.x) {
    int g, r0, r1;
    if (!slot_rows(p, slot, g, r0, r1)) continue;
    if (g != have) {  // means of the graph's groups, from its channel sums
      have = g;
      __syncthreads();
      load_stats(p, s, g, mean, rstd);
      int lo, hi;
      graph_rows(p, g, lo, hi);
      const float* src = p.gchan + (int64_t)g * 2 * p.C;
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      for (int j = warp; j < s.ngroups; j += kThreads / 32) {
        double a = 0.0, b = 0.0;
        for (int c = lane; c < p.cg; c += 32) {
          const int ch = s.c0 + j * p.cg + c;
          const float w = p.w ? (float)static_cast<const T*>(p.w)[ch] : 1.f;
          a += src[ch] * w;
          b += src[p.C + ch] * w;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (lane == 0) {
          const double M = (double)(hi - lo) * p.cg;
          m1[j] = (float)(a / M);
          m2[j] = (float)(b / M);
        }
      }
      __syncthreads();
    }
    slab_bwd_apply<T, V>(p, s, r0, r1, mean, rstd, m1, m2);
  }
}

// --------------------------------------------------------------------- host
// Inputs up to this size, with graphs whose slab of one block is small, take
// the resident kernels.
constexpr int64_t kResidentBytes = 16 << 20, kResidentSlabBytes = 128 << 10;

struct Plan {
  bool resident;
  int slabs;
};

// Sets p.gps, p.R, p.slots.
template <typename T>
Plan plan(NormParams& p, int V) {
  Plan pl;
  const int64_t row = (int64_t)p.C * sizeof(T), group = (int64_t)p.cg * sizeof(T);
  // whole groups of at least 32 bytes a row, so that no sector is read twice
  int gps = (int)((32 + group - 1) / group);
  gps = gps > kMaxSlabGroups ? kMaxSlabGroups : gps;
  gps = gps > p.groups ? p.groups : gps;
  const int64_t slab = (int64_t)gps * group;
  pl.resident = row * p.N <= kResidentBytes && slab * (p.N / p.G) <= kResidentSlabBytes;
  if (!pl.resident) {
    // as many groups as a row of threads covers
    gps = kThreads * V / p.cg;
    gps = gps < 1 ? 1 : gps > kMaxSlabGroups ? kMaxSlabGroups : gps;
    gps = gps > p.groups ? p.groups : gps;
  }
  p.gps = gps;
  pl.slabs = (p.groups + gps - 1) / gps;
  // about eight slots per SM and slab, of at least 64 rows
  const int64_t want = (int64_t)device_sm_count() * 8;
  int64_t R = ((int64_t)p.N * pl.slabs + want - 1) / want;
  p.R = (int)(R < 64 ? 64 : R);
  p.slots = p.N / p.R + p.G;
  return pl;
}

dim3 grid_of(int64_t items, int slabs) {
  const int64_t most = (int64_t)device_sm_count() * 16;
  const int64_t x = (most + slabs - 1) / slabs;
  return dim3((unsigned)(items < x ? items : x), (unsigned)slabs);
}

template <typename T, int V>
cudaError_t norm_fwd(NormParams p, cudaStream_t stream) {
  const Plan pl = plan<T>(p, V);
  if (pl.slabs > 65535) return cudaErrorNotSupported;
  if (pl.resident) {
    norm_fwd_resident<T, V><<<grid_of(p.G, pl.slabs), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  void* scratch = nullptr;
  cudaError_t e = scratch_alloc(&scratch, sizeof(double2) * (size_t)p.slots * p.groups, stream);
  if (e != cudaSuccess) return e;
  p.part = static_cast<double2*>(scratch);
  const dim3 grid = grid_of(p.slots, pl.slabs);
  norm_stats_split<T, V><<<grid, kThreads, 0, stream>>>(p);
  const int64_t joins = (int64_t)p.G * p.groups;
  norm_join_stats<<<(unsigned)(joins < 65536 ? joins : 65536), 128, 0, stream>>>(p);
  norm_apply_split<T, V><<<grid, kThreads, 0, stream>>>(p);
  e = cudaGetLastError();
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : ef;
}

template <typename T, int V>
cudaError_t norm_bwd(NormParams p, void* dweight, void* dbias, cudaStream_t stream) {
  const Plan pl = plan<T>(p, V);
  if (pl.slabs > 65535) return cudaErrorNotSupported;
  const dim3 grid = grid_of(pl.resident ? p.G : p.slots, pl.slabs);
  const int64_t rows = pl.resident ? grid.x : p.slots, cols = 2 * (int64_t)p.C;
  void* scratch = nullptr;
  cudaError_t e = scratch_alloc(
      &scratch, sizeof(float) * (size_t)cols * (size_t)(rows + (pl.resident ? 0 : p.G)), stream);
  if (e != cudaSuccess) return e;
  p.chan = static_cast<float*>(scratch);
  const unsigned tiles = (unsigned)((cols + 31) / 32);
  const float* sums = p.chan;
  int nsums = (int)rows;
  if (pl.resident) {
    norm_bwd_resident<T, V><<<grid, kThreads, 0, stream>>>(p);
  } else {
    float* gchan = p.chan + rows * cols;
    p.gchan = gchan;
    norm_bwd_sums_split<T, V><<<grid, kThreads, 0, stream>>>(p);
    norm_join_graph<<<dim3(tiles, p.G < 65535 ? p.G : 65535), 512, 0, stream>>>(p, gchan);
    norm_bwd_apply_split<T, V><<<grid, kThreads, 0, stream>>>(p);
    sums = gchan;
    nsums = p.G;
  }
  if (p.w)
    norm_join_params<T><<<tiles, 512, 0, stream>>>(sums, nsums, p.C, static_cast<T*>(dweight),
                                                   static_cast<T*>(dbias));
  e = cudaGetLastError();
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : ef;
}

// Widest vector inside one group that every pointer and row allows.
int vector_width(const NormParams& p, size_t esize, bool bwd) {
  const int wide = (int)(16 / esize), options[2] = {wide, esize == 2 ? 2 : 1};
  for (int v : options) {
    const uint64_t bytes = v * esize;
    auto off = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % bytes != 0; };
    if (p.cg % v || off(p.x) || (bwd ? off(p.dy) || off(p.dx) : off(p.y))) continue;
    return v;
  }
  return 1;
}

kmip_status_t check_norm(const int32_t* offsets, int64_t N, int C, int groups, int act,
                         int num_graphs, int dtype) {
  if (N < 0 || N > INT32_MAX || C < 1 || groups < 1 || C % groups) return KMIP_ERR_INVALID_ARG;
  if (dtype != KMIP_BF16 && dtype != KMIP_F32) return KMIP_ERR_INVALID_ARG;
  if (act < KMIP_ACT_NONE || act > KMIP_ACT_RELU) return KMIP_ERR_INVALID_ARG;
  if (offsets && num_graphs < 1) return KMIP_ERR_INVALID_ARG;
  if (C > 65536 || N * (int64_t)C > ((int64_t)1 << 40)) return KMIP_ERR_UNSUPPORTED;
  // slots are numbered in 32 bits
  if (offsets && N / 64 + (int64_t)num_graphs > INT32_MAX) return KMIP_ERR_UNSUPPORTED;
  return KMIP_OK;
}

kmip_status_t to_status(cudaError_t e) {
  if (e == cudaSuccess) return KMIP_OK;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? KMIP_ERR_UNSUPPORTED : KMIP_ERR_CUDA;
}

bool aligned_to(const void* q, size_t n) { return reinterpret_cast<uintptr_t>(q) % n == 0; }

}  // namespace
}  // namespace kmip

using namespace kmip;

extern "C" __attribute__((visibility("default"))) kmip_status_t kmip_group_norm_fwd(
    const void* x, const void* weight, const void* bias, const int32_t* graph_offsets, int64_t N,
    int C, int groups, float eps, kmip_act_t act, void* y, float* mean, float* rstd,
    kmip_stream_t stream_, int num_graphs, kmip_dtype_t dtype) {
  const kmip_status_t st = check_norm(graph_offsets, N, C, groups, act, num_graphs, dtype);
  if (st != KMIP_OK) return st;
  if (!(eps > 0.f) || !isfinite(eps)) return KMIP_ERR_INVALID_ARG;
  if (!mean || !rstd || (N > 0 && (!x || !y)) || !weight != !bias) return KMIP_ERR_INVALID_ARG;
  const size_t es = dtype == KMIP_BF16 ? 2 : 4;
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(weight, es) ||
      !aligned_to(bias, es))
    return KMIP_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.w = weight;
  p.b = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.offsets = graph_offsets;
  p.N = (int)N;
  p.C = C;
  p.G = graph_offsets ? num_graphs : 1;
  p.groups = groups;
  p.cg = C / groups;
  p.act = act;
  p.eps = eps;
  p.status = status_ptr();
  if (!p.status) return KMIP_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int v = vector_width(p, es, false);
  if (dtype == KMIP_BF16)
    return to_status(v == 8   ? norm_fwd<__nv_bfloat16, 8>(p, stream)
                     : v == 2 ? norm_fwd<__nv_bfloat16, 2>(p, stream)
                              : norm_fwd<__nv_bfloat16, 1>(p, stream));
  return to_status(v == 4 ? norm_fwd<float, 4>(p, stream) : norm_fwd<float, 1>(p, stream));
}

extern "C" __attribute__((visibility("default"))) kmip_status_t kmip_group_norm_bwd(
    const void* dy, const void* x, const void* weight, const void* bias,
    const int32_t* graph_offsets, const float* mean, const float* rstd, int64_t N, int C,
    int groups, kmip_act_t act, void* dx, void* dweight, void* dbias, kmip_stream_t stream_,
    int num_graphs, kmip_dtype_t dtype) {
  const kmip_status_t st = check_norm(graph_offsets, N, C, groups, act, num_graphs, dtype);
  if (st != KMIP_OK) return st;
  if (!mean || !rstd || (N > 0 && (!x || !dy || !dx)) || !weight != !bias)
    return KMIP_ERR_INVALID_ARG;
  if (weight && (!dweight || !dbias)) return KMIP_ERR_INVALID_ARG;
  if (N > 0 && dx == x) return KMIP_ERR_INVALID_ARG;
  const size_t es = dtype == KMIP_BF16 ? 2 : 4;
  if (!aligned_to(x, es) || !aligned_to(dy, es) || !aligned_to(dx, es) ||
      !aligned_to(weight, es) || !aligned_to(bias, es) || !aligned_to(dweight, es) ||
      !aligned_to(dbias, es))
    return KMIP_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.w = weight;
  p.b = bias;
  p.dy = dy;
  p.dx = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.offsets = graph_offsets;
  p.N = (int)N;
  p.C = C;
  p.G = graph_offsets ? num_graphs : 1;
  p.groups = groups;
  p.cg = C / groups;
  p.act = act;
  p.status = status_ptr();
  if (!p.status) return KMIP_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int v = vector_width(p, es, true);
  if (dtype == KMIP_BF16)
    return to_status(v == 8   ? norm_bwd<__nv_bfloat16, 8>(p, dweight, dbias, stream)
                     : v == 2 ? norm_bwd<__nv_bfloat16, 2>(p, dweight, dbias, stream)
                              : norm_bwd<__nv_bfloat16, 1>(p, dweight, dbias, stream));
  return to_status(v == 4 ? norm_bwd<float, 4>(p, dweight, dbias, stream)
                          : norm_bwd<float, 1>(p, dweight, dbias, stream));
}
