// kmip_norm.cuh -- group norm per graph with an activation, channels last: what
// its kernels share (kmip_norm_resident.cu, kmip_norm.cu).
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
// channels of vector tx in every TY-th row, kRows rows in flight while the
// next kRows are being loaded.
//
// Two ways over the graphs, chosen by size in plan():
//   resident  one block per (graph, slab), one launch, for inputs that fit in
//             L2 and where launches are what costs.  A graph of up to HOLD TY
//             rows (512 or 1,024) stays in registers or shared memory: sum, then
//             squared deviations from the mean, then the result, with one read
//             of x.  Longer ones are read again.
//   split     rows of each graph cut into slots of R rows; one launch writes
//             each slot's sums, one joins them, one walks the slots again in
//             reverse order, so that what the first pass left in L2 is met
//             first.  Any graph size spreads over all SMs.
//
// Means and variances are formed from differences, so that an offset common to
// all values costs no digits and values that are all alike have variance 0.
// Rows that are held add up in fp32, then their differences to that mean, which
// correct it, and the squares.  Otherwise a thread keeps (n, mean, M2) and adds
// kRows x V values at a time by their deviations from its mean; threads, and
// blocks, join in fp64 sums of n (mean - c) and M2 + n (mean - c)^2, where c is
// the group's first value: (mean - c)^2 is then at most n times the variance,
// and the difference of the two keeps it to n 2^-53.  The backward's channel
// sums are fp32 throughout, joined over threads, slots and graphs.  All sums run
// in a fixed order: no atomics, the same bits every run.
#pragma once

#include "kmip_act.cuh"
#include "kmip_internal.h"

namespace kmip {

constexpr int kMaxSlabGroups = 64;

struct NormParams {
  const void *x, *w, *b, *dy;
  void *y, *dx;
  const int32_t* offsets;
  float *mean, *rstd;            // [G, groups]
  int N, C, G, groups, cg;
  int gps;                       // groups per slab
  float eps;
  int R;                         // split: rows per slot
  int slots;                     // split: N / R + G
  double2* part;                 // split forward: [slots][groups] sums
  float* chan;                   // backward: [blocks or slots][2][C] (db, dw)
  const float* gchan;            // split backward: [G][2][C], per graph
  int once;                      // larger than L2: nothing that is written or
                                 // read for the last time should stay there
  int* status;
};

// ------------------------------------------------------------ element access
template <int BYTES>
struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

// V consecutive elements, widened to fp32.
template <typename T, int V>
struct Row {
  using R = typename Raw<sizeof(T) * V>::type;
  R raw;
  __device__ void load(const T* p) { raw = *reinterpret_cast<const R*>(p); }
  __device__ void load_last(const T* p) { raw = __ldcs(reinterpret_cast<const R*>(p)); }
  // As pairs (P = 1 single, in .x, when V = 1).
  static constexpr int P = V > 1 ? V / 2 : 1;
  __device__ void get(float2 (&f)[P]) const {
    if constexpr (sizeof(T) == 4) {
      const float* q = reinterpret_cast<const float*>(&raw);
#pragma unroll
      for (int e = 0; e < P; ++e)
        f[e] = make_float2(q[V > 1 ? 2 * e : 0], V > 1 ? q[2 * e + 1] : 0.f);
    } else if constexpr (V == 1) {
      f[0] = make_float2(__uint_as_float((uint32_t)raw << 16), 0.f);
    } else {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int e = 0; e < P; ++e)
        f[e] = make_float2(__uint_as_float(q[e] << 16), __uint_as_float(q[e] & 0xffff0000u));
    }
  }
  __device__ void set(const float2 (&f)[P]) {
    if constexpr (sizeof(T) == 4) {
      float* q = reinterpret_cast<float*>(&raw);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        q[V > 1 ? 2 * e : 0] = f[e].x;
        if (V > 1) q[2 * e + 1] = f[e].y;
      }
    } else if constexpr (V == 1) {
      raw = __bfloat16_as_ushort(__float2bfloat16_rn(f[0].x));
    } else {
      __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
      for (int e = 0; e < P; ++e) q[e] = __floats2bfloat162_rn(f[e].x, f[e].y);
    }
  }
  __device__ void store(T* p, int once) const {
    if (once) __stcs(reinterpret_cast<R*>(p), raw);
    else *reinterpret_cast<R*>(p) = raw;
  }
};

// Pairs of V elements; with V = 1 only .x counts, and plain instructions serve.
template <int V>
__device__ __forceinline__ float2 vadd(float2 a, float2 b) {
  return V > 1 ? add2(a, b) : make_float2(a.x + b.x, 0.f);
}
template <int V>
__device__ __forceinline__ float2 vmul(float2 a, float2 b) {
  return V > 1 ? mul2(a, b) : make_float2(a.x * b.x, 0.f);
}
template <int V>
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) {
  return V > 1 ? fma2(a, b, c) : make_float2(fmaf(a.x, b.x, c.x), 0.f);
}

// ---------------------------------------------------------------- row ranges
// Node range of graph g; false (and a status) when its offsets are malformed.
// One of the threads that ask for the same graph reports.
__device__ __forceinline__ bool graph_rows(const NormParams& p, int g, int& lo, int& hi,
                                           bool reports) {
  lo = p.offsets ? p.offsets[g] : 0;
  hi = p.offsets ? p.offsets[g + 1] : p.N;
  const bool ok = lo >= 0 && lo <= hi && hi <= p.N && (g > 0 || lo == 0) &&
                  (g < p.G - 1 || hi == p.N);
  if (!ok && reports) record_status(p.status, KMIP_ERR_BAD_OFFSETS);
  return ok;
}
// (the whole block asks)
__device__ __forceinline__ bool graph_rows(const NormParams& p, int g, int& lo, int& hi) {
  return graph_rows(p, g, lo, hi, threadIdx.x == 0);
}

// Slots: graph g owns slots [lo / R + g, ...), one per R rows; no two graphs'
// slots meet because floor((lo + n) / R) + 1 >= floor(lo / R) + ceil(n / R).
__device__ __forceinline__ int first_slot(const NormParams& p, int g) {
  return (p.offsets ? p.offsets[g] : 0) / p.R + g;
}

// Graph, its first row, and the rows of a slot; false when the slot holds none.
// (The same plain search in every thread: everything that follows from it stays
// in uniform registers.  A search by 32 probes of a warp made the backward's
// passes over single elements a third slower.)
__device__ __forceinline__ bool slot_rows(const NormParams& p, int slot, int& g, int& lo, int& r0,
                                          int& r1) {
  int a = 0, b = p.G - 1;  // last graph whose first slot is <= slot
  while (a < b) {
    const int m = a + ((b - a + 1) >> 1);
    if (first_slot(p, m) <= slot) a = m; else b = m - 1;
  }
  g = a;
  int hi;
  if (!graph_rows(p, g, lo, hi)) return false;
  const int64_t at = lo + (int64_t)(slot - first_slot(p, g)) * p.R;
  if (at < lo || at >= hi) return false;
  r0 = (int)at;
  r1 = (int)min(at + p.R, (int64_t)hi);
  return true;
}

// ------------------------------------------------------------- block's slab
// The slab's vectors go in tiles of at most NT threads; W = tile width, TY
// rows side by side.
struct Slab {
  int c0, vecs, W, TY, tx, ty, ngroups, g0;
};

template <int NT, int V>
__device__ __forceinline__ Slab make_slab(const NormParams& p, int slab) {
  Slab s;
  s.g0 = slab * p.gps;
  s.ngroups = min(p.gps, p.groups - s.g0);
  s.c0 = s.g0 * p.cg;
  s.vecs = s.ngroups * p.cg / V;
  s.W = min(s.vecs, NT);
  s.TY = NT / s.W;
  s.tx = threadIdx.x % s.W;
  s.ty = threadIdx.x / s.W;
  return s;
}

// Rows of a batch in the split kernels' passes over x, and over x and dy: 64
// bytes of each thread on their way twice over (31,623 x 345 fp32 training
// step, single elements: 110 us with half of that, 97 with this).
template <int V>
constexpr int kRowsOne = V >= 4 ? 4 : 16;
template <int V>
constexpr int kRowsTwo = V >= 4 ? 2 : 8;

// Rows r0 + ty, + TY, ... of a column in batches of KR: body(rows, r, n) with
// the n <= KR rows r, r + TY, ..., the next batch already on its way.
template <int KR, typename T, int V, int NIN, typename F>
__device__ __forceinline__ void walk_rows(const Slab& s, int r0, int r1, int64_t ld,
                                          const T* const (&col)[NIN], bool last, F&& body) {
  const int step = KR * s.TY;
  Row<T, V> cur[NIN][KR], nxt[NIN][KR];
  auto fetch = [&](Row<T, V> (&dst)[NIN][KR], int r) {
#pragma unroll
    for (int u = 0; u < KR; ++u)
      if (r + u * s.TY < r1) {
#pragma unroll
        for (int i = 0; i < NIN; ++i) {
          const T* q = col[i] + (int64_t)(r + u * s.TY) * ld;
          if (last) dst[i][u].load_last(q);
          else dst[i][u].load(q);
        }
      }
  };
  int r = r0 + s.ty;
  fetch(cur, r);
  while (r < r1) {
    const int rn = r + step;
    if (rn < r1) fetch(nxt, rn);
    body(cur, r);
    r = rn;
#pragma unroll
    for (int i = 0; i < NIN; ++i)
#pragma unroll
      for (int u = 0; u < KR; ++u) cur[i][u] = nxt[i][u];
  }
}

// Adds x - shift and its square over a row's vector.
template <typename T, int V>
__device__ __forceinline__ void add_deviations(const Row<T, V>& row, float shift, float2& sum,
                                               float2& square) {
  float2 f[Row<T, V>::P];
  row.get(f);
#pragma unroll
  for (int e = 0; e < Row<T, V>::P; ++e) {
    const float2 t = vadd<V>(f[e], make_float2(-shift, V > 1 ? -shift : 0.f));
    sum = vadd<V>(sum, t);
    square = vfma<V>(t, t, square);
  }
}

template <int NT>
struct StatSmem {
  double s0[NT], q[NT];
  double gs0[kMaxSlabGroups], gq[kMaxSlabGroups];
  float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
};

// The value that a group's sums are relative to: its first, of the graph's row
// lo (zero if that is not finite: the others' sums are to stay what they are).
// Loaded ahead of the rows, looked at behind them.
template <typename T>
__device__ __forceinline__ T first_of(const NormParams& p, int lo, int group) {
  return static_cast<const T*>(p.x)[(int64_t)lo * p.C + group * p.cg];
}
template <typename T>
__device__ __forceinline__ float pivot_of(T first) {
  return isfinite((float)first) ? (float)first : 0.f;
}

// Sets sm.gs0, sm.gq to sum(n (mean - c)) and sum(M2 + n (mean - c)^2) of rows
// [r0, r1), c the pivots of the graph that begins at row lo.
template <typename T, int V, int NT, int KR>
__device__ void slab_stats(const NormParams& p, const Slab& s, int lo, int r0, int r1,
                           StatSmem<NT>& sm) {
  if (threadIdx.x < s.ngroups) sm.gs0[threadIdx.x] = sm.gq[threadIdx.x] = 0.0;
  for (int vt = 0; vt < s.vecs; vt += s.W) {
    const int v = vt + s.tx;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    T c = T(0.f);
    if (s.ty < s.TY && v < s.vecs) {
      if (r0 < r1) c = first_of<T>(p, lo, s.g0 + v * V / p.cg);
      const T* const cols[1] = {static_cast<const T*>(p.x) + s.c0 + v * V};
      walk_rows<KR, T, V, 1>(s, r0, r1, p.C, cols, false, [&](Row<T, V> (&rows)[1][KR], int r) {
        // squared deviations from the running mean (at first from one of the
        // values): sum d^2 - (sum d)^2 / n is then a difference of like terms
        // only where it is large itself
        if (n == 0.f) {
          float2 f[Row<T, V>::P];
          rows[0][0].get(f);
          mean = f[0].x;
        }
        float2 sum = make_float2(0.f, 0.f), dev = sum;
        int cnt = 0;
#pragma unroll
        for (int u = 0; u < KR; ++u)
          if (r + u * s.TY < r1) {
            add_deviations<T, V>(rows[0][u], mean, sum, dev);
            ++cnt;
          }
        const float all = n + (float)(cnt * V), d = sum.x + sum.y, share = __fdividef(d, all);
        mean += share;
        m2 += fmaf(-d, share, dev.x + dev.y);
        n = all;
      });
    }
    const double off = (double)mean - pivot_of(c);
    sm.s0[threadIdx.x] = n * off;
    sm.q[threadIdx.x] = m2 + n * off * off;
    __syncthreads();
    // one warp per group of this tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vpg = p.cg / V, tile = min(s.W, s.vecs - vt);
    for (int j = vt / vpg + warp; j < s.ngroups && j * vpg < vt + tile; j += NT / 32) {
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

__device__ __forceinline__ void finish_stats(double s0, double q, double count, float pivot,
                                             float eps, float& mean, float& rstd) {
  const double m = count > 0 ? s0 / count : 0.0;
  double var = count > 0 ? q / count - m * m : 0.0;
  var = var < 0.0 ? 0.0 : var;  // a NaN stays
  mean = (float)(pivot + m);
  rstd = (float)rsqrt(var + (double)eps);
}

// Weight and bias of a vector.
template <typename T, int V>
__device__ __forceinline__ void load_affine(const NormParams& p, int c,
                                            float2 (&w)[Row<T, V>::P], float2 (&b)[Row<T, V>::P]) {
  if (p.w) {
    Row<T, V> r;
    r.load(static_cast<const T*>(p.w) + c);
    r.get(w);
    r.load(static_cast<const T*>(p.b) + c);
    r.get(b);
  } else {
#pragma unroll
    for (int e = 0; e < Row<T, V>::P; ++e) {
      w[e] = splat2(1.f);
      b[e] = splat2(0.f);
    }
  }
}

// z = (x - mean) a + b with a = rstd w.  The difference comes first, for bf16
// too: x a + (b - mean a) would be off by 2^-24 of mean rstd w, and rstd can be
// 300 where all values of a group are alike.
template <typename T, int V>
struct Forward {
  static constexpr int P = Row<T, V>::P;
  float2 a[P], b[P];
  float mean;
  __device__ void set(const NormParams& p, int ch, float m, float rs) {
    load_affine<T, V>(p, ch, a, b);
    mean = m;
#pragma unroll
    for (int e = 0; e < P; ++e) a[e] = vmul<V>(a[e], splat2(rs));
  }
  template <int ACT>
  __device__ void apply(Row<T, V>& row) const {
    float2 f[P];
    row.get(f);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 z = vfma<V>(vadd<V>(f[e], splat2(-mean)), a[e], b[e]);
      f[e] = V > 1 ? act_value2<T, ACT>(z) : make_float2(act_value<T, ACT>(z.x), 0.f);
    }
    row.set(f);
  }
};

// xhat and dz of a vector, likewise.
template <typename T, int V>
struct Backward {
  static constexpr int P = Row<T, V>::P;
  float2 w[P], b[P];
  float mean, rs;
  __device__ void set(const NormParams& p, int ch, float m, float r) {
    load_affine<T, V>(p, ch, w, b);
    mean = m;
    rs = r;
  }
  template <int ACT>
  __device__ void rows(const Row<T, V>& row, const Row<T, V>& grad, float2 (&xh)[P],
                       float2 (&dz)[P]) const {
    row.get(xh);
    grad.get(dz);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      xh[e] = vmul<V>(vadd<V>(xh[e], splat2(-mean)), splat2(rs));
      const float2 z = vfma<V>(xh[e], w[e], b[e]);
      float2 f, g;
      if (V > 1) {
        act_both2<T, ACT>(z, f, g);
      } else {
        act_both<T, ACT>(z.x, f.x, g.x);
        g.y = 0.f;
      }
      dz[e] = vmul<V>(dz[e], g);
    }
  }
  // dx = rs (dz w - m1 - xhat m2), into grad's place
  template <int ACT>
  __device__ void apply(const Row<T, V>& row, Row<T, V>& grad, float m1, float m2) const {
    float2 xh[P], dz[P];
    rows<ACT>(row, grad, xh, dz);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 t = vfma<V>(dz[e], w[e], splat2(-m1));
      dz[e] = vmul<V>(vfma<V>(xh[e], splat2(-m2), t), splat2(rs));
    }
    grad.set(dz);
  }
};

template <typename T, int V, int ACT, int KR>
__device__ void slab_apply(const NormParams& p, const Slab& s, int r0, int r1, const float* mean,
                           const float* rstd) {
  if (s.ty >= s.TY) return;
  for (int v = s.tx; v < s.vecs; v += s.W) {
    const int c = s.c0 + v * V, j = v * V / p.cg;
    Forward<T, V> fw;
    fw.set(p, c, mean[j], rstd[j]);
    const T* const cols[1] = {static_cast<const T*>(p.x) + c};
    T* out = static_cast<T*>(p.y) + c;
    walk_rows<KR, T, V, 1>(s, r0, r1, p.C, cols, p.once, [&](Row<T, V> (&rows)[1][KR], int r) {
#pragma unroll
      for (int u = 0; u < KR; ++u)
        if (r + u * s.TY < r1) {
          fw.template apply<ACT>(rows[0][u]);
          rows[0][u].store(out + (int64_t)(r + u * s.TY) * p.C, p.once);
        }
    });
  }
}

// ---------------------------------------------------------------- backward
// (At most 42 KB with 256 threads, 162 KB with 1,024; the resident kernels keep
// 64 KB of rows beside it.)
template <int NT, int V>
struct BwdSmem {
  float red[2][NT * V / 2 * 3];  // [channel of the tile][TY, or TY + 1 if even]
  float2 sums[NT * V];           // of the tile's channels, times weight
  double gm1[kMaxSlabGroups], gm2[kMaxSlabGroups];
  float m1[kMaxSlabGroups], m2[kMaxSlabGroups];
};

// Channel sums of the threads of a tile of vectors (at vector vt of the
// slab): sdb, sdw of each thread, over ty, to dst[0][c], dst[1][c] (added to
// what is there unless `first`); with GROUPS also added to sm.gm1, sm.gm2.
template <typename T, int V, int NT, bool GROUPS>
__device__ void join_channels(const NormParams& p, const Slab& s, int vt,
                              const float2 (&sdb)[Row<T, V>::P], const float2 (&sdw)[Row<T, V>::P],
                              float* dst, bool first, BwdSmem<NT, V>& sm) {
  const int pitch = s.TY | 1, tile = min(s.W, s.vecs - vt) * V;
  if (s.ty < s.TY) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sm.red[0][(s.tx * V + e) * pitch + s.ty] = e & 1 ? sdb[e / 2].y : sdb[e / 2].x;
      sm.red[1][(s.tx * V + e) * pitch + s.ty] = e & 1 ? sdw[e / 2].y : sdw[e / 2].x;
    }
  }
  __syncthreads();
  // L lanes share the threads' sums of one channel
  int L = 1;
  while (L < 32 && L < s.TY && tile * L * 2 <= NT) L *= 2;
  const int part = threadIdx.x & (L - 1);
  for (int c0 = 0; c0 < tile; c0 += NT / L) {  // uniform, for the shuffles
    const int c = c0 + threadIdx.x / L;
    float a = 0.f, q = 0.f;
    if (c < tile)
      for (int y = part; y < s.TY; y += L) {
        a += sm.red[0][c * pitch + y];
        q += sm.red[1][c * pitch + y];
      }
    for (int o = L >> 1; o; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (c < tile && part == 0) {
      const int ch = s.c0 + vt * V + c;
      dst[ch] = first ? a : dst[ch] + a;
      dst[p.C + ch] = first ? q : dst[p.C + ch] + q;
      if (GROUPS) {
        const float w = p.w ? (float)static_cast<const T*>(p.w)[ch] : 1.f;
        sm.sums[c] = make_float2(a * w, q * w);
      }
    }
  }
  __syncthreads();
  if (GROUPS) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = vt * V;
    for (int j = base / p.cg + warp; j < s.ngroups && j * p.cg < base + tile; j += NT / 32) {
      const int a = max(j * p.cg - base, 0), b = min((j + 1) * p.cg - base, tile);
      double s1 = 0.0, s2 = 0.0;
      for (int i = a + lane; i < b; i += 32) {
        s1 += sm.sums[i].x;
        s2 += sm.sums[i].y;
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

// Channel sums (db, dw) of rows [r0, r1), as in join_channels.
template <typename T, int V, int ACT, int NT, bool GROUPS, int KR>
__device__ void slab_bwd_sums(const NormParams& p, const Slab& s, int r0, int r1,
                              const float* mean, const float* rstd, float* dst, bool first,
                              BwdSmem<NT, V>& sm) {
  for (int vt = 0; vt < s.vecs; vt += s.W) {
    const int v = vt + s.tx;
    constexpr int P = Row<T, V>::P;
    float2 sdb[P], sdw[P];
#pragma unroll
    for (int e = 0; e < P; ++e) sdb[e] = sdw[e] = splat2(0.f);
    if (s.ty < s.TY && v < s.vecs) {
      const int c = s.c0 + v * V, j = v * V / p.cg;
      Backward<T, V> bw;
      bw.set(p, c, mean[j], rstd[j]);
      const T* const cols[2] = {static_cast<const T*>(p.x) + c, static_cast<const T*>(p.dy) + c};
      walk_rows<KR, T, V, 2>(s, r0, r1, p.C, cols, false, [&](Row<T, V> (&rows)[2][KR], int r) {
#pragma unroll
        for (int u = 0; u < KR; ++u)
          if (r + u * s.TY < r1) {
            float2 xh[P], dz[P];
            bw.template rows<ACT>(rows[0][u], rows[1][u], xh, dz);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              sdb[e] = vadd<V>(sdb[e], dz[e]);
              sdw[e] = vfma<V>(dz[e], xh[e], sdw[e]);
            }
          }
      });
    }
    join_channels<T, V, NT, GROUPS>(p, s, vt, sdb, sdw, dst, first, sm);
  }
}

template <typename T, int V, int ACT, int KR>
__device__ void slab_bwd_apply(const NormParams& p, const Slab& s, int r0, int r1,
                               const float* mean, const float* rstd, const float* m1,
                               const float* m2) {
  if (s.ty >= s.TY) return;
  for (int v = s.tx; v < s.vecs; v += s.W) {
    const int c = s.c0 + v * V, j = v * V / p.cg;
    Backward<T, V> bw;
    bw.set(p, c, mean[j], rstd[j]);
    const float a1 = m1[j], a2 = m2[j];
    const T* const cols[2] = {static_cast<const T*>(p.x) + c, static_cast<const T*>(p.dy) + c};
    T* out = static_cast<T*>(p.dx) + c;
    walk_rows<KR, T, V, 2>(s, r0, r1, p.C, cols, p.once, [&](Row<T, V> (&rows)[2][KR], int r) {
#pragma unroll
      for (int u = 0; u < KR; ++u)
        if (r + u * s.TY < r1) {
          bw.template apply<ACT>(rows[0][u], rows[1][u], a1, a2);
          rows[1][u].store(out + (int64_t)(r + u * s.TY) * p.C, p.once);
        }
    });
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

// The resident kernels (kmip_norm_resident.cu); p.gps is set.
// norm_resident_blocks: rows of p.chan that the backward writes.
int norm_resident_blocks(const NormParams& p, int slabs);
cudaError_t launch_norm_fwd_resident(kmip_dtype_t dtype, int v, int act, const NormParams& p,
                                     int slabs, cudaStream_t stream);
cudaError_t launch_norm_bwd_resident(kmip_dtype_t dtype, int v, int act, const NormParams& p,
                                     int slabs, cudaStream_t stream);

// Calls f.template operator()<T, V, ACT>() for the element type, the vector
// width and the activation.
template <typename F>
cudaError_t norm_dispatch(kmip_dtype_t dtype, int v, int act, F&& f) {
  cudaError_t e = cudaErrorInvalidValue;
  KMIP_ACT_SWITCH(act, {
    if (dtype == KMIP_BF16)
      e = v == 8   ? f.template operator()<__nv_bfloat16, 8, ACT>()
          : v == 2 ? f.template operator()<__nv_bfloat16, 2, ACT>()
                   : f.template operator()<__nv_bfloat16, 1, ACT>();
    else
      e = v == 4 ? f.template operator()<float, 4, ACT>() : f.template operator()<float, 1, ACT>();
  })
  return e;
}

}  // namespace kmip
