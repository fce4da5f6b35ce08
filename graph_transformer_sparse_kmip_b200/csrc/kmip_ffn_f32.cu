// kmip_ffn_f32.cu -- the gated feed-forward block for fp32 inputs.
//
// The products run as fp32 fused multiply-adds, like the fp32 attention: the
// tensor cores' accumulation truncates (1e-6 of the result after 1,024 terms,
// 2e-5 after 32,768, measured with exact products), which is worse than fp32
// arithmetic would be, however the operands are split.
//
// One tiled GEMM serves all products: a block computes a TM x TM tile over a
// range of the contraction, 16 x 16 threads with (TM / 16)^2 outputs each,
// tiles double-buffered in shared memory with the next step's loads in
// registers.  A launch holds up to three independent products (a, b and dh;
// the three weight gradients).  Bound: the FMA pipe for large sizes; launches
// and the length of the contraction for small ones, so products with few
// tiles split it, and a second kernel adds the parts in order.
#include "kmip_act.cuh"
#include "kmip_ffn.h"

namespace kmip {
namespace {

constexpr int kBK = 16;
constexpr int kThreads = 256;

// out [M, N] = sum over segments of A_s B_s; element (m, k) of A is at
// m lda + k when a_k (k contiguous), else at k lda + m; B likewise with n.
struct Product {
  const float *a[2], *b[2];
  int K[2];
  int segs;
  int M, N;
  int64_t lda, ldb;
  bool a_k, b_k;
  float* out;
};

struct Products {
  Product q[3];
  int tile0[4];   // first tile of each product
  int count;
  int splits;
  float* part;    // splits > 1: [splits][elements of all products]
  int64_t elems[4];  // first element of each product in a part
};

// Loads a [kBK, TM] step of an operand: element (k, i), i < extent, k < K.
template <int TM>
struct Loader {
  static constexpr int kVecs = TM * kBK / 4 / kThreads;
  float4 v[kVecs];
  __device__ void load(const float* src, int64_t ld, bool k_contig, int i0, int extent, int k0,
                       int k1) {
#pragma unroll
    for (int t = 0; t < kVecs; ++t) {
      const int id = t * kThreads + threadIdx.x;
      v[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k_contig) {
        const int i = i0 + id / (kBK / 4), k = k0 + id % (kBK / 4) * 4;
        if (i < extent && k < k1)
          v[t] = *reinterpret_cast<const float4*>(src + (int64_t)i * ld + k);
      } else {
        const int k = k0 + id / (TM / 4), i = i0 + id % (TM / 4) * 4;
        if (i < extent && k < k1)
          v[t] = *reinterpret_cast<const float4*>(src + (int64_t)k * ld + i);
      }
    }
  }
  __device__ void store(float (*s)[TM + 4], bool k_contig) const {
#pragma unroll
    for (int t = 0; t < kVecs; ++t) {
      const int id = t * kThreads + threadIdx.x;
      if (k_contig) {
        const int i = id / (kBK / 4), k = id % (kBK / 4) * 4;
        s[k][i] = v[t].x;
        s[k + 1][i] = v[t].y;
        s[k + 2][i] = v[t].z;
        s[k + 3][i] = v[t].w;
      } else {
        const int k = id / (TM / 4), i = id % (TM / 4) * 4;
        *reinterpret_cast<float4*>(&s[k][i]) = v[t];
      }
    }
  }
};

template <int TM>
__global__ void __launch_bounds__(kThreads) ffn_f32_gemm(const Products ps) {
  constexpr int R = TM / 16;  // outputs of a thread per side, in runs of 4
  __shared__ float sa[2][kBK][TM + 4], sb[2][kBK][TM + 4];
  int pi = 0;
  while (pi + 1 < ps.count && (int)blockIdx.x >= ps.tile0[pi + 1]) ++pi;
  const Product& q = ps.q[pi];
  const int tiles_n = (q.N + TM - 1) / TM, tile = blockIdx.x - ps.tile0[pi];
  const int m0 = tile / tiles_n * TM, n0 = tile % tiles_n * TM;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

  // this block's steps: an equal share of the steps of both segments
  const int steps0 = (q.K[0] + kBK - 1) / kBK;
  const int steps = steps0 + (q.segs > 1 ? (q.K[1] + kBK - 1) / kBK : 0);
  const int s0 = (int)((int64_t)steps * blockIdx.y / ps.splits);
  const int s1 = (int)((int64_t)steps * (blockIdx.y + 1) / ps.splits);

  float acc[R][R];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] = 0.f;

  Loader<TM> la, lb;
  auto fetch = [&](int s) {
    const int seg = s >= steps0, k0 = (seg ? s - steps0 : s) * kBK;
    la.load(q.a[seg], q.lda, q.a_k, m0, q.M, k0, q.K[seg]);
    lb.load(q.b[seg], q.ldb, q.b_k, n0, q.N, k0, q.K[seg]);
  };
  if (s0 < s1) fetch(s0);
  for (int s = s0; s < s1; ++s) {
    const int buf = (s - s0) & 1;
    la.store(sa[buf], q.a_k);
    lb.store(sb[buf], q.b_k);
    __syncthreads();
    if (s + 1 < s1) fetch(s + 1);
#pragma unroll
    for (int k = 0; k < kBK; ++k) {
      float a[R], b[R];
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        *reinterpret_cast<float4*>(a + i) =
            *reinterpret_cast<const float4*>(&sa[buf][k][i * 16 + ty * 4]);
        *reinterpret_cast<float4*>(b + i) =
            *reinterpret_cast<const float4*>(&sb[buf][k][i * 16 + tx * 4]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
  }
  float* out = ps.splits > 1 ? ps.part + blockIdx.y * ps.elems[ps.count] + ps.elems[pi] : q.out;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = m0 + i / 4 * 64 + ty * 4 + i % 4;
    if (m >= q.M) continue;
#pragma unroll
    for (int j = 0; j < R; j += 4) {
      const int n = n0 + j * 16 + tx * 4;  // N is a multiple of 4
      if (n < q.N)
        *reinterpret_cast<float4*>(out + (int64_t)m * q.N + n) =
            make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
    }
  }
}

__global__ void __launch_bounds__(kThreads) ffn_f32_join(const Products ps) {
  const int64_t total = ps.elems[ps.count];
  for (int64_t i = (blockIdx.x * (int64_t)kThreads + threadIdx.x) * 4; i < total;
       i += (int64_t)gridDim.x * kThreads * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = 0; t < ps.splits; ++t) {
      const float4 v = *reinterpret_cast<const float4*>(ps.part + t * total + i);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    int pi = 0;
    while (pi + 1 < ps.count && i >= ps.elems[pi + 1]) ++pi;
    *reinterpret_cast<float4*>(ps.q[pi].out + (i - ps.elems[pi])) = s;
  }
}

// h = act(a) * b, over a; with dh: da over a, db over b, h over dh.
template <int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads) ffn_f32_glu(float4* a, float4* b, float4* dh,
                                                        int64_t n4) {
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < n4;
       i += (int64_t)gridDim.x * kThreads) {
    float4 va = a[i], vb = b[i], vd = BWD ? dh[i] : va;
    float* pa = &va.x;
    float* pb = &vb.x;
    float* pd = &vd.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (BWD) {
        float f, g;
        act_both<float, ACT>(pa[e], f, g);
        const float d = pd[e], u = pb[e];
        pa[e] = d * u * g;
        pb[e] = d * f;
        pd[e] = f * u;
      } else {
        pa[e] = act_value<float, ACT>(pa[e]) * pb[e];
      }
    }
    a[i] = va;
    if (BWD) {
      b[i] = vb;
      dh[i] = vd;
    }
  }
}

template <bool BWD>
cudaError_t glu(int act, float* a, float* b, float* dh, int64_t n, cudaStream_t stream) {
  const int64_t n4 = n / 4, most = (int64_t)device_sm_count() * 8;
  const int64_t want = (n4 + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)(want < most ? want : most);
  float4 *pa = reinterpret_cast<float4*>(a), *pb = reinterpret_cast<float4*>(b),
         *pd = reinterpret_cast<float4*>(dh);
  KMIP_ACT_SWITCH(act, ffn_f32_glu<ACT, BWD><<<grid, kThreads, 0, stream>>>(pa, pb, pd, n4))
  return cudaGetLastError();
}

constexpr int kMaxSplits = 16;

Product product(const float* a, bool a_k, const float* b, bool b_k, int M, int N, int K,
                float* out) {
  Product q{};
  q.a[0] = a;
  q.b[0] = b;
  q.K[0] = K;
  q.segs = 1;
  q.M = M;
  q.N = N;
  q.a_k = a_k;
  q.b_k = b_k;
  q.lda = a_k ? K : M;
  q.ldb = b_k ? K : N;
  q.out = out;
  return q;
}

// Tile size and splits of a launch; `part_elems` of scratch may be used.
int plan(Products& ps, int64_t part_elems) {
  const int sms = device_sm_count();
  int tm = 128;
  int64_t tiles = 0;
  int steps = 0;
  for (;; tm = 64) {
    tiles = 0;
    steps = 0;
    ps.elems[0] = 0;
    for (int i = 0; i < ps.count; ++i) {
      const Product& q = ps.q[i];
      ps.tile0[i] = (int)tiles;
      tiles += (int64_t)((q.M + tm - 1) / tm) * ((q.N + tm - 1) / tm);
      ps.elems[i + 1] = ps.elems[i] + (int64_t)q.M * q.N;
      int s = 0;
      for (int g = 0; g < q.segs; ++g) s += (q.K[g] + kBK - 1) / kBK;
      if (s > steps) steps = s;
    }
    // the wide tile wants a block for every SM
    if (tm == 64 || tiles >= sms) break;
  }
  ps.tile0[ps.count] = (int)tiles;
  // two blocks an SM, at least eight steps each
  int64_t splits = 2 * sms / tiles;
  if (splits > steps / 8) splits = steps / 8;
  if (splits > kMaxSplits) splits = kMaxSplits;
  while (splits > 1 && splits * ps.elems[ps.count] > part_elems) --splits;
  ps.splits = splits < 1 ? 1 : (int)splits;
  return tm;
}

cudaError_t run(Products& ps, float* part, int64_t part_elems, cudaStream_t stream) {
  const int tm = plan(ps, part_elems);
  ps.part = part;
  const dim3 grid(ps.tile0[ps.count], ps.splits);
  if (tm == 128)
    ffn_f32_gemm<128><<<grid, kThreads, 0, stream>>>(ps);
  else
    ffn_f32_gemm<64><<<grid, kThreads, 0, stream>>>(ps);
  if (ps.splits > 1) {
    const int64_t n4 = (ps.elems[ps.count] + 3) / 4, most = (int64_t)device_sm_count() * 8;
    const int64_t want = (n4 + kThreads - 1) / kThreads;
    ffn_f32_join<<<(unsigned)(want < most ? want : most), kThreads, 0, stream>>>(ps);
  }
  return cudaGetLastError();
}

// Parts for products of few tiles: of at most two blocks an SM.
int64_t part_elems_of() { return (int64_t)2 * device_sm_count() * 64 * 64 * 2; }

}  // namespace

size_t ffn_f32_scratch() { return sizeof(float) * (size_t)part_elems_of(); }

// ab: [2][N, F] scratch for a and b.
cudaError_t launch_ffn_f32_fwd(const FfnArgs& a, float* ab, float* y, float* part,
                               cudaStream_t stream) {
  const auto f = [](const void* p) { return static_cast<const float*>(p); };
  const int64_t nf = (int64_t)a.N * a.F;
  Products ps{};
  ps.count = 2;
  ps.q[0] = product(f(a.x), true, f(a.wg), true, a.N, a.F, a.C, ab);
  ps.q[1] = product(f(a.x), true, f(a.wu), true, a.N, a.F, a.C, ab + nf);
  cudaError_t e = run(ps, part, part_elems_of(), stream);
  if (e == cudaSuccess) e = glu<false>(a.act, ab, ab + nf, nullptr, nf, stream);
  if (e != cudaSuccess) return e;
  Products pd{};
  pd.count = 1;
  pd.q[0] = product(ab, true, f(a.wd), true, a.N, a.C, a.F, y);
  return run(pd, part, part_elems_of(), stream);
}

// abd: [3][N, F] scratch for a, b, dh, then dA, dB, h.
cudaError_t launch_ffn_f32_bwd(const FfnArgs& a, const float* dy, float* abd, float* dx,
                               float* dwg, float* dwu, float* dwd, float* part,
                               cudaStream_t stream) {
  const auto f = [](const void* p) { return static_cast<const float*>(p); };
  const int64_t nf = (int64_t)a.N * a.F;
  float *da = abd, *db = abd + nf, *h = abd + 2 * nf;
  Products ps{};
  ps.count = 3;
  ps.q[0] = product(f(a.x), true, f(a.wg), true, a.N, a.F, a.C, da);
  ps.q[1] = product(f(a.x), true, f(a.wu), true, a.N, a.F, a.C, db);
  ps.q[2] = product(dy, true, f(a.wd), false, a.N, a.F, a.C, h);
  cudaError_t e = run(ps, part, part_elems_of(), stream);
  if (e == cudaSuccess) e = glu<true>(a.act, da, db, h, nf, stream);
  if (e != cudaSuccess) return e;
  Products px{};
  px.count = 1;
  px.q[0] = product(da, true, f(a.wg), false, a.N, a.C, a.F, dx);
  px.q[0].segs = 2;
  px.q[0].a[1] = db;
  px.q[0].b[1] = f(a.wu);
  px.q[0].K[1] = a.F;
  e = run(px, part, part_elems_of(), stream);
  if (e != cudaSuccess) return e;
  Products pw{};
  pw.count = 3;
  pw.q[0] = product(da, false, f(a.x), false, a.F, a.C, a.N, dwg);
  pw.q[1] = product(db, false, f(a.x), false, a.F, a.C, a.N, dwu);
  pw.q[2] = product(dy, false, h, false, a.C, a.F, a.N, dwd);
  return run(pw, part, part_elems_of(), stream);
}

}  // namespace kmip
