// kmip_ffn_f32.cu -- the gated feed-forward block for fp32 inputs.
//
// The products run as fp32 fused multiply-adds, like the fp32 attention: the
// tensor cores' accumulation truncates (1e-6 of the result after 1,024 terms,
// 2e-5 after 32,768, measured with exact products), which is worse than fp32
// arithmetic would be, however the operands are split.
//
// Two kernels.  ffn_f32_glu computes a = x Wg^T and b = x Wu^T of a tile of at
// most 64 x 64 (backward: dh = dy Wd too) and writes h, or dA, dB and h: no launch and
// no memory between the products and the activation.  ffn_f32_gemm computes
// up to three independent products of a kind (y; dx as two contractions in a
// row; the three weight gradients), with tiles of 128 x 128 or 64 x 64; few
// tiles split the contraction, and a third kernel adds the parts in order.
//
// Both: 16 x 16 threads; cp.async brings steps of 16 contraction indices into
// a ring of kStages shared buffers, each operand as it lies in memory.  A
// thread holds the fragments of one side for four indices and streams the
// other's, 16 bytes a shared load either way.  Bound: the FMA pipe for large
// sizes; launches and the length of the contraction for small ones.
#include "kmip_act.cuh"
#include "kmip_ffn.h"
#include "kmip_launch.cuh"

namespace kmip {
namespace {

constexpr int kBK = 16;
constexpr int kThreads = 256;
constexpr int kStages = 4;
constexpr int kPitch = kBK + 4;  // of a row of contraction indices: no bank conflicts

__device__ __forceinline__ void copy16(uint32_t dst, const float* src, bool on) {
  // (nothing is read when off: 16 zero bytes)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
}

// An operand's step in shared memory: [TM][kPitch] when the contraction is
// innermost (KIN), else [kBK][TM + 4].
template <int TM>
constexpr int kStepFloats = TM * kPitch;
static_assert(kStepFloats<32> >= kBK * (32 + 4) && kStepFloats<128> >= kBK * (128 + 4));

// Starts the copies of elements (k, i), k0 <= k < K, i0 <= i < extent; the
// innermost extent is a multiple of 4.
template <int TM, bool KIN>
__device__ __forceinline__ void copy_step(uint32_t dst, const float* src, int64_t ld, int i0,
                                          int extent, int k0, int K) {
  constexpr int kVecs = TM * kBK / 4;
#pragma unroll
  for (int t = 0; t < (kVecs + kThreads - 1) / kThreads; ++t) {
    const int id = t * kThreads + threadIdx.x;
    if (kVecs < kThreads && id >= kVecs) break;
    const int i = KIN ? id / (kBK / 4) : id % (TM / 4) * 4;
    const int k = KIN ? id % (kBK / 4) * 4 : id / (TM / 4);
    const bool on = i0 + i < extent && k0 + k < K;
    const float* at =
        src + (KIN ? (int64_t)(i0 + i) * ld + k0 + k : (int64_t)(k0 + k) * ld + i0 + i);
    copy16(dst + (KIN ? i * kPitch + k : k * (TM + 4) + i) * 4, on ? at : src, on);
  }
}

// Element r of thread t on one side is row (of the tile)
template <bool KIN>
__device__ __forceinline__ int row_of(int r, int t) {
  return KIN ? r * 16 + t : r / 4 * 64 + t * 4 + r % 4;
}

// f[e][kk] = element (k + kk, row_of(r0 + e)), e < E (4 where !KIN).
template <int TM, bool KIN, int E>
__device__ __forceinline__ void four_steps(const float* s, int k, int r0, int t,
                                           float (&f)[E][4]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (KIN) {
      *reinterpret_cast<float4*>(f[e]) =
          *reinterpret_cast<const float4*>(s + ((r0 + e) * 16 + t) * kPitch + k);
    } else {  // e runs over the contraction here
      const float4 v =
          *reinterpret_cast<const float4*>(s + (k + e) * (TM + 4) + r0 * 16 + t * 4);
      f[0][e] = v.x;
      f[1][e] = v.y;
      f[2][e] = v.z;
      f[3][e] = v.w;
    }
  }
}

// out [M, N] = sum over segments of A_s B_s; element (m, k) of A is at
// m lda + k when the contraction is innermost, else at k lda + m; B likewise.
struct Product {
  const float *a[2], *b[2];
  int K[2];
  int segs;
  int M, N;
  int64_t lda, ldb;
  float* out;
};

struct Products {
  Product q[3];
  int tile0[4];      // first tile of each product
  int count;
  int splits;
  float* part;       // splits > 1: [splits][elements of all products]
  int64_t elems[4];  // first element of each product in a part
};

template <int TM>
constexpr int gemm_smem() { return kStages * 2 * kStepFloats<TM> * 4; }

template <int TM, bool AKIN, bool BKIN>
__global__ void __launch_bounds__(kThreads, 2) ffn_f32_gemm(const Products ps) {
  after_previous();
  constexpr int R = TM / 16;  // outputs of a thread per side
  extern __shared__ float4 dyn[];
  float* buffers = reinterpret_cast<float*>(dyn);  // [kStages][A, B]
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(buffers));
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

  auto fetch = [&](int s) {
    if (s < s1) {
      const int seg = s >= steps0, k0 = (seg ? s - steps0 : s) * kBK;
      const uint32_t dst = base + (s % kStages) * 2 * kStepFloats<TM> * 4;
      copy_step<TM, AKIN>(dst, q.a[seg], q.lda, m0, q.M, k0, q.K[seg]);
      copy_step<TM, BKIN>(dst + kStepFloats<TM> * 4, q.b[seg], q.ldb, n0, q.N, k0, q.K[seg]);
    }
    copy_commit();
  };
  for (int s = 0; s < kStages - 1; ++s) fetch(s0 + s);
  for (int s = s0; s < s1; ++s) {
    copy_wait();
    __syncthreads();  // step s has landed; step s - 1 has been used by all
    fetch(s + kStages - 1);
    const float* sa = buffers + (s % kStages) * 2 * kStepFloats<TM>;
    const float* sb = sa + kStepFloats<TM>;
#pragma unroll
    for (int k = 0; k < kBK; k += 4) {
      float b[R / 4][4][4];
#pragma unroll
      for (int j = 0; j < R / 4; ++j) four_steps<TM, BKIN, 4>(sb, k, 4 * j, tx, b[j]);
#pragma unroll
      for (int i = 0; i < R / 4; ++i) {
        float a[4][4];
        four_steps<TM, AKIN, 4>(sa, k, 4 * i, ty, a);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < R; ++j)
              acc[4 * i + e][j] = fmaf(a[e][kk], b[j / 4][j % 4][kk], acc[4 * i + e][j]);
      }
    }
  }
  float* out = ps.splits > 1 ? ps.part + blockIdx.y * ps.elems[ps.count] + ps.elems[pi] : q.out;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = m0 + row_of<AKIN>(i, ty);
    if (m >= q.M) continue;
#pragma unroll
    for (int j = 0; j < R; j += BKIN ? 1 : 4) {
      const int n = n0 + row_of<BKIN>(j, tx);
      if (n >= q.N) continue;
      float* at = out + (int64_t)m * q.N + n;
      if constexpr (BKIN)
        *at = acc[i][j];
      else
        *reinterpret_cast<float4*>(at) =
            make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
    }
  }
}

__global__ void __launch_bounds__(kThreads) ffn_f32_join(const Products ps) {
  after_previous();
  const int64_t total = ps.elems[ps.count];
  for (int64_t i = (blockIdx.x * (int64_t)kThreads + threadIdx.x) * 4; i < total;
       i += (int64_t)gridDim.x * kThreads * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
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

// h = act(a) * b; BWD: dA, dB, h.  Tiles of 16 R x 16 Q of [N, F].
template <int ACT, bool BWD, int R, int Q>
__global__ void __launch_bounds__(kThreads, 2)
ffn_f32_glu(const float* x, const float* wg, const float* wu, const float* dy, const float* wd,
            int N, int C, int F, float* da, float* db, float* h) {
  after_previous();
  constexpr int TM = 16 * R, TN = 16 * Q;
  constexpr int kFloatsM = kStepFloats<TM>, kFloatsN = kStepFloats<TN>;
  constexpr int kBuf = kFloatsM + 2 * kFloatsN;  // x, Wg, Wu; or dy, Wd
  extern __shared__ float4 dyn[];
  float* buffers = reinterpret_cast<float*>(dyn);
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(buffers));
  const int tiles_n = (F + TN - 1) / TN;
  const int m0 = blockIdx.x / tiles_n * TM, n0 = blockIdx.x % tiles_n * TN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int steps = (C + kBK - 1) / kBK, all = BWD ? 2 * steps : steps;

  float g[R][Q], u[R][Q], d[R][Q];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < Q; ++j) g[i][j] = u[i][j] = d[i][j] = 0.f;

  auto fetch = [&](int s) {
    if (s < all) {
      const uint32_t dst = base + (s % kStages) * kBuf * 4;
      if (s < steps) {
        copy_step<TM, true>(dst, x, C, m0, N, s * kBK, C);
        copy_step<TN, true>(dst + kFloatsM * 4, wg, C, n0, F, s * kBK, C);
        copy_step<TN, true>(dst + (kFloatsM + kFloatsN) * 4, wu, C, n0, F, s * kBK, C);
      } else if (BWD) {
        copy_step<TM, true>(dst, dy, C, m0, N, (s - steps) * kBK, C);
        copy_step<TN, false>(dst + kFloatsM * 4, wd, F, n0, F, (s - steps) * kBK, C);
      }
    }
    copy_commit();
  };
  for (int s = 0; s < kStages - 1; ++s) fetch(s);
  for (int s = 0; s < all; ++s) {
    copy_wait();
    __syncthreads();
    fetch(s + kStages - 1);
    const float* sa = buffers + (s % kStages) * kBuf;
    const float* sg = sa + kFloatsM;
    const float* su = sg + kFloatsN;
    if (s < steps) {
#pragma unroll
      for (int k = 0; k < kBK; k += 4) {
        float a[R][4], b[Q][4], c[Q][4];
        four_steps<TM, true, R>(sa, k, 0, ty, a);
        four_steps<TN, true, Q>(sg, k, 0, tx, b);
        four_steps<TN, true, Q>(su, k, 0, tx, c);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < Q; ++j) {
              g[i][j] = fmaf(a[i][kk], b[j][kk], g[i][j]);
              u[i][j] = fmaf(a[i][kk], c[j][kk], u[i][j]);
            }
      }
    } else if (BWD) {
#pragma unroll
      for (int k = 0; k < kBK; k += 4) {
        float a[R][4];
        four_steps<TM, true, R>(sa, k, 0, ty, a);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float b[Q];  // columns as in the first products: j * 16 + tx
#pragma unroll
          for (int j = 0; j < Q; ++j) b[j] = sg[(k + kk) * (TN + 4) + j * 16 + tx];
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < Q; ++j) d[i][j] = fmaf(a[i][kk], b[j], d[i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = m0 + i * 16 + ty;
    if (m >= N) continue;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int n = n0 + j * 16 + tx;
      if (n >= F) continue;
      const int64_t at = (int64_t)m * F + n;
      if (BWD) {
        float f, slope;
        act_both<float, ACT>(g[i][j], f, slope);
        da[at] = d[i][j] * u[i][j] * slope;
        db[at] = d[i][j] * f;
        h[at] = f * u[i][j];
      } else {
        h[at] = act_value<float, ACT>(g[i][j]) * u[i][j];
      }
    }
  }
}

int64_t glu_tiles(const FfnArgs& a, int R, int Q) {
  return (int64_t)((a.N + 16 * R - 1) / (16 * R)) * ((a.F + 16 * Q - 1) / (16 * Q));
}

template <int ACT, bool BWD, int R, int Q>
cudaError_t launch_glu(const FfnArgs& a, const float* dy, float* da, float* db, float* h,
                       cudaStream_t stream) {
  constexpr int smem = kStages * (kStepFloats<16 * R> + 2 * kStepFloats<16 * Q>) * 4;
  const auto f = [](const void* p) { return static_cast<const float*>(p); };
  auto kern = ffn_f32_glu<ACT, BWD, R, Q>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)glu_tiles(a, R, Q), kThreads, smem, stream>>>(
      f(a.x), f(a.wg), f(a.wu), dy, f(a.wd), a.N, a.C, a.F, da, db, h);
  return cudaGetLastError();
}

// A step of a 64 x 64 tile keeps an SM's FMA pipe busy for 0.55 us, so few
// tiles are made smaller until they fill the SMs.
template <bool BWD>
cudaError_t glu(const FfnArgs& a, const float* dy, float* da, float* db, float* h,
                cudaStream_t stream) {
  const int64_t enough = device_sm_count() * 3 / 2;
  cudaError_t e = cudaSuccess;
  KMIP_ACT_SWITCH(a.act, {
    if (glu_tiles(a, 4, 4) >= enough)
      e = launch_glu<ACT, BWD, 4, 4>(a, dy, da, db, h, stream);
    else if (glu_tiles(a, 4, 2) >= enough)
      e = launch_glu<ACT, BWD, 4, 2>(a, dy, da, db, h, stream);
    else
      e = launch_glu<ACT, BWD, 2, 2>(a, dy, da, db, h, stream);
  })
  return e;
}

constexpr int kMaxSplits = 16;

Product product(const float* a, int64_t lda, const float* b, int64_t ldb, int M, int N, int K,
                float* out) {
  Product q{};
  q.a[0] = a;
  q.b[0] = b;
  q.K[0] = K;
  q.segs = 1;
  q.M = M;
  q.N = N;
  q.lda = lda;
  q.ldb = ldb;
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

// Parts for products of few tiles: of at most two blocks an SM.
int64_t part_elems_of() { return (int64_t)2 * device_sm_count() * 64 * 64 * 2; }

template <int TM, bool AKIN, bool BKIN>
cudaError_t launch(const Products& ps, cudaStream_t stream) {
  auto kern = ffn_f32_gemm<TM, AKIN, BKIN>;
  const cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm_smem<TM>());
  if (e != cudaSuccess) return e;
  return launch_next(kern, dim3(ps.tile0[ps.count], ps.splits), kThreads, gemm_smem<TM>(), stream,
                     ps);
}

template <bool AKIN, bool BKIN>
cudaError_t run(Products& ps, float* part, cudaStream_t stream) {
  const int tm = plan(ps, part_elems_of());
  ps.part = part;
  const cudaError_t e = tm == 128 ? launch<128, AKIN, BKIN>(ps, stream)
                                  : launch<64, AKIN, BKIN>(ps, stream);
  if (e != cudaSuccess) return e;
  if (ps.splits > 1) {
    const int64_t n4 = (ps.elems[ps.count] + 3) / 4, most = (int64_t)device_sm_count() * 8;
    const int64_t want = (n4 + kThreads - 1) / kThreads;
    return launch_next(ffn_f32_join, dim3((unsigned)(want < most ? want : most)), kThreads, 0,
                       stream, ps);
  }
  return cudaSuccess;
}

}  // namespace

size_t ffn_f32_scratch() { return sizeof(float) * (size_t)part_elems_of(); }

cudaError_t launch_ffn_f32_fwd(const FfnArgs& a, float* h, float* y, float* part,
                               cudaStream_t stream) {
  const cudaError_t e = glu<false>(a, nullptr, nullptr, nullptr, h, stream);
  if (e != cudaSuccess) return e;
  Products ps{};
  ps.count = 1;
  ps.q[0] = product(h, a.F, static_cast<const float*>(a.wd), a.F, a.N, a.C, a.F, y);
  return run<true, true>(ps, part, stream);
}

cudaError_t launch_ffn_f32_bwd(const FfnArgs& a, const float* dy, float* abd, float* dx,
                               float* dwg, float* dwu, float* dwd, float* part,
                               cudaStream_t stream) {
  const auto f = [](const void* p) { return static_cast<const float*>(p); };
  const int64_t nf = (int64_t)a.N * a.F;
  float *da = abd, *db = abd + nf, *h = abd + 2 * nf;
  cudaError_t e = glu<true>(a, dy, da, db, h, stream);
  if (e != cudaSuccess) return e;
  Products px{};
  px.count = 1;
  px.q[0] = product(da, a.F, f(a.wg), a.C, a.N, a.C, a.F, dx);
  px.q[0].segs = 2;
  px.q[0].a[1] = db;
  px.q[0].b[1] = f(a.wu);
  px.q[0].K[1] = a.F;
  e = run<true, false>(px, part, stream);
  if (e != cudaSuccess) return e;
  Products pw{};
  pw.count = 3;
  pw.q[0] = product(da, a.F, f(a.x), a.C, a.F, a.C, a.N, dwg);
  pw.q[1] = product(db, a.F, f(a.x), a.C, a.F, a.C, a.N, dwu);
  pw.q[2] = product(dy, a.C, h, a.F, a.C, a.F, a.N, dwd);
  return run<false, false>(pw, part, stream);
}

}  // namespace kmip
