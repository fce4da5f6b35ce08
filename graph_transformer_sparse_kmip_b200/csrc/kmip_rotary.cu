// kmip_rotary.cu -- rotary positions with several axes (kmip_rotary).
//
// Point clouds and superpixel graphs (the workloads of k-Maximum Inner
// Product Attention for Graph Transformers ..., Tables 2, 3 and 13) place
// their nodes by two or three coordinates.  Pair p of a head turns by
//   angle = pos[n, axis[p]] * freq[p]
// so that the inner product of a turned query and key depends on the
// difference of their coordinates only.
//
// Angles: the product is taken in fp64 in units of one revolution and reduced
// to [-1/2, 1/2] there, so that far positions keep their angle (an fp32
// product of 2e5 rad is off by 8e-3 rad); the reduced angle is rounded to fp32
// (off by at most 2^-25 revolutions) and goes through sincospif.
//
// Bound: HBM traffic, one read and one write of x.  The angles of a node are
// the same for all of its heads: a block computes those of its nodes once
// into shared memory while its loads of x are in flight, so the sine and
// cosine cost 1 / H of a per-element evaluation.
#include "kmip_internal.h"

namespace kmip {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;         // units in flight per thread
constexpr int kMaxTable = 2048;   // cos/sin pairs a block keeps (16 KiB)

struct RotaryParams {
  const void* x;
  void* out;
  int64_t x_row, x_head, out_row, out_head;  // strides in elements
  const void* pos;
  const double* freq;
  const int32_t* axis;
  int64_t N;
  int H, d, pairs, axes;
  int nodes;        // nodes per block
  int chunks;       // units per head
  int interleaved;
  float sign;       // -1: inverse rotation
  int copy_tail;    // 0: in place, elements behind the pairs stay
  int* status;
};

// V elements as one load or store.
template <int BYTES>
struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
struct Pack {
  using R = typename Raw<sizeof(T) * V>::type;
  union {
    R raw;
    T e[V];
  };
  __device__ Pack() {}
  __device__ void load(const T* p) { raw = *reinterpret_cast<const R*>(p); }
  __device__ void store(T* p) const { *reinterpret_cast<R*>(p) = raw; }
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float& d, float v) { d = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ void turn(T& u, T& v, float2 cs) {
  const float a = widen(u), b = widen(v);
  narrow(u, fmaf(a, cs.x, -b * cs.y));
  narrow(v, fmaf(a, cs.y, b * cs.x));
}

// A unit is what one thread turns at a time: with halves, V pairs (p, p + P)
// or V elements behind them; interleaved, V elements (V / 2 pairs).
template <typename T, int V, typename PosT, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 table[];  // [nodes][pairs]
  const int64_t n0 = (int64_t)blockIdx.x * p.nodes;
  const int nodes = (int)min((int64_t)p.nodes, p.N - n0);
  const int per_node = p.H * p.chunks;
  const int units = nodes * per_node;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  const int rot_chunks = INTER ? p.chunks : p.pairs / V;
  bool have_table = false;

  for (int base = 0; base < units; base += kBatch * kThreads) {
    Pack<T, V> a[kBatch], b[kBatch];
    int at[kBatch];        // (node << 16) | chunk, -1 = none
    int64_t dst[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const int i = base + t * kThreads + threadIdx.x;
      at[t] = -1;
      if (i < units) {
        const int node = i / per_node, r = i - node * per_node;
        const int head = r / p.chunks, c = r - head * p.chunks;
        const bool pair = c < rot_chunks;
        if (pair || p.copy_tail) {
          // tail chunks (halves only) start behind both halves
          const int e = pair ? c * V : 2 * p.pairs + (c - rot_chunks) * V;
          const T* src = x + (n0 + node) * p.x_row + head * p.x_head + e;
          dst[t] = (n0 + node) * p.out_row + head * p.out_head + e;
          a[t].load(src);
          if (!INTER && pair) b[t].load(src + p.pairs);
          at[t] = (node << 16) | c;
        }
      }
    }
    if (!have_table) {
      have_table = true;
      for (int i = threadIdx.x; i < nodes * p.pairs; i += kThreads) {
        const int node = i / p.pairs, q = i - node * p.pairs;
        const int ax = p.axis[q];
        double rev = 0.0;
        if ((unsigned)ax < (unsigned)p.axes)
          rev = (double)static_cast<const PosT*>(p.pos)[(n0 + node) * p.axes + ax] *
                (p.freq[q] * 0.15915494309189535);  // 1 / (2 pi)
        else
          record_status(p.status, KMIP_ERR_BAD_INDEX);
        const float half_turns = (float)(2.0 * (rev - rint(rev)));
        float2 cs;
        sincospif(half_turns, &cs.y, &cs.x);
        cs.y *= p.sign;
        table[i] = cs;
      }
      __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      if (at[t] < 0) continue;
      const int c = at[t] & 0xffff;
      const float2* cs = table + (at[t] >> 16) * p.pairs;
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const int q = c * (V / 2) + e;
          if (q < p.pairs) turn(a[t].e[2 * e], a[t].e[2 * e + 1], cs[q]);
        }
        a[t].store(out + dst[t]);
      } else {
        if (c < rot_chunks) {
#pragma unroll
          for (int e = 0; e < V; ++e) turn(a[t].e[e], b[t].e[e], cs[c * V + e]);
          b[t].store(out + dst[t] + p.pairs);
        }
        a[t].store(out + dst[t]);
      }
    }
  }
}

template <typename T, int V, typename PosT, bool INTER>
cudaError_t launch(RotaryParams p, cudaStream_t stream) {
  // interleaved units are V elements; with halves the pairs and the tail
  // each make whole units
  p.chunks = INTER ? p.d / V : p.pairs / V + (p.d - 2 * p.pairs) / V;
  const int per_node = p.H * p.chunks;
  int nodes = kBatch * kThreads / per_node;
  if (p.pairs && nodes > kMaxTable / p.pairs) nodes = kMaxTable / p.pairs;
  // few nodes: one per block, so that more SMs share the latency
  if (nodes > (p.N + 591) / 592) nodes = (int)((p.N + 591) / 592);
  p.nodes = nodes < 1 ? 1 : nodes;
  const int64_t blocks = (p.N + p.nodes - 1) / p.nodes;
  const size_t smem = sizeof(float2) * (size_t)p.nodes * p.pairs;
  rotary_kernel<T, V, PosT, INTER><<<(unsigned)blocks, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, typename PosT>
cudaError_t launch_layout(const RotaryParams& p, cudaStream_t stream) {
  if constexpr (V >= 2) {
    if (p.interleaved) return launch<T, V, PosT, true>(p, stream);
  }
  return launch<T, V, PosT, false>(p, stream);
}

template <typename T, int V>
cudaError_t launch_pos(const RotaryParams& p, kmip_pos_t pos_type, cudaStream_t stream) {
  switch (pos_type) {
    case KMIP_POS_F32: return launch_layout<T, V, float>(p, stream);
    case KMIP_POS_I32: return launch_layout<T, V, int32_t>(p, stream);
    default: return launch_layout<T, V, int64_t>(p, stream);
  }
}

// The widest unit that every row, head and part of a head is a multiple of.
// (Interleaved pairs are two elements: their unit is at least 2 elements,
// moved as one load where the strides allow it.)
template <typename T>
int unit_width(const RotaryParams& p) {
  int v = 16 / (int)sizeof(T);
  auto fits = [&](int w) {
    const uint64_t bytes = w * sizeof(T);
    if (reinterpret_cast<uintptr_t>(p.x) % bytes || reinterpret_cast<uintptr_t>(p.out) % bytes)
      return false;
    if (p.x_row % w || p.x_head % w || p.out_row % w || p.out_head % w) return false;
    return p.interleaved ? p.d % w == 0 : p.pairs % w == 0 && (p.d - 2 * p.pairs) % w == 0;
  };
  while (v > 1 && !fits(v)) v /= 2;
  return v;
}

}  // namespace
}  // namespace kmip

using namespace kmip;

extern "C" __attribute__((visibility("default"))) kmip_status_t kmip_rotary(
    const void* x, int64_t x_row, int64_t x_head, const void* pos, kmip_pos_t pos_type, int axes,
    const double* freq, const int32_t* axis, int pairs, int interleaved, int inverse, int64_t N,
    int H, int d, void* out, int64_t out_row, int64_t out_head, kmip_stream_t stream_,
    kmip_dtype_t dtype) {
  if (N < 0 || N > INT32_MAX || H < 1 || d < 2 || axes < 1 || pairs < 0 || x_row < 0 ||
      x_head < 0 || out_row < 0 || out_head < 0)
    return KMIP_ERR_INVALID_ARG;
  if (dtype != KMIP_BF16 && dtype != KMIP_F32) return KMIP_ERR_INVALID_ARG;
  if (pos_type != KMIP_POS_F32 && pos_type != KMIP_POS_I32 && pos_type != KMIP_POS_I64)
    return KMIP_ERR_INVALID_ARG;
  if (d % 2 || d > 512 || H > 4096 || axes > 64) return KMIP_ERR_UNSUPPORTED;
  if (2 * pairs > d) return KMIP_ERR_INVALID_ARG;
  if (N == 0) return KMIP_OK;
  if (!x || !out || !pos || (pairs && (!freq || !axis))) return KMIP_ERR_INVALID_ARG;
  const bool in_place = x == out;
  if (in_place && (x_row != out_row || x_head != out_head)) return KMIP_ERR_INVALID_ARG;
  const size_t esize = dtype == KMIP_BF16 ? 2 : 4;
  // interleaved pairs move as one element of twice the size
  const size_t least = interleaved ? 2 * esize : esize;
  if (reinterpret_cast<uintptr_t>(x) % least || reinterpret_cast<uintptr_t>(out) % least)
    return KMIP_ERR_INVALID_ARG;
  if (interleaved && (x_row % 2 || x_head % 2 || out_row % 2 || out_head % 2))
    return KMIP_ERR_UNSUPPORTED;
  // rows and heads of the output may not share elements
  if ((H > 1 && out_head < d) || (N > 1 && H == 1 && out_row < d) ||
      (N > 1 && H > 1 && out_row < d) ||
      (N > 1 && H > 1 && out_head < out_row && (H - 1) * out_head + d > out_row) ||
      (N > 1 && H > 1 && out_row <= out_head && (N - 1) * out_row + d > out_head))
    return KMIP_ERR_INVALID_ARG;
  int* status = status_ptr();
  if (!status) return KMIP_ERR_CUDA;
  RotaryParams p{};
  p.x = x;
  p.out = out;
  p.x_row = x_row;
  p.x_head = x_head;
  p.out_row = out_row;
  p.out_head = out_head;
  p.pos = pos;
  p.freq = freq;
  p.axis = axis;
  p.N = N;
  p.H = H;
  p.d = d;
  p.pairs = pairs;
  p.axes = axes;
  p.interleaved = interleaved != 0;
  p.sign = inverse ? -1.f : 1.f;
  p.copy_tail = !in_place;
  p.status = status;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (dtype == KMIP_BF16) {
    switch (unit_width<__nv_bfloat16>(p)) {
      case 8: e = launch_pos<__nv_bfloat16, 8>(p, pos_type, stream); break;
      case 4: e = launch_pos<__nv_bfloat16, 4>(p, pos_type, stream); break;
      case 2: e = launch_pos<__nv_bfloat16, 2>(p, pos_type, stream); break;
      default: e = launch_pos<__nv_bfloat16, 1>(p, pos_type, stream);
    }
  } else {
    switch (unit_width<float>(p)) {
      case 4: e = launch_pos<float, 4>(p, pos_type, stream); break;
      case 2: e = launch_pos<float, 2>(p, pos_type, stream); break;
      default: e = launch_pos<float, 1>(p, pos_type, stream);
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return KMIP_ERR_CUDA;
  }
  return KMIP_OK;
}
