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
// (off by at most 2^-25 revolutions).  Its sine and cosine: sincospif for
// fp32 outputs; for bf16, whose half step is 2^-9 or more of the value, the
// fast ones (2^-20 of the pair in [-pi, pi]) in a fifth of the instructions.
//
// Bound: HBM traffic, one read and one write of x.  The angles of a node are
// the same for all of its heads: a block computes those of its nodes once
// into shared memory while its loads of x are in flight, so the sine and
// cosine cost 1 / H of a per-element evaluation.  Blocks stay and walk over
// tiles of nodes, because what a thread does inside a tile (which node, head
// and elements, which angles: three divisions) is the same for every tile.
#include "kmip_internal.h"

namespace kmip {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;
constexpr int kEvals = 2;                     // angles of a thread per tile
constexpr int kMaxTable = kEvals * kThreads;  // cos/sin pairs of a tile

// Units of a thread per tile: 64 bytes of x in flight either way.
constexpr int batch_of(bool inter) { return inter ? 4 : 2; }

struct RotaryParams {
  const void* x;
  void* out;
  int64_t x_row, x_head, out_row, out_head;  // strides in elements
  const void* pos;
  const double* freq;
  const int32_t* axis;
  int64_t N;
  int H, d, pairs, axes;
  int nodes;        // nodes per tile
  int chunks;       // units per head
  int64_t tiles;
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

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) {
  return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(a, cs.y, b * cs.x));
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int V>
struct Pack {
  using R = typename Raw<sizeof(T) * V>::type;
  union {
    R raw;
    T e[V];
    uint32_t w[sizeof(T) * V < 4 ? 1 : sizeof(T) * V / 4];
  };
  __device__ Pack() {}
  __device__ void load(const T* p) { raw = *reinterpret_cast<const R*>(p); }
  __device__ void store(T* p) const { *reinterpret_cast<R*>(p) = raw; }

  // Adjacent elements are the pairs; the first n of them turn.
  __device__ void turn_inside(const float2* cs, int n) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (i >= n) break;
      if constexpr (sizeof(T) == 4) {
        const float2 r = turned(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]), cs[i]);
        w[2 * i] = __float_as_uint(r.x);
        w[2 * i + 1] = __float_as_uint(r.y);
      } else {
        const float2 r = turned(low(w[i]), high(w[i]), cs[i]);
        w[i] = pack(r.x, r.y);
      }
    }
  }
  // Element i here and in `o` are a pair.
  __device__ void turn_with(Pack& o, const float2* cs) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 r = turned(__uint_as_float(w[i]), __uint_as_float(o.w[i]), cs[i]);
        w[i] = __float_as_uint(r.x);
        o.w[i] = __float_as_uint(r.y);
      }
    } else if constexpr (V == 1) {
      const float2 r = turned(__bfloat162float(e[0]), __bfloat162float(o.e[0]), cs[0]);
      e[0] = __float2bfloat16_rn(r.x);
      o.e[0] = __float2bfloat16_rn(r.y);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 r = turned(low(w[i]), low(o.w[i]), cs[2 * i]);
        const float2 q = turned(high(w[i]), high(o.w[i]), cs[2 * i + 1]);
        w[i] = pack(r.x, q.x);
        o.w[i] = pack(r.y, q.y);
      }
    }
  }
};

// (cos, sin) of an angle in revolutions.
template <typename T>
__device__ __forceinline__ float2 unit_circle(double rev) {
  const float r = (float)(rev - rint(rev));
  float2 cs;
  if constexpr (sizeof(T) == 4)
    sincospif(2.f * r, &cs.y, &cs.x);
  else
    __sincosf(6.2831853071795865f * r, &cs.y, &cs.x);
  return cs;
}

// A unit is what one thread turns at a time: with halves, V pairs (p, p + P)
// or V elements behind them; interleaved, V elements (V / 2 pairs).  A tile is
// p.nodes nodes with all their units, or (grid.y) a slice of one node's units.
template <typename T, int V, typename PosT, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rotary_kernel(const RotaryParams p) {
  constexpr int kBatch = batch_of(INTER);
  extern __shared__ float2 tables[];  // [2][nodes][pairs]
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  const PosT* pos = static_cast<const PosT*>(p.pos);
  const int per_node = p.H * p.chunks;
  const int rot_chunks = INTER ? p.chunks : p.pairs / V;

  // What this thread does in every tile.
  uint32_t src[kBatch], dst[kBatch];  // from the tile's first node, in units
  int node[kBatch], chunk[kBatch];    // node = p.nodes: no unit
#pragma unroll
  for (int t = 0; t < kBatch; ++t) {
    const int i = (blockIdx.y * kBatch + t) * kThreads + threadIdx.x;
    const int n = i / per_node, r = i - n * per_node;
    const int head = r / p.chunks, c = r - head * p.chunks;
    const bool pair = c < rot_chunks;
    node[t] = n < p.nodes && (pair || p.copy_tail) ? n : p.nodes;
    chunk[t] = c;
    // tail chunks (halves only) start behind both halves
    const int e = pair ? c * V : 2 * p.pairs + (c - rot_chunks) * V;
    src[t] = (uint32_t)((n * p.x_row + head * p.x_head + e) / V);
    dst[t] = (uint32_t)((n * p.out_row + head * p.out_head + e) / V);
  }
  double freq[kEvals];  // revolutions per unit
  int from[kEvals];     // place of the position in the tile's
  int last[kEvals];     // node
#pragma unroll
  for (int k = 0; k < kEvals; ++k) {
    const int i = k * kThreads + threadIdx.x;
    last[k] = p.nodes;
    freq[k] = 0.0;
    from[k] = 0;
    if (i < p.nodes * p.pairs) {
      const int n = i / p.pairs, q = i - n * p.pairs;
      const int ax = p.axis[q];
      last[k] = n;
      if ((unsigned)ax < (unsigned)p.axes) {
        freq[k] = p.freq[q] * 0.15915494309189535;  // 1 / (2 pi)
        from[k] = n * p.axes + ax;
      } else {
        from[k] = -1;  // its pair stays as it is
        record_status(p.status, KMIP_ERR_BAD_INDEX);
      }
    }
  }

  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t n0 = tile * p.nodes;
    const int nodes = (int)min((int64_t)p.nodes, p.N - n0);
    const T* xt = x + n0 * p.x_row;
    T* ot = out + n0 * p.out_row;
    Pack<T, V> a[kBatch], b[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t)
      if (node[t] < nodes) {
        a[t].load(xt + (size_t)src[t] * V);
        if (!INTER && chunk[t] < rot_chunks) b[t].load(xt + (size_t)src[t] * V + p.pairs);
      }
    // Two tables in turn: a block-wide barrier per tile keeps a thread from
    // writing a table that another still reads.
    float2* table = tables + buf * p.nodes * p.pairs;
    PosT where[kEvals];
#pragma unroll
    for (int k = 0; k < kEvals; ++k)
      if (last[k] < nodes && from[k] >= 0) where[k] = pos[n0 * p.axes + from[k]];
#pragma unroll
    for (int k = 0; k < kEvals; ++k)
      if (last[k] < nodes) {
        float2 cs = make_float2(1.f, 0.f);
        if (from[k] >= 0) cs = unit_circle<T>((double)where[k] * freq[k]);
        cs.y *= p.sign;
        table[k * kThreads + threadIdx.x] = cs;
      }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      if (node[t] >= nodes) continue;
      const int c = chunk[t];
      const float2* cs = table + node[t] * p.pairs;
      if constexpr (INTER) {
        a[t].turn_inside(cs + c * (V / 2), p.pairs - c * (V / 2));
      } else if (c < rot_chunks) {
        a[t].turn_with(b[t], cs + c * V);
        b[t].store(ot + (size_t)dst[t] * V + p.pairs);
      }
      a[t].store(ot + (size_t)dst[t] * V);
    }
  }
}

template <typename T, int V, typename PosT, bool INTER>
cudaError_t launch(RotaryParams p, cudaStream_t stream) {
  // interleaved units are V elements; with halves the pairs and the tail
  // each make whole units
  p.chunks = INTER ? p.d / V : p.pairs / V + (p.d - 2 * p.pairs) / V;
  constexpr int kUnits = batch_of(INTER) * kThreads;
  const int per_node = p.H * p.chunks, sms = device_sm_count();
  int64_t nodes = kUnits / per_node;
  if (p.pairs && nodes > kMaxTable / p.pairs) nodes = kMaxTable / p.pairs;
  // few nodes: smaller tiles, one for every block that can be resident
  const int most = kBlocksPerSm * sms;
  const int64_t share = (p.N + most - 1) / most;
  if (nodes > share) nodes = share;
  // a thread's offsets in a tile are held in 32 bits, in units of V elements
  const int64_t row = p.x_row > p.out_row ? p.x_row : p.out_row;
  const int64_t head = p.x_head > p.out_head ? p.x_head : p.out_head;
  auto reach = [&](int64_t n) { return ((n - 1) * row + (p.H - 1) * head + p.d) / V; };
  if (nodes < 1 || reach(nodes) > UINT32_MAX) nodes = 1;
  if (reach(1) > UINT32_MAX) {  // heads far apart: one launch for each
    const int H = p.H;
    p.H = 1;
    for (int h = 0; h < H; ++h) {
      const cudaError_t e = launch<T, V, PosT, INTER>(p, stream);
      if (e != cudaSuccess) return e;
      p.x = static_cast<const T*>(p.x) + p.x_head;
      p.out = static_cast<T*>(p.out) + p.out_head;
    }
    return cudaSuccess;
  }
  p.nodes = (int)nodes;
  p.tiles = (p.N + p.nodes - 1) / p.nodes;
  const size_t smem = 2 * sizeof(float2) * (size_t)p.nodes * p.pairs;
  const dim3 grid((unsigned)(p.tiles < most ? p.tiles : most),
                  (unsigned)((per_node + kUnits - 1) / kUnits));
  rotary_kernel<T, V, PosT, INTER><<<grid, kThreads, smem, stream>>>(p);
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

// Whether N rows of H heads of d elements at x and at out, `delta` elements
// further on, share one.  Blocks read and write in no order, so they may not.
// With the same strides the two may lie between one another (other heads of
// the same rows); with different ones they are taken to meet as soon as the
// ranges that they span do.
bool shares_elements(int64_t delta, int64_t N, int64_t H, int64_t d, int64_t x_row,
                     int64_t x_head, int64_t out_row, int64_t out_head) {
  const int64_t x_span = (N - 1) * x_row + (H - 1) * x_head + d;
  const int64_t out_span = (N - 1) * out_row + (H - 1) * out_head + d;
  if (delta >= x_span || delta <= -out_span) return false;
  if (x_row != out_row || x_head != out_head) return true;
  for (int64_t j = 1 - H; j < H; ++j) {
    const int64_t rest = delta - j * x_head;  // to be met by a difference of rows
    const int64_t i = x_row ? rest / x_row : 0;     // the closest is i, i - 1 or i + 1
    for (int64_t r = i - 1; r <= i + 1; ++r) {
      if (r <= -N || r >= N) continue;
      const int64_t gap = rest - r * x_row;
      if (gap < d && gap > -d) return true;
    }
  }
  return false;
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
  // the stride of a single row or head says nothing
  if (N == 1) x_row = out_row = 0;
  if (H == 1) x_head = out_head = 0;
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
  const int64_t delta = static_cast<int64_t>(reinterpret_cast<uintptr_t>(out) -
                                             reinterpret_cast<uintptr_t>(x)) /
                        static_cast<int64_t>(esize);
  if (!in_place && shares_elements(delta, N, H, d, x_row, x_head, out_row, out_head))
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
