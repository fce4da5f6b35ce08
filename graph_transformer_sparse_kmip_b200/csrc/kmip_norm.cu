// kmip_norm.cu -- group norm per graph with an activation: entry points
// (kmip_group_norm_fwd, kmip_group_norm_bwd), the choice between the two ways
// over the graphs, and the kernels of the split one.
#include "kmip_launch.cuh"
#include "kmip_norm.cuh"

namespace kmip {
namespace {

// Threads of a split block: 256, or 384 where single elements or pairs of a row
// fill more of those (345 channels: 345 of 384, not 253 and 92 of 256 each).
constexpr int kSplitThreads = 256, kWideThreads = 384;
// Blocks that can be resident on an SM, by registers.
constexpr int split_blocks(int nt) { return nt == kSplitThreads ? 4 : 2; }

template <typename T, int V, int NT>
__global__ void __launch_bounds__(NT, split_blocks(NT)) norm_stats_split(const NormParams p) {
  after_previous();
  __shared__ StatSmem<NT> sm;
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  for (int slot = blockIdx.x; slot < p.slots; slot += gridDim.x) {
    int g, lo, r0, r1;
    if (!slot_rows(p, slot, g, lo, r0, r1)) continue;
    slab_stats<T, V, NT, kRowsOne<V>>(p, s, lo, r0, r1, sm);
    if (threadIdx.x < s.ngroups)
      p.part[(int64_t)slot * p.groups + s.g0 + threadIdx.x] =
          make_double2(sm.gs0[threadIdx.x], sm.gq[threadIdx.x]);
    __syncthreads();
  }
}

// One block per (graph, group): joins the graph's slots in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) norm_join_stats(const NormParams p) {
  after_previous();
  __shared__ double s0[8], s1[8];
  for (int64_t i = blockIdx.x; i < (int64_t)p.G * p.groups; i += gridDim.x) {
    const int g = (int)(i / p.groups), j = (int)(i % p.groups);
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) continue;
    const int a = first_slot(p, g), n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    const T c = lo < hi ? first_of<T>(p, lo, j) : T(0.f);
    double x = 0.0, q = 0.0;
#pragma unroll 4
    for (int t = threadIdx.x; t < n; t += 256) {
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
      for (int k = 1; k < 8; ++k) {
        x += s0[k];
        q += s1[k];
      }
      float m, r;
      finish_stats(x, q, (double)(hi - lo) * p.cg, pivot_of(c), p.eps, m, r);
      p.mean[i] = m;
      p.rstd[i] = r;
    }
    __syncthreads();
  }
}

// The same for graphs of a few slots: one thread per (graph, group).
template <typename T>
__global__ void __launch_bounds__(256) norm_join_stats_few(const NormParams p) {
  after_previous();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < (int64_t)p.G * p.groups;
       i += gridDim.x * 256ll) {
    const int g = (int)(i / p.groups), j = (int)(i % p.groups);
    int lo, hi;
    if (!graph_rows(p, g, lo, hi, true)) continue;
    const int a = first_slot(p, g), n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    const T c = lo < hi ? first_of<T>(p, lo, j) : T(0.f);
    double x = 0.0, q = 0.0;
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      const double2 v = p.part[(int64_t)(a + t) * p.groups + j];
      x += v.x;
      q += v.y;
    }
    finish_stats(x, q, (double)(hi - lo) * p.cg, pivot_of(c), p.eps, p.mean[i], p.rstd[i]);
  }
}

template <typename T, int V, int ACT, int NT>
__global__ void __launch_bounds__(NT, split_blocks(NT)) norm_apply_split(const NormParams p) {
  after_previous();
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  for (int slot = p.slots - 1 - (int)blockIdx.x; slot >= 0; slot -= gridDim.x) {
    int g, lo, r0, r1;
    if (!slot_rows(p, slot, g, lo, r0, r1)) continue;
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_apply<T, V, ACT, kRowsOne<V>>(p, s, r0, r1, mean, rstd);
    __syncthreads();
  }
}

template <typename T, int V, int ACT, int NT>
__global__ void __launch_bounds__(NT, NT == kSplitThreads ? 3 : 2)
norm_bwd_sums_split(const NormParams p) {
  after_previous();
  extern __shared__ float4 dyn[];
  BwdSmem<NT, V>& sm = *reinterpret_cast<BwdSmem<NT, V>*>(dyn);
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  for (int slot = blockIdx.x; slot < p.slots; slot += gridDim.x) {
    int g, lo, r0, r1;
    if (!slot_rows(p, slot, g, lo, r0, r1)) continue;
    load_stats(p, s, g, mean, rstd);
    __syncthreads();
    slab_bwd_sums<T, V, ACT, NT, false, kRowsTwo<V>>(
        p, s, r0, r1, mean, rstd, p.chan + (int64_t)slot * 2 * p.C, true, sm);
  }
}

// Sums of 32 channel columns over `rows` rows of src: 1,024 threads.
__device__ __forceinline__ float join_column(const float* src, int64_t cols, int rows,
                                             int64_t col, float (*red)[33]) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float a = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int r = ty; r < rows; r += 32) a += src[(int64_t)r * cols + col];
  }
  red[ty][tx] = a;
  __syncthreads();
  a = red[tx][ty];  // warp ty adds up column ty
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  __syncthreads();
  return a;  // every lane of warp w: the sum of column w
}

// Channel sums of each graph; with one graph, the parameters' gradients too.
template <typename T>
__global__ void __launch_bounds__(1024) norm_join_graph(const NormParams p, float* gchan, T* dw,
                                                        T* db) {
  after_previous();
  __shared__ float red[32][33];
  const int64_t cols = 2 * (int64_t)p.C, c0 = blockIdx.x * 32ll;
  for (int g = blockIdx.y; g < p.G; g += gridDim.y) {
    int lo, hi;
    if (!graph_rows(p, g, lo, hi)) lo = hi = 0;
    const int n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    const float* src = p.chan + (hi > lo ? (int64_t)first_slot(p, g) * cols : 0);
    const float sum = join_column(src, cols, n, c0 + (threadIdx.x & 31), red);
    const int64_t col = c0 + (threadIdx.x >> 5);
    if ((threadIdx.x & 31) == 0 && col < cols) {
      gchan[(int64_t)g * cols + col] = sum;
      if (dw) {
        if (col < p.C) db[col] = (T)sum;
        else dw[col - p.C] = (T)sum;
      }
    }
  }
}

// The same for graphs of a few slots: one warp per graph and 32 columns.
__global__ void __launch_bounds__(256) norm_join_graph_few(const NormParams p, float* gchan) {
  after_previous();
  const int64_t cols = 2 * (int64_t)p.C, col = blockIdx.x * 32ll + (threadIdx.x & 31);
  if (col >= cols) return;
  for (int64_t g = blockIdx.y * 8ll + (threadIdx.x >> 5); g < p.G; g += gridDim.y * 8ll) {
    int lo, hi;
    if (!graph_rows(p, (int)g, lo, hi, (threadIdx.x & 31) == 0)) lo = hi = 0;
    const int n = (int)(((int64_t)hi - lo + p.R - 1) / p.R);
    const float* src = p.chan + (hi > lo ? (int64_t)first_slot(p, (int)g) * cols : 0) + col;
    float a = 0.f;
#pragma unroll 4
    for (int r = 0; r < n; ++r) a += src[r * cols];
    gchan[g * cols + col] = a;
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_join_params(const float* src, int rows, int C, T* dw,
                                                         T* db) {
  after_previous();
  __shared__ float red[32][33];
  const int64_t cols = 2 * (int64_t)C, c0 = blockIdx.x * 32ll;
  const float sum = join_column(src, cols, rows, c0 + (threadIdx.x & 31), red);
  const int64_t col = c0 + (threadIdx.x >> 5);
  if ((threadIdx.x & 31) == 0 && col < cols) {
    if (col < C) db[col] = (T)sum;
    else dw[col - C] = (T)sum;
  }
}

template <typename T, int V, int ACT, int NT>
__global__ void __launch_bounds__(NT, NT == kSplitThreads ? 3 : 2)
norm_bwd_apply_split(const NormParams p) {
  after_previous();
  __shared__ float mean[kMaxSlabGroups], rstd[kMaxSlabGroups];
  __shared__ float m1[kMaxSlabGroups], m2[kMaxSlabGroups];
  const Slab s = make_slab<NT, V>(p, blockIdx.y);
  int have = -1;
  for (int slot = p.slots - 1 - (int)blockIdx.x; slot >= 0; slot -= gridDim.x) {
    int g, lo, r0, r1;
    if (!slot_rows(p, slot, g, lo, r0, r1)) continue;
    if (g != have) {  // means of the graph's groups, from its channel sums
      have = g;
      __syncthreads();
      load_stats(p, s, g, mean, rstd);
      int hi;
      graph_rows(p, g, lo, hi);
      const float* src = p.gchan + (int64_t)g * 2 * p.C;
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      for (int j = warp; j < s.ngroups; j += NT / 32) {
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
    slab_bwd_apply<T, V, ACT, kRowsTwo<V>>(p, s, r0, r1, mean, rstd, m1, m2);
  }
}

// --------------------------------------------------------------------- host
// Inputs up to this size, with graphs whose slab of one block is small, take
// the resident kernels (100,000 x 128 bf16 in 210 graphs: 16 us forward where the
// split ones take 30; 200,000 x 128 in 10,000: 103 and 198).  Where groups allow
// no wide loads the split ones win earlier (150,000 x 155 bf16 in 1,500 graphs:
// 129 us resident, 112 split).
constexpr int64_t kResidentBytes = 64 << 20, kResidentNarrowBytes = 16 << 20;
constexpr int64_t kResidentSlabBytes = 128 << 10;
// Bytes of a graph that a resident block should have to itself, if there are
// as many: it spends 3 to 4 us on a graph apart from its rows.
constexpr int64_t kResidentWorth = 16 << 10;
// A block spends about 2 us on a slot before and after its rows.
constexpr int64_t kSlotBytes = 32 << 10;
// Inputs above this do not stay in L2 (126 MB, beside what is written).
constexpr int64_t kOnceBytes = 64 << 20;

struct Plan {
  bool resident;
  int slabs;
  int nt;  // threads of a split block
};

// Sets p.gps, p.R, p.slots, p.once.
Plan plan(NormParams& p, int V, size_t esize) {
  Plan pl;
  const int64_t row = (int64_t)p.C * esize, group = (int64_t)p.cg * esize;
  auto slab_groups = [&](int64_t bytes) {
    int64_t n = (bytes + group - 1) / group;
    if (n > kMaxSlabGroups) n = kMaxSlabGroups;
    return (int)(n > p.groups ? p.groups : n);
  };
  const int sms = device_sm_count();
  // whole groups of at least 32 bytes a row, so that no sector is read twice;
  // of 64, with half as many blocks, where that still fills the SMs; and wider
  // where graphs are short, so that a graph's slab is worth a block's while
  int gps = slab_groups(64);
  if ((int64_t)p.G * ((p.groups + gps - 1) / gps) < sms) gps = slab_groups(32);
  const int64_t rows = p.N / p.G + 1;
  if (rows * gps * group < kResidentWorth) {
    int wide = slab_groups(kResidentWorth / rows);
    if ((int64_t)wide * p.cg / V > 256) wide = 256 * V / p.cg;  // one tile of vectors
    if (wide > gps) gps = wide;
  }
  pl.resident = row * p.N <= (V > 2 ? kResidentBytes : kResidentNarrowBytes) &&
                gps * group * (p.N / p.G) <= kResidentSlabBytes;
  pl.nt = kSplitThreads;
  p.gps = gps;
  if (!pl.resident) {
    // even slabs of as many groups as a row of threads covers, with the
    // number of threads that leaves fewer of them idle
    double best = -1.0;
    for (int nt : {kSplitThreads, kWideThreads}) {
      if (nt != kSplitThreads && V > 2) break;
      int64_t most = (int64_t)nt * V / p.cg;
      most = most < 1 ? 1 : most > kMaxSlabGroups ? kMaxSlabGroups : most;
      const int64_t slabs = (p.groups + most - 1) / most, even = (p.groups + slabs - 1) / slabs;
      const int64_t vecs = even * p.cg / V, w = vecs < nt ? vecs : nt;
      const int64_t rounds = (vecs + w - 1) / w;  // column tiles of a slab
      const double used = (double)p.groups * p.cg / V * (nt / w) / ((double)slabs * rounds * nt);
      if (used > best + 0.05) {
        best = used;
        pl.nt = nt;
        p.gps = (int)even;
      }
    }
  }
  pl.slabs = (p.groups + p.gps - 1) / p.gps;
  // one slot for every block that can be resident, of at least 64 rows and 32 KB
  const int64_t want = (int64_t)sms * split_blocks(pl.nt);
  const int64_t least = kSlotBytes / ((int64_t)p.gps * group);
  int64_t R = ((int64_t)p.N * pl.slabs + want - 1) / want;
  if (R < least) R = least;
  p.R = (int)(R < 64 ? 64 : R);
  p.slots = p.N / p.R + p.G;
  p.once = row * p.N > kOnceBytes;
  return pl;
}

template <int V, typename F>
cudaError_t with_threads(int nt, F&& f) {
  if constexpr (V <= 2) {
    if (nt == kWideThreads) return f.template operator()<kWideThreads>();
  }
  return f.template operator()<kSplitThreads>();
}

// Many graphs of a few slots each on average: joining them block by block costs
// more than the passes (50,000 x 480 bf16 in 2,000 graphs, training: 1,180 us with
// a block for each join, 340 with a warp or a thread).
bool few_slots(const NormParams& p) { return p.G > 1 && p.slots / p.G <= 16; }

dim3 split_grid(const NormParams& p, int slabs) {
  const int64_t x = ((int64_t)device_sm_count() * 16 + slabs - 1) / slabs;
  return dim3((unsigned)(p.slots < x ? p.slots : x), (unsigned)slabs);
}

cudaError_t norm_fwd(kmip_dtype_t dtype, int v, int act, NormParams p, cudaStream_t stream) {
  const Plan pl = plan(p, v, dtype == KMIP_BF16 ? 2 : 4);
  if (pl.slabs > 65535) return cudaErrorNotSupported;
  if (pl.resident) return launch_norm_fwd_resident(dtype, v, act, p, pl.slabs, stream);
  void* scratch = nullptr;
  cudaError_t e = scratch_alloc(&scratch, sizeof(double2) * (size_t)p.slots * p.groups, stream);
  if (e != cudaSuccess) return e;
  p.part = static_cast<double2*>(scratch);
  const dim3 grid = split_grid(p, pl.slabs);
  e = norm_dispatch(dtype, v, act, [&]<typename T, int V, int ACT>() {
    return with_threads<V>(pl.nt, [&]<int NT>() {
      norm_stats_split<T, V, NT><<<grid, NT, 0, stream>>>(p);
      const int64_t joins = (int64_t)p.G * p.groups;
      if (few_slots(p))
        launch_next(norm_join_stats_few<T>,
                    dim3(joins < 65536 * 256ll ? (unsigned)((joins + 255) / 256) : 65536u), 256, 0,
                    stream, p);
      else
        launch_next(norm_join_stats<T>, dim3(joins < 65536 ? (unsigned)joins : 65536u), 256, 0,
                    stream, p);
      launch_next(norm_apply_split<T, V, ACT, NT>, grid, NT, 0, stream, p);
      return cudaGetLastError();
    });
  });
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : ef;
}

cudaError_t norm_bwd(kmip_dtype_t dtype, int v, int act, NormParams p, void* dweight, void* dbias,
                     cudaStream_t stream) {
  const Plan pl = plan(p, v, dtype == KMIP_BF16 ? 2 : 4);
  if (pl.slabs > 65535) return cudaErrorNotSupported;
  const dim3 grid = split_grid(p, pl.slabs);
  const int64_t rows = pl.resident ? norm_resident_blocks(p, pl.slabs) : p.slots;
  const int64_t cols = 2 * (int64_t)p.C;
  void* scratch = nullptr;
  cudaError_t e = scratch_alloc(
      &scratch, sizeof(float) * (size_t)cols * (size_t)(rows + (pl.resident ? 0 : p.G)), stream);
  if (e != cudaSuccess) return e;
  p.chan = static_cast<float*>(scratch);
  if (pl.resident) e = launch_norm_bwd_resident(dtype, v, act, p, pl.slabs, stream);
  if (e == cudaSuccess)
    e = norm_dispatch(dtype, v, act, [&]<typename T, int V, int ACT>() {
      const unsigned tiles = (unsigned)((cols + 31) / 32);
      T *dw = static_cast<T*>(dweight), *db = static_cast<T*>(dbias);
      const float* sums = p.chan;
      int nsums = (int)rows;
      bool params = p.w != nullptr;
      if (!pl.resident) {
        float* gchan = p.chan + rows * cols;
        const bool direct = params && p.G == 1;
        p.gchan = gchan;
        const cudaError_t el = with_threads<V>(pl.nt, [&]<int NT>() {
          norm_bwd_sums_split<T, V, ACT, NT><<<grid, NT, sizeof(BwdSmem<NT, V>), stream>>>(p);
          if (few_slots(p))
            launch_next(norm_join_graph_few, dim3(tiles, p.G < 8 * 65535 ? (p.G + 7) / 8 : 65535),
                        256, 0, stream, p, gchan);
          else
            launch_next(norm_join_graph<T>, dim3(tiles, p.G < 65535 ? p.G : 65535), 1024, 0,
                        stream, p, gchan, direct ? dw : nullptr, db);
          launch_next(norm_bwd_apply_split<T, V, ACT, NT>, grid, NT, 0, stream, p);
          return cudaGetLastError();
        });
        if (el != cudaSuccess) return el;
        sums = gchan;
        nsums = p.G;
        params = params && !direct;
      }
      if (params)
        launch_next(norm_join_params<T>, dim3(tiles), 1024, 0, stream, sums, nsums, p.C, dw, db);
      return cudaGetLastError();
    });
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : ef;
}

// Widest vector inside one group that every pointer and row allows.
int vector_width(const NormParams& p, size_t esize, bool bwd) {
  const int wide = (int)(16 / esize), options[2] = {wide, esize == 2 ? 2 : 1};
  for (int v : options) {
    const uint64_t bytes = v * esize;
    auto off = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % bytes != 0; };
    if (p.cg % v || off(p.x) || off(p.w) || off(p.b)) continue;
    if (bwd ? off(p.dy) || off(p.dx) : off(p.y)) continue;
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
  if (N > kMaxRows || C > 65536 || N * (int64_t)C > ((int64_t)1 << 40))
    return KMIP_ERR_UNSUPPORTED;
  // graphs and slots are numbered, and stepped over, in 32 bits
  if (offsets && N / 64 + (int64_t)num_graphs > kMaxRows) return KMIP_ERR_UNSUPPORTED;
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
  const int G = graph_offsets ? num_graphs : 1;
  const size_t nc = es * N * C, c = weight ? es * C : 0, stats = sizeof(float) * G * groups;
  const size_t off = graph_offsets ? sizeof(int32_t) * ((size_t)G + 1) : 0;
  if (overlapping({{y, nc}, {mean, stats}, {rstd, stats}, {x, y == x ? 0 : nc}, {weight, c},
                   {bias, c}, {graph_offsets, off}}, 3) ||
      overlapping({{x, nc}, {mean, stats}, {rstd, stats}}, 1))
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
  p.G = G;
  p.groups = groups;
  p.cg = C / groups;
  p.eps = eps;
  p.status = status_ptr();
  if (!p.status) return KMIP_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return to_status(norm_fwd(dtype, vector_width(p, es, false), act, p, stream));
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
  const size_t es = dtype == KMIP_BF16 ? 2 : 4;
  if (!aligned_to(x, es) || !aligned_to(dy, es) || !aligned_to(dx, es) ||
      !aligned_to(weight, es) || !aligned_to(bias, es) || !aligned_to(dweight, es) ||
      !aligned_to(dbias, es))
    return KMIP_ERR_INVALID_ARG;
  const int G = graph_offsets ? num_graphs : 1;
  const size_t nc = es * N * C, c = weight ? es * C : 0, stats = sizeof(float) * G * groups;
  const size_t off = graph_offsets ? sizeof(int32_t) * ((size_t)G + 1) : 0;
  if (overlapping({{dx, nc}, {dweight, c}, {dbias, c}, {dy, dx == dy ? 0 : nc}, {x, nc},
                   {weight, c}, {bias, c}, {mean, stats}, {rstd, stats}, {graph_offsets, off}}, 3) ||
      overlapping({{dy, nc}, {dweight, c}, {dbias, c}}, 1))
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
  p.G = G;
  p.groups = groups;
  p.cg = C / groups;
  p.status = status_ptr();
  if (!p.status) return KMIP_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return to_status(norm_bwd(dtype, vector_width(p, es, true), act, p, dweight, dbias, stream));
}
