// kmip_ffn_tc.cu -- the gated feed-forward block on tcgen05 tensor cores
// (bf16 operands, fp32 accumulation).
//
// With x, dy [N, C], Wg, Wu [F, C], Wd [C, F]:
//   forward   h = act(x Wg^T) * (x Wu^T),  y = h Wd^T
//   backward  a = x Wg^T, b = x Wu^T, dh = dy Wd, all three of one tile in
//             tensor memory; its epilogue writes dA = dh b act'(a),
//             dB = dh act(a), h = act(a) b; then
//             dx = dA Wg + dB Wu,
//             dWg = dA^T x, dWu = dB^T x, dWd^T = h^T dy.
// a and b are recomputed instead of kept from the forward: nothing of size
// [N, F] outlives a call, and the gradients see a, b and dh in fp32 -- the
// one rounding to bf16 between them and the gradients is that of dA, dB, h,
// which the tensor cores need.  It costs 4 N C F of 22 N C F operations.
//
// One kernel, five uses.  A cluster of two CTAs works on a tile of 256 rows
// and BN columns (cta_group::2): each CTA stages its 128 rows of A and half
// of B's rows, so a pair reads 64 KB per 256 x 256 x 64 step where two single
// CTAs would read 96 KB; at 8192 flop per cycle and SM a step takes 512
// cycles, and 64 bytes per cycle and SM is what L2 can feed.  Warp 8 issues
// TMA loads into a ring of 32 KB stages, warp 9 of the leading CTA issues the
// MMAs, warps 0-7 of both CTAs read the accumulators (128 lanes each, two
// warps per quarter, one per half of the columns), compute and hand swizzled
// boxes to TMA stores.  Accumulators are double-buffered; the backward's
// three need 384 of 512 columns, so there dh alone has two buffers, and dh of
// the next tile runs while a and b are read.
//
// The weight gradients contract over N: both operands have the contraction
// index outermost.  They are few tiles and long sums, so the work units
// (tile, 64 rows) are dealt to the clusters in equal contiguous runs; a tile
// cut by a run's end leaves fp32 partials that a second kernel adds in the
// order of the runs: the same bits every time.
#include <cuda.h>

#include "kmip_act.cuh"
#include "kmip_ffn.h"
#include "kmip_gemm.cuh"
#include "kmip_internal.h"
#include "kmip_tensormap.h"

namespace kmip {
namespace {

using namespace sm100;

enum Mode {
  kGlu,    // h = act(x Wg^T) * (x Wu^T)
  kNT,     // out = A B^T, B [n][k]
  kNN,     // out = A0 B0 + A1 B1, B [k][n]
  kGluBwd, // dA, dB, h
  kTN      // dWg, dWu, dWd: A^T B, A [k][m], B [k][n]
};

constexpr int kBK = 64;              // contraction step of a stage
constexpr int kHalfM = 128;          // rows of one CTA
constexpr int kTileM = 2 * kHalfM;
constexpr int kGluF = 128;           // F columns of a GLU tile
constexpr int kStageA = kHalfM * kBK * 2;   // 16 KB
constexpr int kStageB = 128 * kBK * 2;      // at most
constexpr int kStage = kStageA + kStageB;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s

constexpr int stages_of(Mode m) { return m == kGluBwd ? 5 : 6; }
constexpr int staging_of(Mode m) {
  // a box of 64 columns per half, or three of 32 (dA, dB, h)
  return m == kGluBwd ? 2 * 3 * kHalfM * 64 : 2 * kHalfM * 128;
}
constexpr int smem_of(Mode m) { return 1024 + stages_of(m) * kStage + staging_of(m) + 256; }
static_assert(smem_of(kGlu) <= 232448 && smem_of(kGluBwd) <= 232448, "shared memory");

struct alignas(64) Maps {
  CUtensorMap m[8];
};

struct GemmParams {
  int rows, cols;      // output extent (kGlu, kGluBwd: N x F)
  int tiles_n;         // column tiles
  int tiles;           // all tiles
  int kb0, kb1;        // steps of the two segments
  int tiles_p;         // kTN: row tiles of one of the three gradients
  float4* part;        // kTN: partial tiles, two per cluster
  __nv_bfloat16* dwd;  // kTN: [cols][rows]
  int* status;
};

// A cluster's share of the work: tiles c, c + clusters, ... or, for kTN, the
// units [c U / clusters, (c + 1) U / clusters) of U = tiles * kb0.
struct Item {
  int tile, k0, kn;
};

__device__ __forceinline__ int64_t run_start(int64_t units, int c, int clusters) {
  return units * c / clusters;
}

template <int MODE>
struct Walk {
  int64_t u, end;
  int step, kb;
  __device__ Walk(const GemmParams& p, int c, int clusters) {
    kb = p.kb0;
    if (MODE == kTN) {
      const int64_t units = (int64_t)p.tiles * kb;
      u = run_start(units, c, clusters);
      end = run_start(units, c + 1, clusters);
    } else {
      u = c;
      end = p.tiles;
      step = clusters;
    }
  }
  __device__ bool next(Item& it) {
    if (u >= end) return false;
    if (MODE == kTN) {
      it.tile = (int)(u / kb);
      it.k0 = (int)(u % kb);
      const int64_t left = end - u;
      it.kn = (int)(left < kb - it.k0 ? left : kb - it.k0);
      u += it.kn;
    } else {
      it.tile = (int)u;
      it.k0 = 0;
      it.kn = kb;
      u += step;
    }
    return true;
  }
};

// 32 packed bf16 pairs of a row into a box of 64 columns (128-byte rows,
// 128-byte swizzle), columns 32 c ..; or into a box of 32 (64-byte rows).
__device__ __forceinline__ void put_box64(uint32_t box, int row, int c, const uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t at = box + row * 128 + (((c * 4 + q) ^ (row & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
  }
}
__device__ __forceinline__ void put_box32(uint32_t box, int row, const uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t at = box + row * 64 + ((q ^ ((row >> 1) & 3)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int MODE, int BN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ffn_gemm_kernel(const __grid_constant__ Maps maps, const GemmParams p) {
  using T = __nv_bfloat16;
  constexpr int kStages = stages_of((Mode)MODE);
  constexpr int kBufs = MODE == kGluBwd ? 1 : 2;
  constexpr int kBufCols = MODE == kGluBwd ? 0 : BN;
  constexpr int kTmemCols = MODE == kGluBwd ? 512 : 2 * BN;
  constexpr int kSegs = MODE == kNN || MODE == kGluBwd ? 2 : 1;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t staging = base + kStages * kStage;
  const uint32_t bars = staging + staging_of((Mode)MODE);
  const uint32_t full = bars, empty = bars + 8 * kStages;
  const uint32_t tfull = empty + 8 * kStages, tempty = tfull + 16;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_store;
  volatile int* abort_flag = &abort_store;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    abort_store = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + 8 * b, 1);
      mbar_init(tempty + 8 * b, 2 * kEpiWarps);
    }
    fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tmem_alloc_pair(smem_addr(&tmem_slot), kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = map_to_cta(full, 0);
      uint32_t it_no = 0;
      Walk<MODE> walk(p, cluster, clusters);
      Item it;
      bool ok = true;
      while (ok && walk.next(it)) {
        const int mt = it.tile / p.tiles_n, nt = it.tile % p.tiles_n;
        for (int seg = 0; seg < kSegs && ok; ++seg) {
          const int kn = seg ? p.kb1 : (MODE == kTN ? it.kn : p.kb0);
          for (int kb = 0; kb < kn; ++kb, ++it_no) {
            const uint32_t s = it_no % kStages, ph = (it_no / kStages) & 1;
            if (!mbar_wait(empty + 8 * s, ph ^ 1, abort_flag, kTimeoutNs)) {
              ok = false;
              break;
            }
            const uint32_t a = base + s * kStage, b = a + kStageA, bar = full0 + 8 * s;
            const int k = (it.k0 + kb) * kBK;
            constexpr uint32_t kBytesB =
                MODE == kGlu || MODE == kGluBwd ? kStageB : (uint32_t)(BN / 2) * kBK * 2;
            const uint32_t bytes =
                2 * (kStageA + (MODE == kGluBwd && seg == 0 ? kStageB / 2 : kBytesB));
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
            if constexpr (MODE == kGlu) {
              tma_load_2d_pair(a, &maps.m[0], bar, k, mt * kTileM + rank * kHalfM);
              tma_load_2d_pair(b, &maps.m[1 + rank], bar, k, nt * kGluF);
            } else if constexpr (MODE == kNT) {
              tma_load_2d_pair(a, &maps.m[0], bar, k, mt * kTileM + rank * kHalfM);
              tma_load_2d_pair(b, &maps.m[1], bar, k, nt * BN + rank * (BN / 2));
            } else if constexpr (MODE == kNN) {
              tma_load_2d_pair(a, &maps.m[seg], bar, k, mt * kTileM + rank * kHalfM);
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tma_load_2d_pair(b + j * 8192, &maps.m[2 + seg], bar,
                                 nt * BN + rank * (BN / 2) + 64 * j, k);
            } else if constexpr (MODE == kGluBwd) {
              if (seg == 0) {
                tma_load_2d_pair(a, &maps.m[0], bar, k, mt * kTileM + rank * kHalfM);
                tma_load_2d_pair(b, &maps.m[1], bar, nt * kGluF + rank * 64, k);
              } else {
                tma_load_2d_pair(a, &maps.m[2], bar, k, mt * kTileM + rank * kHalfM);
                tma_load_2d_pair(b, &maps.m[3 + rank], bar, k, nt * kGluF);
              }
            } else {
              const int prob = mt / p.tiles_p, m0 = (mt % p.tiles_p) * kTileM + rank * kHalfM;
              tma_load_2d_pair(a, &maps.m[prob], bar, m0, k);
              tma_load_2d_pair(a + 8192, &maps.m[prob], bar, m0 + 64, k);
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tma_load_2d_pair(b + j * 8192, &maps.m[3 + (prob == 2)], bar,
                                 nt * BN + rank * (BN / 2) + 64 * j, k);
            }
          }
        }
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0 && rank == 0) {
      uint32_t it_no = 0, tile_no = 0;
      Walk<MODE> walk(p, cluster, clusters);
      Item it;
      bool ok = true;
      while (ok && walk.next(it)) {
        const uint32_t buf = kBufs == 2 ? tile_no & 1 : 0;
        const uint32_t use = kBufs == 2 ? tile_no >> 1 : tile_no;
        if (MODE != kGluBwd) {
          if (!mbar_wait_cluster(tempty + 8 * buf, (use & 1) ^ 1, abort_flag, kTimeoutNs)) break;
          tc_fence_after();
        }
        for (int seg = 0; seg < kSegs && ok; ++seg) {
          uint32_t d = tmem + buf * kBufCols;
          if (MODE == kGluBwd) {
            if (seg == 0) {
              d = tmem + 256 + (tile_no & 1) * 128;
            } else {
              d = tmem;
              if (!mbar_wait_cluster(tempty, (use & 1) ^ 1, abort_flag, kTimeoutNs)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
          }
          constexpr bool a_outer = MODE == kTN;
          const bool b_outer = MODE == kTN || MODE == kNN || (MODE == kGluBwd && seg == 0);
          const int n = MODE == kGlu || (MODE == kGluBwd && seg == 1) ? 256
                        : MODE == kGluBwd                               ? 128
                                                                        : BN;
          const uint32_t idesc = idesc_bf16_f32(kTileM, n) | (a_outer ? kIdescAOuterK : 0u) |
                                 (b_outer ? kIdescBOuterK : 0u);
          const int kn = seg ? p.kb1 : (MODE == kTN ? it.kn : p.kb0);
          const bool keep = MODE == kNN && seg == 1;  // adds to the first segment
          for (int kb = 0; kb < kn; ++kb, ++it_no) {
            const uint32_t s = it_no % kStages, ph = (it_no / kStages) & 1;
            if (!mbar_wait_cluster(full + 8 * s, ph, abort_flag, kTimeoutNs)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = base + s * kStage, b = a + kStageA;
            const uint64_t da = a_outer ? smem_desc_mn(a, 8192) : smem_desc(a, 1024, 2);
            const uint64_t db = b_outer ? smem_desc_mn(b, 8192) : smem_desc(b, 1024, 2);
            // 16 contraction indices on: 32 bytes along a row, or 16 rows
            const uint64_t sa = a_outer ? 128 : 2, sb = b_outer ? 128 : 2;
#pragma unroll
            for (int q = 0; q < kBK / 16; ++q)
              mma_bf16_pair(d, da + q * sa, db + q * sb, idesc, kb || q || keep);
            mma_commit_pair(empty + 8 * s);
          }
        }
        if (ok) mma_commit_pair(tfull + 8 * buf);
        ++tile_no;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool issuer = (threadIdx.x & 127) == 0;
    const uint32_t box = staging + half * (staging_of((Mode)MODE) / 2);
    const uint32_t tempty0 = map_to_cta(tempty, 0);
    uint32_t tile_no = 0;
    Walk<MODE> walk(p, cluster, clusters);
    Item it;
    while (walk.next(it)) {
      const int mt = it.tile / p.tiles_n, nt = it.tile % p.tiles_n;
      const uint32_t buf = kBufs == 2 ? tile_no & 1 : 0;
      const uint32_t use = kBufs == 2 ? tile_no >> 1 : tile_no;
      // the half's four warps go on or give up together (they meet at barriers)
      if (!named_all(1 + half, 128, mbar_wait(tfull + 8 * buf, use & 1, abort_flag, kTimeoutNs)))
        break;
      tc_fence_after();
      const uint32_t acc = lanes + buf * kBufCols;
      const int m0 = mt * kTileM + rank * kHalfM;

      // This thread has read what it needs of the accumulators.
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
      };
      // The half's staging is free again / complete and on its way out.
      auto staging_free = [&] {
        if (issuer) bulk_wait_read();
        named_sync(1 + half, 128);
      };

      if constexpr (MODE == kGlu) {
        const int f0 = nt * kGluF + half * 64;
        uint32_t w[2][16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float g[32], u[32];
          tmem_ld32(acc + half * 64 + c * 32, g);
          tmem_ld32(acc + 128 + half * 64 + c * 32, u);
          tmem_ld_wait_all();
          reg_fence(g);
          reg_fence(u);
          if (c == 1) release();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[c][e] = pack2(act_value<T, ACT>(g[2 * e]) * u[2 * e],
                            act_value<T, ACT>(g[2 * e + 1]) * u[2 * e + 1]);
        }
        staging_free();
        put_box64(box, row, 0, w[0]);
        put_box64(box, row, 1, w[1]);
        fence_async_shared();
        named_sync(1 + half, 128);
        if (issuer && m0 < p.rows && f0 < p.cols) {
          tma_store_2d(&maps.m[3], box, f0, m0);
          bulk_commit();
        }
      } else if constexpr (MODE == kGluBwd) {
        const uint32_t acc_dh = lanes + 256 + (tile_no & 1) * 128;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = half * 64 + c * 32, f0 = nt * kGluF + col;
          float a[32], b[32], dh[32];
          tmem_ld32(acc + col, a);
          tmem_ld32(acc + 128 + col, b);
          tmem_ld32(acc_dh + col, dh);
          tmem_ld_wait_all();
          reg_fence(a);
          reg_fence(b);
          reg_fence(dh);
          if (c == 1) release();
          uint32_t wa[16], wb[16], wh[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float ra[2], rb[2], rh[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float f, g;
              act_both<T, ACT>(a[2 * e + z], f, g);
              ra[z] = dh[2 * e + z] * b[2 * e + z] * g;
              rb[z] = dh[2 * e + z] * f;
              rh[z] = f * b[2 * e + z];
            }
            wa[e] = pack2(ra[0], ra[1]);
            wb[e] = pack2(rb[0], rb[1]);
            wh[e] = pack2(rh[0], rh[1]);
          }
          staging_free();
          put_box32(box, row, wa);
          put_box32(box + 8192, row, wb);
          put_box32(box + 16384, row, wh);
          fence_async_shared();
          named_sync(1 + half, 128);
          if (issuer && m0 < p.rows && f0 < p.cols) {
            tma_store_2d(&maps.m[5], box, f0, m0);
            tma_store_2d(&maps.m[6], box + 8192, f0, m0);
            tma_store_2d(&maps.m[7], box + 16384, f0, m0);
            bulk_commit();
          }
        }
      } else {
        const bool partial = MODE == kTN && it.kn < p.kb0;
        const int prob = MODE == kTN ? mt / p.tiles_p : 0;
        const int r0 = MODE == kTN ? (mt % p.tiles_p) * kTileM + (int)rank * kHalfM : m0;
        // this cluster's first run starts inside the tile: slot 0; its last
        // one ends inside: slot 1
        float4* part = MODE == kTN
                           ? p.part + ((int64_t)(2 * cluster + (it.k0 == 0)) * 2 + rank) *
                                          (BN / 4 * kHalfM)
                           : nullptr;
#pragma unroll 1
        for (int j = 0; j < BN / 128; ++j) {
          const int col = half * (BN / 2) + j * 64, c0 = nt * BN + col;
          float v[2][32];
          tmem_ld32(acc + col, v[0]);
          tmem_ld32(acc + col + 32, v[1]);
          tmem_ld_wait_all();
          reg_fence(v[0]);
          reg_fence(v[1]);
          if (j == BN / 128 - 1) release();
          if (partial) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              part[(int64_t)(col / 4 + e) * kHalfM + row] =
                  make_float4(v[e / 8][4 * (e % 8)], v[e / 8][4 * (e % 8) + 1],
                              v[e / 8][4 * (e % 8) + 2], v[e / 8][4 * (e % 8) + 3]);
          } else if (MODE == kTN && prob == 2) {
            // dWd is [C][F]: neighbouring lanes hold neighbouring F
            if (r0 + row < p.rows) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (c0 + e < p.cols)
                  p.dwd[(int64_t)(c0 + e) * p.rows + r0 + row] =
                      __float2bfloat16_rn(v[e / 32][e % 32]);
            }
          } else {
            uint32_t w[2][16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              w[0][e] = pack2(v[0][2 * e], v[0][2 * e + 1]);
              w[1][e] = pack2(v[1][2 * e], v[1][2 * e + 1]);
            }
            staging_free();
            put_box64(box, row, 0, w[0]);
            put_box64(box, row, 1, w[1]);
            fence_async_shared();
            named_sync(1 + half, 128);
            if (issuer && r0 < p.rows && c0 < p.cols) {
              tma_store_2d(&maps.m[MODE == kTN ? 5 + prob : 4], box, c0, r0);
              bulk_commit();
            }
          }
        }
      }
      ++tile_no;
    }
    if (issuer) bulk_wait_all();
  }

  // ------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (*abort_flag && threadIdx.x == 0) record_status(p.status, KMIP_ERR_TIMEOUT);
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Adds the partial tiles of the weight gradients in the order of the runs.
// Grid: (tile, CTA of the pair, 32-column group); 128 threads, one per row.
template <int BN>
__global__ void __launch_bounds__(128) ffn_join_kernel(const GemmParams p, int clusters,
                                                       __nv_bfloat16* dwg, __nv_bfloat16* dwu) {
  const int tile = blockIdx.x, rank = blockIdx.y, row = threadIdx.x;
  const int64_t units = (int64_t)p.tiles * p.kb0, u0 = (int64_t)tile * p.kb0, u1 = u0 + p.kb0;
  // the cluster whose run holds unit u0
  int c = (int)(u0 * clusters / units);
  while (run_start(units, c + 1, clusters) <= u0) ++c;
  while (run_start(units, c, clusters) > u0) --c;
  if (run_start(units, c, clusters) <= u0 && run_start(units, c + 1, clusters) >= u1)
    return;  // written whole by its cluster
  float4 v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (; c < clusters && run_start(units, c, clusters) < u1; ++c) {
    const int64_t start = run_start(units, c, clusters);
    if (run_start(units, c + 1, clusters) == start) continue;  // empty run
    const float4* src = p.part +
                        ((int64_t)(2 * c + (start <= u0)) * 2 + rank) * (BN / 4 * kHalfM) +
                        (int64_t)blockIdx.z * 8 * kHalfM + row;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 t = src[(int64_t)e * kHalfM];
      v[e].x += t.x;
      v[e].y += t.y;
      v[e].z += t.z;
      v[e].w += t.w;
    }
  }
  const int mt = tile / p.tiles_n, nt = tile % p.tiles_n, prob = mt / p.tiles_p;
  const int r = (mt % p.tiles_p) * kTileM + rank * kHalfM + row;
  const int c0 = nt * BN + blockIdx.z * 32;
  if (r >= p.rows) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int col = c0 + 4 * e;  // cols is a multiple of 8
    if (col >= p.cols) break;
    if (prob == 2) {
      p.dwd[(int64_t)col * p.rows + r] = __float2bfloat16_rn(v[e].x);
      p.dwd[(int64_t)(col + 1) * p.rows + r] = __float2bfloat16_rn(v[e].y);
      p.dwd[(int64_t)(col + 2) * p.rows + r] = __float2bfloat16_rn(v[e].z);
      p.dwd[(int64_t)(col + 3) * p.rows + r] = __float2bfloat16_rn(v[e].w);
    } else {
      *reinterpret_cast<uint2*>((prob ? dwu : dwg) + (int64_t)r * p.cols + col) =
          make_uint2(pack2(v[e].x, v[e].y), pack2(v[e].z, v[e].w));
    }
  }
}

// ------------------------------------------------------------------ host side

int clusters_for(int64_t tiles) {
  const int most = device_sm_count() / 2;
  return (int)(tiles < most ? tiles : most);
}

template <int MODE, int BN, int ACT>
cudaError_t launch_gemm(const Maps& maps, const GemmParams& p, int clusters, cudaStream_t stream) {
  auto kern = ffn_gemm_kernel<MODE, BN, ACT>;
  constexpr int smem = smem_of((Mode)MODE);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<2 * clusters, kThreads, smem, stream>>>(maps, p);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_act(int act, const Maps& maps, const GemmParams& p, cudaStream_t stream) {
  const int c = clusters_for(p.tiles);
  switch (act) {
    case KMIP_ACT_SILU: return launch_gemm<MODE, 256, KMIP_ACT_SILU>(maps, p, c, stream);
    case KMIP_ACT_GELU: return launch_gemm<MODE, 256, KMIP_ACT_GELU>(maps, p, c, stream);
    case KMIP_ACT_RELU: return launch_gemm<MODE, 256, KMIP_ACT_RELU>(maps, p, c, stream);
    default: return launch_gemm<MODE, 256, KMIP_ACT_NONE>(maps, p, c, stream);
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Columns of an output tile: 256 reads A half as often, but is not worth a
// quarter more of columns behind the edge.
int tile_cols(int cols) {
  return ceil_div(cols, 256) * 256 * 4 >= ceil_div(cols, 128) * 128 * 5 ? 128 : 256;
}

}  // namespace

cudaError_t launch_ffn_glu(const FfnArgs& a, void* h, cudaStream_t stream) {
  Maps m;
  GemmParams p{};
  p.rows = a.N;
  p.cols = a.F;
  p.tiles_n = ceil_div(a.F, kGluF);
  p.tiles = ceil_div(a.N, kTileM) * p.tiles_n;
  p.kb0 = ceil_div(a.C, kBK);
  p.status = a.status;
  if (!encode_map_2d(&m.m[0], a.x, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wg, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[2], a.wu, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[3], h, a.N, a.F, 64, kHalfM))
    return cudaErrorInvalidValue;
  return launch_act<kGlu>(a.act, m, p, stream);
}

cudaError_t launch_ffn_down(const FfnArgs& a, const void* h, void* y, cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p{};
  p.rows = a.N;
  p.cols = a.C;
  p.tiles_n = ceil_div(a.C, bn);
  p.tiles = ceil_div(a.N, kTileM) * p.tiles_n;
  p.kb0 = ceil_div(a.F, kBK);
  p.status = a.status;
  if (!encode_map_2d(&m.m[0], h, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wd, a.C, a.F, 64, bn / 2) ||
      !encode_map_2d(&m.m[4], y, a.N, a.C, 64, kHalfM))
    return cudaErrorInvalidValue;
  const int c = clusters_for(p.tiles);
  return bn == 256 ? launch_gemm<kNT, 256, 0>(m, p, c, stream)
                   : launch_gemm<kNT, 128, 0>(m, p, c, stream);
}

cudaError_t launch_ffn_glu_bwd(const FfnArgs& a, const void* dy, void* da, void* db, void* h,
                               cudaStream_t stream) {
  Maps m;
  GemmParams p{};
  p.rows = a.N;
  p.cols = a.F;
  p.tiles_n = ceil_div(a.F, kGluF);
  p.tiles = ceil_div(a.N, kTileM) * p.tiles_n;
  p.kb0 = p.kb1 = ceil_div(a.C, kBK);
  p.status = a.status;
  if (!encode_map_2d(&m.m[0], dy, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wd, a.C, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[2], a.x, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[3], a.wg, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[4], a.wu, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[5], da, a.N, a.F, 32, kHalfM) ||
      !encode_map_2d(&m.m[6], db, a.N, a.F, 32, kHalfM) ||
      !encode_map_2d(&m.m[7], h, a.N, a.F, 32, kHalfM))
    return cudaErrorInvalidValue;
  return launch_act<kGluBwd>(a.act, m, p, stream);
}

cudaError_t launch_ffn_dx(const FfnArgs& a, const void* da, const void* db, void* dx,
                          cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p{};
  p.rows = a.N;
  p.cols = a.C;
  p.tiles_n = ceil_div(a.C, bn);
  p.tiles = ceil_div(a.N, kTileM) * p.tiles_n;
  p.kb0 = p.kb1 = ceil_div(a.F, kBK);
  p.status = a.status;
  if (!encode_map_2d(&m.m[0], da, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], db, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[2], a.wg, a.F, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[3], a.wu, a.F, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[4], dx, a.N, a.C, 64, kHalfM))
    return cudaErrorInvalidValue;
  const int c = clusters_for(p.tiles);
  return bn == 256 ? launch_gemm<kNN, 256, 0>(m, p, c, stream)
                   : launch_gemm<kNN, 128, 0>(m, p, c, stream);
}

// Clusters and partial-tile bytes of the weight gradients.
namespace {
void wgrad_plan(const FfnArgs& a, int bn, GemmParams& p, int& clusters) {
  p.rows = a.F;
  p.cols = a.C;
  p.tiles_n = ceil_div(a.C, bn);
  p.tiles_p = ceil_div(a.F, kTileM);
  p.tiles = 3 * p.tiles_p * p.tiles_n;
  p.kb0 = ceil_div(a.N, kBK);
  clusters = clusters_for((int64_t)p.tiles * p.kb0);
  p.status = a.status;
}
}  // namespace

size_t ffn_wgrad_scratch(const FfnArgs& a) {
  const int bn = tile_cols(a.C);
  GemmParams p{};
  int clusters;
  wgrad_plan(a, bn, p, clusters);
  return (size_t)clusters * 2 * kTileM * bn * sizeof(float);
}

cudaError_t launch_ffn_wgrad(const FfnArgs& a, const void* dy, const void* da, const void* db,
                             const void* h, void* dwg, void* dwu, void* dwd, void* scratch,
                             cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p{};
  int c;
  wgrad_plan(a, bn, p, c);
  p.part = static_cast<float4*>(scratch);
  p.dwd = static_cast<__nv_bfloat16*>(dwd);
  if (!encode_map_2d(&m.m[0], da, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[1], db, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[2], h, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[3], a.x, a.N, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[4], dy, a.N, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[5], dwg, a.F, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[6], dwu, a.F, a.C, 64, kHalfM))
    return cudaErrorInvalidValue;
  cudaError_t e = bn == 256 ? launch_gemm<kTN, 256, 0>(m, p, c, stream)
                            : launch_gemm<kTN, 128, 0>(m, p, c, stream);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.tiles, 2, bn / 32);
  __nv_bfloat16 *g = static_cast<__nv_bfloat16*>(dwg), *u = static_cast<__nv_bfloat16*>(dwu);
  if (bn == 256)
    ffn_join_kernel<256><<<grid, 128, 0, stream>>>(p, c, g, u);
  else
    ffn_join_kernel<128><<<grid, 128, 0, stream>>>(p, c, g, u);
  return cudaGetLastError();
}

}  // namespace kmip
