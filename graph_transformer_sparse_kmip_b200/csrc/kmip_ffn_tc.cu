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
// MMAs, warps 0-15 of both CTAs read the accumulators (a quarter of the lanes
// and of the columns each), compute, and hand boxes of 32 rows by 32 columns
// to TMA stores through a corner of shared memory of their own, so no warp
// waits for another.  (Stores from registers, 32 bytes a lane, took 2.3
// cycles a sector: 7,700 cycles for dA, dB, h of a 256 x 128 tile.)
// Accumulators are double-buffered.  The backward's three need 384 of 512
// columns, so there dh alone has two buffers, and dh of the next tile runs
// while a and b are read.  (A step of 128 columns takes a pair as long as one
// of 256, 541 cycles, so dh costs twice its share.  As a product of its own
// with 256 columns, through 4 N F bytes of memory, it was no faster: 1.55 for
// 1.51 ms of a training step at 31,623 x 1,024 x 2,816.)
//
// The weight gradients contract over N: both operands have the contraction
// index outermost.  Tiles that fill all clusters are computed whole, all
// clusters at the same rows, so that operands come out of L2; the remaining
// tiles are cut along N into parts, fp32 partial tiles that a second kernel
// adds in order: the same bits every time.
#include <cuda.h>

#include "kmip_act.cuh"
#include "kmip_ffn.h"
#include "kmip_gemm.cuh"
#include "kmip_internal.h"
#include "kmip_launch.cuh"
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
constexpr int kEpiWarps = 16;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s
constexpr uint64_t kSettleNs = 10000000ull;     // 10 ms: what is in flight takes microseconds

constexpr int kBox = 32 * 32 * 2;    // a warp's output box

constexpr int boxes_of(int mode) { return mode == kGluBwd ? 3 : 1; }
constexpr int stages_of(int mode) { return mode == kGluBwd ? 4 : 6; }
constexpr int smem_of(int mode) {
  return 1024 + stages_of(mode) * kStage + kEpiWarps * boxes_of(mode) * kBox + 256;
}
static_assert(smem_of(kGlu) <= 232448 && smem_of(kGluBwd) <= 232448, "shared memory");

struct alignas(64) Maps {
  CUtensorMap m[5];    // operands
  CUtensorMap out[3];  // kGlu h; kNT, kNN out; kGluBwd dA, dB, h; kTN dWg, dWu
};

struct GemmParams {
  int rows, cols;      // output extent (kGlu, kGluBwd: N x F)
  int tiles_n;         // column tiles
  int tiles;           // all tiles
  int kb0, kb1;        // steps of the contraction, or of its two segments
  int whole;           // tiles computed whole
  int parts;           // parts of each of the others
  float4* part;        // their partial tiles, joined into out[0] (kNT, kNN) or
  __nv_bfloat16* out[3];  // dWg, dWu [rows][cols], dWd [cols][rows] (kTN)
  int tiles_p;         // kTN: row tiles of one of the three gradients
  int* status;
};

// A piece of a cluster's work: steps [k0, k0 + kn) of a tile; slot = the
// partial tile it goes to, or -1.
struct Item {
  int tile, k0, kn, slot;
};

// Cluster c takes tiles c, c + clusters, ...: first whole ones, then parts of
// the others, numbered with the tile running fastest.
struct Walk {
  int64_t i;
  int clusters, steps;
  __device__ Walk(int c, int n, int steps_) : i(c), clusters(n), steps(steps_) {}
  __device__ bool next(const GemmParams& p, Item& it) {
    if (i >= p.whole) {
      const int rest = p.tiles - p.whole;
      const int64_t j = i - p.whole;
      if (j >= (int64_t)rest * p.parts) return false;
      const int s = (int)(j / rest);
      it.tile = p.whole + (int)(j % rest);
      it.k0 = (int)((int64_t)steps * s / p.parts);
      it.kn = (int)((int64_t)steps * (s + 1) / p.parts) - it.k0;
      it.slot = p.parts > 1 ? (int)j : -1;
    } else {
      it.tile = (int)i;
      it.k0 = 0;
      it.kn = steps;
      it.slot = -1;
    }
    i += clusters;
    return true;
  }
};

// 16 packed bf16 columns of a row into a box of 32 (64-byte rows with their
// swizzle): the left (c = 0) or right half.
__device__ __forceinline__ void put_box(uint32_t box, int lane, int c, const uint32_t (&w)[8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t at = box + lane * 64 + (((2 * c + q) ^ ((lane >> 1) & 3)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack2(float2 v) { return pack2(v.x, v.y); }

template <int MODE, int BN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ffn_gemm_kernel(const __grid_constant__ Maps maps, const GemmParams p) {
  using T = __nv_bfloat16;
  constexpr int kStages = stages_of(MODE);
  constexpr int kBufs = MODE == kGluBwd ? 1 : 2;
  constexpr int kBufCols = MODE == kGluBwd ? 0 : BN;
  constexpr int kTmemCols = MODE == kGluBwd ? 512 : 2 * BN;
  constexpr int kSegs = MODE == kGluBwd ? 2 : 1;
  // kNN's two products are one contraction here
  const int steps = MODE == kNN ? p.kb0 + p.kb1 : p.kb0;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t boxes = base + kStages * kStage;
  const uint32_t bars = boxes + kEpiWarps * boxes_of(MODE) * kBox;
  const uint32_t full = bars, empty = bars + 8 * kStages;
  const uint32_t tfull = empty + 8 * kStages, tempty = tfull + 16, settled = tempty + 16;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_store;
  volatile int* abort_flag = &abort_store;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  uint32_t issued = 0;  // steps that the producer has loaded

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
    mbar_init(settled, 1);
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
  after_previous();

  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = map_to_cta(full, 0);
      Walk walk(cluster, clusters, steps);
      Item it;
      bool ok = true;
      while (ok && walk.next(p, it)) {
        const int mt = it.tile / p.tiles_n, nt = it.tile % p.tiles_n;
        for (int seg = 0; seg < kSegs && ok; ++seg) {
          const int kn = seg ? p.kb1 : it.kn;
          for (int kb = 0; kb < kn; ++kb, ++issued) {
            const uint32_t s = issued % kStages, ph = (issued / kStages) & 1;
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
              const int second = it.k0 + kb >= p.kb0;
              const int ks = k - second * p.kb0 * kBK;
              tma_load_2d_pair(a, &maps.m[second], bar, ks, mt * kTileM + rank * kHalfM);
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tma_load_2d_pair(b + j * 8192, &maps.m[2 + second], bar,
                                 nt * BN + rank * (BN / 2) + 64 * j, ks);
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
      Walk walk(cluster, clusters, steps);
      Item it;
      bool ok = true;
      while (ok && walk.next(p, it)) {
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
          const int kn = seg ? p.kb1 : it.kn;
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
              mma_bf16_pair(d, da + q * sa, db + q * sb, idesc, kb || q);
            mma_commit_pair(empty + 8 * s);
          }
        }
        if (ok) mma_commit_pair(tfull + 8 * buf);
        ++tile_no;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tempty0 = map_to_cta(tempty, 0);
    const uint32_t box = boxes + warp * boxes_of(MODE) * kBox;
    // The warp's boxes are free again / filled and on their way out.
    auto boxes_free = [&] {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    };
    auto send = [&](int n, int first, int x, int y) {
      fence_async_shared();
      __syncwarp();
      if (lane == 0 && y < p.rows && x < p.cols) {
        for (int i = 0; i < n; ++i) tma_store_2d(&maps.out[first + i], box + i * kBox, x, y);
        bulk_commit();
      }
    };
    uint32_t tile_no = 0;
    Walk walk(cluster, clusters, steps);
    Item it;
    while (walk.next(p, it)) {
      const int mt = it.tile / p.tiles_n, nt = it.tile % p.tiles_n;
      const uint32_t buf = kBufs == 2 ? tile_no & 1 : 0;
      const uint32_t use = kBufs == 2 ? tile_no >> 1 : tile_no;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(tfull + 8 * buf, use & 1, abort_flag, kTimeoutNs)))
        break;
      tc_fence_after();
      const uint32_t acc = lanes + buf * kBufCols;
      // This warp has read what it needs of the accumulators.
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
      };
      const int m0 = (MODE == kTN ? mt % p.tiles_p : mt) * kTileM + (int)rank * kHalfM +
                     (warp & 3) * 32;

      if constexpr (MODE == kGlu) {
        const int f0 = nt * kGluF + quarter * 32;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = quarter * 32 + c * 16;
          float g[16], u[16];
          tmem_ld16(acc + col, g);
          tmem_ld16(acc + kGluF + col, u);
          tmem_ld_wait_all();
          reg_fence(g);
          reg_fence(u);
          if (c == 1) release();
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = pack2(mul2(act_value2<T, ACT>(make_float2(g[2 * e], g[2 * e + 1])),
                              make_float2(u[2 * e], u[2 * e + 1])));
          if (c == 0) boxes_free();
          put_box(box, lane, c, w);
        }
        send(1, 0, f0, m0);
      } else if constexpr (MODE == kGluBwd) {
        const uint32_t acc_dh = lanes + 2 * kGluF + (tile_no & 1) * kGluF;
        const int f0 = nt * kGluF + quarter * 32;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = quarter * 32 + c * 16;
          float a[16], b[16], dh[16];
          tmem_ld16(acc + col, a);
          tmem_ld16(acc + kGluF + col, b);
          tmem_ld16(acc_dh + col, dh);
          tmem_ld_wait_all();
          reg_fence(a);
          reg_fence(b);
          reg_fence(dh);
          if (c == 1) release();
          uint32_t wa[8], wb[8], wh[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 av = make_float2(a[2 * e], a[2 * e + 1]);
            const float2 bv = make_float2(b[2 * e], b[2 * e + 1]);
            const float2 dv = make_float2(dh[2 * e], dh[2 * e + 1]);
            float2 f, g;
            act_both2<T, ACT>(av, f, g);
            wa[e] = pack2(mul2(mul2(dv, bv), g));
            wb[e] = pack2(mul2(dv, f));
            wh[e] = pack2(mul2(f, bv));
          }
          if (c == 0) boxes_free();
          put_box(box, lane, c, wa);
          put_box(box + kBox, lane, c, wb);
          put_box(box + 2 * kBox, lane, c, wh);
        }
        send(3, 0, f0, m0);
      } else {
        const int prob = MODE == kTN ? mt / p.tiles_p : 0;
        float4* part = p.part + ((int64_t)it.slot * 2 + rank) * (BN / 4 * kHalfM);
#pragma unroll 1
        for (int j = 0; j < BN / 128; ++j) {
          const int col = quarter * (BN / 4) + j * 32, n = nt * BN + col;
          float v[32];
          tmem_ld32(acc + col, v);
          tmem_ld_wait_all();
          reg_fence(v);
          if (j == BN / 128 - 1) release();
          if (it.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              part[(int64_t)(col / 4 + e) * kHalfM + row] =
                  make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          } else if (MODE == kTN && prob == 2) {
            // dWd is [C][F]: neighbouring lanes hold neighbouring F
            if (m0 + lane < p.rows) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (n + e < p.cols)
                  p.out[2][(int64_t)(n + e) * p.rows + m0 + lane] = __float2bfloat16_rn(v[e]);
            }
          } else {
            uint32_t w[2][8];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e / 8][e % 8] = pack2(v[2 * e], v[2 * e + 1]);
            boxes_free();
            put_box(box, lane, 0, w[0]);
            put_box(box, lane, 1, w[1]);
            send(1, prob, n, m0);
          }
        }
      }
      ++tile_no;
    }
    if (lane == 0) bulk_wait_all();
  }

  // ------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // A wait ran out, so work may still be in flight; neither CTA frees tensor
    // memory or leaves before it has landed, or as long as kSettleNs later.
    const auto settle = [](uint32_t bar, uint32_t parity) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(bar, parity) && global_ns() - t0 < kSettleNs) {
      }
    };
    if (warp == kEpiWarps && lane == 0) {
      if (rank == 0) {  // where the copies of both CTAs are counted
        for (uint32_t s = 0; s < (uint32_t)kStages; ++s)
          if (issued > s) settle(full + 8 * s, (issued - 1 - s) / kStages & 1);
      } else {          // copies of a step that the other CTA did not begin
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kSettleNs) {
        }
      }
    }
    if (warp == kEpiWarps + 1 && lane == 0) {
      if (rank == 0) mma_commit_pair(settled);
      settle(settled, 0);
    }
  }
  __syncwarp();
  cluster_sync();
  if (*abort_flag && threadIdx.x == 0) record_status(p.status, KMIP_ERR_TIMEOUT);
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Adds partial tiles in order.  Grid: (tile that
// was cut, CTA of the pair, 8-column group); 128 threads, one per row.
template <int BN>
__global__ void __launch_bounds__(128) ffn_join_kernel(const GemmParams p) {
  after_previous();
  const int rest = p.tiles - p.whole, tile = p.whole + blockIdx.x, rank = blockIdx.y;
  const int row = threadIdx.x;
  float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  const float4* src = p.part + ((int64_t)blockIdx.x * 2 + rank) * (BN / 4 * kHalfM) +
                      (int64_t)blockIdx.z * 2 * kHalfM + row;
  const int64_t step = (int64_t)rest * 2 * (BN / 4 * kHalfM);
#pragma unroll 4
  for (int s = 0; s < p.parts; ++s, src += step) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 t = src[e * kHalfM];
      v[e].x += t.x;
      v[e].y += t.y;
      v[e].z += t.z;
      v[e].w += t.w;
    }
  }
  const int mt = tile / p.tiles_n, nt = tile % p.tiles_n, prob = mt / p.tiles_p;
  const int r = (mt % p.tiles_p) * kTileM + rank * kHalfM + row;
  const int c = nt * BN + blockIdx.z * 8;
  if (r >= p.rows || c >= p.cols) return;  // cols is a multiple of 8
  if (prob == 2) {
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p.out[2][(int64_t)(c + e) * p.rows + r] = __float2bfloat16_rn(f[e]);
  } else {
    *reinterpret_cast<uint4*>((prob ? p.out[1] : p.out[0]) + (int64_t)r * p.cols + c) =
        make_uint4(pack2(v[0].x, v[0].y), pack2(v[0].z, v[0].w), pack2(v[1].x, v[1].y),
                   pack2(v[1].z, v[1].w));
  }
}

// ------------------------------------------------------------------ host side

int clusters_for(int64_t tiles) {
  const int most = device_sm_count() / 2;
  return (int)(tiles < most ? tiles : most);
}

template <int MODE, int BN, int ACT>
cudaError_t launch_gemm(const Maps& maps, const GemmParams& p, int clusters, cudaStream_t stream,
                        bool next) {
  auto kern = ffn_gemm_kernel<MODE, BN, ACT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_of(MODE));
  if (e != cudaSuccess) return e;
  if (next) return launch_next(kern, dim3(2 * clusters), kThreads, smem_of(MODE), stream, maps, p);
  kern<<<2 * clusters, kThreads, smem_of(MODE), stream>>>(maps, p);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_act(int act, const Maps& maps, const GemmParams& p, cudaStream_t stream) {
  const int c = clusters_for(p.tiles);
  switch (act) {
    case KMIP_ACT_SILU: return launch_gemm<MODE, 256, KMIP_ACT_SILU>(maps, p, c, stream, false);
    case KMIP_ACT_GELU: return launch_gemm<MODE, 256, KMIP_ACT_GELU>(maps, p, c, stream, false);
    case KMIP_ACT_RELU: return launch_gemm<MODE, 256, KMIP_ACT_RELU>(maps, p, c, stream, false);
    default: return launch_gemm<MODE, 256, KMIP_ACT_NONE>(maps, p, c, stream, false);
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Columns of an output tile: 256 reads A half as often, but is not worth a
// quarter more of columns behind the edge.
int tile_cols(int cols) {
  return ceil_div(cols, 256) * 256 * 4 >= ceil_div(cols, 128) * 128 * 5 ? 128 : 256;
}

// Steps of the contraction that a part costs beside its products (its first
// loads, its partial tile written and read again by one more launch: 5 to 6 us
// where a step takes 0.4 us).
constexpr int kPartCost = 14;

// Output of rows x cols in tiles of kTileM x bn, a contraction of length k;
// `times` outputs side by side (kTN), `segs` contractions after one another.
// With `split`, tiles beyond what fills all clusters evenly are cut into the
// number of parts whose last round of clusters idles least.
GemmParams params(const FfnArgs& a, int rows, int cols, int bn, int k, bool split = false,
                  int segs = 1, int times = 1) {
  GemmParams p{};
  p.rows = rows;
  p.cols = cols;
  p.tiles_n = ceil_div(cols, bn);
  p.tiles_p = ceil_div(rows, kTileM);
  p.tiles = times * p.tiles_p * p.tiles_n;
  p.kb0 = p.kb1 = ceil_div(k, kBK);
  p.whole = p.tiles;
  p.parts = 1;
  p.status = a.status;
  if (split) {
    const int all = device_sm_count() / 2, steps = segs * p.kb0;
    p.whole = p.tiles / all * all;
    const int rest = p.tiles - p.whole;
    int64_t best = rest ? steps - kPartCost : 0;  // or left whole
    for (int s = 2; s <= steps && (int64_t)rest * s <= 4 * all; ++s) {
      const int64_t cost =
          (int64_t)ceil_div((int64_t)rest * s, all) * (ceil_div(steps, s) + kPartCost);
      if (cost < best) {
        best = cost;
        p.parts = s;
      }
    }
    if (p.parts == 1) p.whole = p.tiles;
  }
  return p;
}

size_t part_bytes(const GemmParams& p, int bn) {
  return (size_t)(p.tiles - p.whole) * p.parts * kTileM * bn * sizeof(float);
}

// The GEMM (after another kernel of the call) and, where tiles were cut, the
// join of their parts.
template <int MODE>
cudaError_t launch_split(const Maps& m, const GemmParams& p, int bn, cudaStream_t stream) {
  const int rest = p.tiles - p.whole;
  const int c = clusters_for(p.whole + (int64_t)rest * p.parts);
  const cudaError_t e = bn == 256 ? launch_gemm<MODE, 256, 0>(m, p, c, stream, true)
                                  : launch_gemm<MODE, 128, 0>(m, p, c, stream, true);
  if (e != cudaSuccess || !rest) return e;
  const dim3 grid(rest, 2, bn / 8);
  return launch_next(bn == 256 ? ffn_join_kernel<256> : ffn_join_kernel<128>, grid, 128, 0, stream,
                     p);
}

GemmParams down_params(const FfnArgs& a, int bn) {
  return params(a, a.N, a.C, bn, a.F, true);
}
GemmParams dx_params(const FfnArgs& a, int bn) {
  return params(a, a.N, a.C, bn, a.F, true, 2);
}
GemmParams wgrad_params(const FfnArgs& a, int bn) {
  return params(a, a.F, a.C, bn, a.N, true, 1, 3);
}

bool out_map(CUtensorMap* m, const void* ptr, int rows, int cols) {
  return encode_map_2d(m, ptr, rows, cols, 32, 32);
}

}  // namespace

cudaError_t launch_ffn_glu(const FfnArgs& a, void* h, cudaStream_t stream) {
  Maps m;
  const GemmParams p = params(a, a.N, a.F, kGluF, a.C);
  if (!encode_map_2d(&m.m[0], a.x, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wg, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[2], a.wu, a.F, a.C, 64, kGluF) || !out_map(&m.out[0], h, a.N, a.F))
    return cudaErrorInvalidValue;
  return launch_act<kGlu>(a.act, m, p, stream);
}

size_t ffn_fwd_scratch(const FfnArgs& a) {
  const int bn = tile_cols(a.C);
  return part_bytes(down_params(a, bn), bn);
}

cudaError_t launch_ffn_down(const FfnArgs& a, const void* h, void* y, void* scratch,
                            cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p = down_params(a, bn);
  p.part = static_cast<float4*>(scratch);
  p.out[0] = static_cast<__nv_bfloat16*>(y);
  if (!encode_map_2d(&m.m[0], h, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wd, a.C, a.F, 64, bn / 2) || !out_map(&m.out[0], y, a.N, a.C))
    return cudaErrorInvalidValue;
  return launch_split<kNT>(m, p, bn, stream);
}

cudaError_t launch_ffn_glu_bwd(const FfnArgs& a, const void* dy, void* da, void* db, void* h,
                               cudaStream_t stream) {
  Maps m;
  const GemmParams p = params(a, a.N, a.F, kGluF, a.C);
  if (!encode_map_2d(&m.m[0], dy, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], a.wd, a.C, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[2], a.x, a.N, a.C, 64, kHalfM) ||
      !encode_map_2d(&m.m[3], a.wg, a.F, a.C, 64, kGluF) ||
      !encode_map_2d(&m.m[4], a.wu, a.F, a.C, 64, kGluF) || !out_map(&m.out[0], da, a.N, a.F) ||
      !out_map(&m.out[1], db, a.N, a.F) || !out_map(&m.out[2], h, a.N, a.F))
    return cudaErrorInvalidValue;
  return launch_act<kGluBwd>(a.act, m, p, stream);
}

size_t ffn_bwd_scratch(const FfnArgs& a) {
  const int bn = tile_cols(a.C);
  const size_t x = part_bytes(dx_params(a, bn), bn), w = part_bytes(wgrad_params(a, bn), bn);
  return x > w ? x : w;
}

cudaError_t launch_ffn_dx(const FfnArgs& a, const void* da, const void* db, void* dx,
                          void* scratch, cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p = dx_params(a, bn);
  p.part = static_cast<float4*>(scratch);
  p.out[0] = static_cast<__nv_bfloat16*>(dx);
  if (!encode_map_2d(&m.m[0], da, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[1], db, a.N, a.F, 64, kHalfM) ||
      !encode_map_2d(&m.m[2], a.wg, a.F, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[3], a.wu, a.F, a.C, 64, kBK) || !out_map(&m.out[0], dx, a.N, a.C))
    return cudaErrorInvalidValue;
  return launch_split<kNN>(m, p, bn, stream);
}

cudaError_t launch_ffn_wgrad(const FfnArgs& a, const void* dy, const void* da, const void* db,
                             const void* h, void* dwg, void* dwu, void* dwd, void* scratch,
                             cudaStream_t stream) {
  Maps m;
  const int bn = tile_cols(a.C);
  GemmParams p = wgrad_params(a, bn);
  p.part = static_cast<float4*>(scratch);
  p.out[0] = static_cast<__nv_bfloat16*>(dwg);
  p.out[1] = static_cast<__nv_bfloat16*>(dwu);
  p.out[2] = static_cast<__nv_bfloat16*>(dwd);
  if (!encode_map_2d(&m.m[0], da, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[1], db, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[2], h, a.N, a.F, 64, kBK) ||
      !encode_map_2d(&m.m[3], a.x, a.N, a.C, 64, kBK) ||
      !encode_map_2d(&m.m[4], dy, a.N, a.C, 64, kBK) || !out_map(&m.out[0], dwg, a.F, a.C) ||
      !out_map(&m.out[1], dwu, a.F, a.C))
    return cudaErrorInvalidValue;
  return launch_split<kTN>(m, p, bn, stream);
}

}  // namespace kmip
