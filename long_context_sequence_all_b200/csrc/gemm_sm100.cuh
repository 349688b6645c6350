// Matrix products C[M][N] = A[M][K] B[N][K]^T on the 5th-generation tensor
// cores with an epilogue of the caller's, for the token-wise operators (the
// linear product and its gradients, the linear loss and its gradients).
//
// bf16 operands, fp32 accumulators.  A cluster of two CTAs on neighbouring SMs
// computes one 256 x 256 tile (tcgen05 cta_group::2, M = 256; 256 x 128 where
// that puts more SMs to work on a small product): each CTA holds 128 rows of A,
// half the rows of B and the accumulator of its own 128 rows, so
// every byte of B in shared memory feeds two tensor cores and a k-step of 64
// costs each SM 32 KB of loads instead of the 48 KB of a 128 x 256 tile of its
// own.  K runs in steps of 64 columns (one 128-byte swizzle span).  The kernel
// is persistent: one cluster per SM pair walks the work units (a tile, or one
// of `splits` parts of a tile's k-steps).
//
// Warps (384 threads): 0 TMA (both CTAs load their own halves, all completing
// on the leader's barriers), 1 MMA issue (the leader CTA's), 2 tensor memory,
// 4-11 epilogue: two warpgroups take the two halves of the columns of the CTA's
// 128 rows, one row a thread, while the next tile fills the other accumulator.
//
// An operand is K-major (rows of K contiguous elements, 128-row boxes) or
// MN-major (rows of M or N contiguous elements, 64 x 64 boxes).  Elements
// past any edge are read as zeros and never stored, so M, N and K are free.
//
// A thread holds one row of C, so its own 16-byte stores would fill half a
// 32-byte sector each, 32 rows apart.  Outputs go through shared memory
// instead, 128 bytes of a warp's 32 rows at a time, and leave by TMA (8192 x 2560
// -> 2 x 10240 gated with z kept: 711 -> 675 us; 8192 x 64 -> 8192: 28 us).
//
// Every wait is bounded (ULY_ERR_TIMEOUT); a launch that gives up lets its
// copies land before it frees its tensor memory and returns.
#pragma once

#include <limits.h>

#include <type_traits>

#include "prof.cuh"
#include "sm100.cuh"

namespace uly {
namespace gemm {

using namespace sm100;

constexpr int kTile = 256;       // rows of a cluster's tile, and its columns unless it is a narrow one (128)
constexpr int kNarrow = 128;
constexpr int kHalf = 128;       // rows of A in one CTA
constexpr int kBK = 64;
// Elements: operands of this library's own making have rows of whole 128-byte
// lines (dW of 1503 tokens, 520 over 32003: 73 us with rows of 1040 and 64016
// bytes, 60 this way).
constexpr int kRowAlign = 64;
constexpr int kOutSlots = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kABytes = kHalf * kBK * 2;             // 16 KB
constexpr uint32_t kOutSlot = 32 * 128;                   // 32 rows of 64 two-byte or 32 four-byte columns
// Shared memory of one CTA for tiles of TN columns: the ring of k-steps, the
// epilogue warps' output slots, barriers.
template <int TN>
struct Layout {
  static constexpr int kStages = TN == kTile ? 5 : 6;
  static constexpr uint32_t kStage = kABytes + TN / 2 * kBK * 2;
  static constexpr uint32_t kOffOut = kStages * kStage;
  static constexpr uint32_t kOffBar = kOffOut + kEpiWarps * kOutSlots * kOutSlot;
  static constexpr uint32_t kBytes = kOffBar + 256 + 1024;   // barriers + alignment slack
};
constexpr long long kLandCycles = 1 << 20;                 // after giving up: the copies in flight land (~0.5 ms)

// The product and how it is cut into work.
struct Shape {
  int m_tiles, n_tiles;
  int full, splits;     // tiles taken whole, and the parts of each other one
  int k_steps;          // ceil(K / 64)
  int group_m;          // tiles in flight form blocks of group_m rows of tiles (operands shared in L2)
  int b_step, b_half;   // B row of tile nt, CTA r: nt * b_step + r * b_half
  int *err;
  long long wait_limit;
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of the same shared-memory location in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Relaxed: what it hands over is tensor memory that has been read into registers.
// A release would wait for this thread's stores too (37 tokens' dW over 151936 x
// 2560, one k-step a tile: 207 us; this way, and with 128-byte rows, 157).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile load into this CTA's shared memory, completing on a barrier of the
// CTA pair's leader.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive once on the barrier at `bar`'s offset in both CTAs when every MMA
// this thread issued so far has completed.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

// One epilogue warp's way out: 32 rows (one a lane) x 128 bytes of columns a slot,
// staged with the 128-byte swizzle of make_out_map(); two slots, one leaves while
// the other is filled.
struct OutRing {
  uint32_t base, turn;   // turn: which slot
  int lane;
  __device__ __forceinline__ uint32_t chunk(int row, int c) const {   // 16 bytes
    return base + turn * kOutSlot + row * 128 + ((c ^ (row & 7)) << 4);
  }
  // All lanes of the warp together: the slot is free ...
  __device__ __forceinline__ void begin() {
    if (lane == 0) bulk_wait_group_read<1>();
    __syncwarp();
  }
  // ... take something read along the rows (v[i]: chunk lane % 8 of row 4 i + lane / 8)
  // to give it back a row a lane, half i of the row ...
  __device__ __forceinline__ void stage(const uint4 (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) st_shared_v4(chunk(4 * i + (lane >> 3), lane & 7), v[i].x, v[i].y, v[i].z, v[i].w);
    __syncwarp();
  }
  __device__ __forceinline__ void read(int i, uint32_t (&v)[16]) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[4 * c]), "=r"(v[4 * c + 1]), "=r"(v[4 * c + 2]), "=r"(v[4 * c + 3])
                   : "r"(chunk(lane, 4 * i + c))
                   : "memory");
  }
  // ... take half i of this lane's columns (64 of two bytes, packed, or 32 of four) ...
  __device__ __forceinline__ void write(int i, const uint32_t (&v)[16]) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) st_shared_v4(chunk(lane, 4 * i + c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  }
  // ... and leave.
  __device__ __forceinline__ void end(const CUtensorMap *map, int col0, int row0) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, base + turn * kOutSlot, col0, row0);
      bulk_commit_group();
    }
    turn ^= 1;
  }
};

// A tile's place; tiles go down group_m rows before the next column.
__device__ __forceinline__ void place_of(const Shape &s, int tile, int &mt, int &nt) {
  const int per = s.group_m * s.n_tiles, g = tile / per, in = tile - g * per;
  const int first = g * s.group_m, rows = min(s.group_m, s.m_tiles - first);
  nt = in / rows;
  mt = first + in - nt * rows;
}
// Which tile and which of its k-steps a work unit is.  The parts of a cut tile
// follow one another.
struct Unit {
  int mt, nt, part;   // part: index of its partial tile, -1 for a whole tile
  int k0, k1;
};
__device__ __forceinline__ Unit unit_of(const Shape &s, int u) {
  Unit r;
  const int v = u - s.full;
  if (v < 0) {
    place_of(s, u, r.mt, r.nt);
    r.part = -1;
    r.k0 = 0;
    r.k1 = s.k_steps;
  } else {
    const int t = v / s.splits, split = v - t * s.splits;
    place_of(s, s.full + t, r.mt, r.nt);
    r.part = s.splits > 1 ? v : -1;
    r.k0 = (int)((long long)s.k_steps * split / s.splits);
    r.k1 = (int)((long long)s.k_steps * (split + 1) / s.splits);
  }
  return r;
}
__host__ __device__ __forceinline__ int units_of(const Shape &s) {
  return s.full + (s.m_tiles * s.n_tiles - s.full) * s.splits;
}

// A partial tile [256][TN]: this warp's 32 rows of half the columns, fp32.
template <int TN>
__device__ __forceinline__ void store_partial(const CUtensorMap *map, const Unit &w, uint32_t acc, int row_in_tile,
                                              int half, OutRing &out) {
#pragma unroll 1
  for (int c = half * TN / 2; c < (half + 1) * TN / 2; c += 32) {
    uint32_t a[32], v[16];
    tmem_ld32(acc + c, a);
    out.begin();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = a[16 * h + e];
      out.write(h, v);
    }
    out.end(map, c, w.part * kTile + row_in_tile);
  }
}

// Epi::Params,
//   Epi::before<TN>(params, unit, row0, half, lane): what the epilogue of a whole
//   tile asks for before its product is there (rows [row0, row0 + 32)), and
//   Epi::tile<TN>(params, unit, acc, row, half, asked, out): one thread's TN / 2
//   accumulators (read from tensor memory, that half of the columns from acc on,
//   before it returns) of C row `row`, in tile column unit.nt.
struct Nothing {};

template <class Epi, int TN, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_pair_sm100_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmPart, const __grid_constant__ Shape sh,
                           const __grid_constant__ typename Epi::Params ep) {
  using L = Layout<TN>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  enum { B_FULL = 0, B_EMPTY = kStages, B_ACCF = 2 * kStages, B_ACCE = B_ACCF + 2, B_N = B_ACCE + 2 };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffBar + 8 * B_N);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffBar + 8 * B_N + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int units = units_of(sh);

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_N; ++i) mbar_init(bar(i), i >= B_ACCE ? 2 * kEpiWarps : 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any arrival crosses over
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 1;   // the ring's slots start free
      bool ok = true;
      for (int u = cluster; ok && u < units; u += clusters) {
        const Unit w = unit_of(sh, u);
        const int a0 = w.mt * kTile + (int)rank * kHalf, b0 = w.nt * sh.b_step + (int)rank * sh.b_half;
        for (int k = w.k0; k < w.k1; ++k) {
          ok = mbar_wait(bar(B_EMPTY + stage), phase, abort_flag, sh.err, sh.wait_limit);
          if (!ok) break;
          const uint32_t sA = sb + stage * L::kStage, sB = sA + kABytes;
          // the leader's barrier counts the bytes of both CTAs
          const uint32_t full = map_cta(bar(B_FULL + stage), 0);
          if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + stage), 2 * L::kStage);
          if (A_MN) {
            tma_load_2d_pair(sA, &tmA, full, a0, k * kBK);
            tma_load_2d_pair(sA + 8192, &tmA, full, a0 + 64, k * kBK);
          } else {
            tma_load_2d_pair(sA, &tmA, full, k * kBK, a0);
          }
          if (B_MN) {
            tma_load_2d_pair(sB, &tmB, full, b0, k * kBK);
            if (TN == kTile) tma_load_2d_pair(sB + 8192, &tmB, full, b0 + 64, k * kBK);
          } else {
            tma_load_2d_pair(sB, &tmB, full, k * kBK, b0);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kTile, TN, A_MN, B_MN);
      // K-major: 16 K-elements are 32 bytes along a row; MN-major: 16 K-rows
      // are 2048 bytes, the 64-element MN chunks 8 KB apart (LBO)
      constexpr uint32_t astep = A_MN ? 2048 : 32, bstep = B_MN ? 2048 : 32;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;
      for (int u = cluster; ok && u < units; u += clusters, ++it) {
        const Unit w = unit_of(sh, u);
        const int buf = it & 1;
        if (it >= 2) {
          ok = mbar_wait(bar(B_ACCE + buf), (uint32_t)(((it >> 1) - 1) & 1), abort_flag, sh.err, sh.wait_limit);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t acc = tmem + buf * TN;
        for (int k = w.k0; k < w.k1; ++k) {
          const uint32_t sA = sb + stage * L::kStage, sB = sA + kABytes;
          const uint64_t da = A_MN ? sdesc_sw128(sA, 8192, 1024) : sdesc_sw128(sA, 16, 1024);
          const uint64_t db = B_MN ? sdesc_sw128(sB, 8192, 1024) : sdesc_sw128(sB, 16, 1024);
          ok = mbar_wait(bar(B_FULL + stage), phase, abort_flag, sh.err, sh.wait_limit);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma_pair(acc, sdesc_add(da, kk * astep), sdesc_add(db, kk * bstep), idesc,
                     (k > w.k0 || kk > 0) ? 1u : 0u);
          tc_commit_pair(bar(B_EMPTY + stage));
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        tc_commit_pair(bar(B_ACCF + buf));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    OutRing out{sb + L::kOffOut + (uint32_t)(warp - 4) * kOutSlots * kOutSlot, 0, lane};
    int it = 0;
    for (int u = cluster; u < units; u += clusters, ++it) {
      const int buf = it & 1;
      const Unit w = unit_of(sh, u);
      const int row0 = (int)rank * kHalf + quarter * 32;
      auto asked = Epi::template before<TN>(ep, w, w.part < 0 ? w.mt * kTile + row0 : INT_MAX, half, lane);
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_ACCF + buf), (uint32_t)((it >> 1) & 1), abort_flag, sh.err,
                                             sh.wait_limit)))
        break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + buf * TN;
      if (w.part >= 0) store_partial<TN>(&tmPart, w, acc, row0, half, out);
      else Epi::template tile<TN>(ep, w, acc, w.mt * kTile + row0 + lane, half, asked, out);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(map_cta(bar(B_ACCE + buf), 0));
    }
    if (lane == 0) bulk_wait_group_read<0>();   // the slots' memory outlives the copies out of it
  }

  // Normal end: every copy was consumed by an MMA and every MMA was waited for
  // by both CTAs' epilogues.  After giving up, copies and MMAs may still be in
  // flight: give them time to finish before the pair parts.
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    const long long t0 = clock64();
    while (clock64() - t0 < kLandCycles) __nanosleep(1000);
  }
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------- host

// 2-D map of a [rows][inner] matrix with rows `stride` elements apart.
// Elements past either edge read as zero and are not written.
inline bool make_map_of(CUtensorMap *map, const void *base, long long inner, long long rows, long long stride,
                        int box_cols, int box_rows, CUtensorMapSwizzle swizzle, bool f32 = false) {
  static std::atomic<void *> fn{nullptr};
  void *p = fn.load(std::memory_order_acquire);
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn.store(p, std::memory_order_release);
  }
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)stride * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)(
             map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An operand: boxes of 64 columns and box_rows rows (128: K-major, 64: MN-major).
inline bool make_map(CUtensorMap *map, const void *base, long long inner, long long rows, long long stride,
                     int box_rows) {
  return make_map_of(map, base, inner, rows, stride, kBK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
// An output leaving through an OutRing.
inline bool make_out_map(CUtensorMap *map, const void *base, long long inner, long long rows, long long stride,
                         bool f32 = false) {
  return make_map_of(map, base, inner, rows, stride, f32 ? 32 : 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, f32);
}

// The tiles' width, how many of them are taken whole and the parts of each of the
// others: the least of a sum of microseconds.  Whole tiles in full turns of the SM
// pairs; a turn costs k_steps (0.3, bound by the tensor cores; 0.25 for a narrow
// tile, bound by its loads), the last one ceil(tiles left * splits / pairs) of
// k_steps / splits and, if cut, a second kernel over fp32 partial tiles (written
// and read once, mostly in L2) of at most `budget` bytes; the last tile's epilogue
// is not hidden.  A tile of many steps has as many parts as there are pairs (32
// tokens' dx over 143987 columns, 88 wide: 26 us, 106 in eight parts).
// 320 tiles of 320 steps on 74 pairs: 4 turns and 24 tiles cut in 3, 4.33 turns
// instead of 5.  1003 x 1032 -> 1544: 52 narrow tiles 11.9 us, 28 wide ones 13.8;
// 256 x 10240 -> 2560: 10 wide tiles cut in 7 20.6 us, narrow ones 25.7.
struct Cut {
  int tn = kTile;     // columns of a tile
  int full = 0, splits = 1;
  size_t bytes = 0;   // of the partial tiles
  double us = 0;      // the sum
};
inline Cut choose_cut(long long m_tiles, long long n_tiles, long long n_narrow, long long k_steps,
                      size_t budget = SIZE_MAX) {
  const int pairs = device_sm_count() / 2, steps = (int)k_steps;
  Cut best;
  double best_us = 1e300;   // the parts looked at: 1 to 8, then an eighth more each time
  for (int tn : {kTile, kNarrow}) {
    const long long tiles = m_tiles * (tn == kTile ? n_tiles : n_narrow);
    const int left = (int)(tiles % pairs);
    const double step = tn == kTile ? 0.3 : 0.25, end = tn == kTile ? 2.0 : 1.2;
    const double fixed = (double)(tiles / pairs) * (double)k_steps * step + end;
    for (int s = 1; s <= pairs && (s == 1 || (left > 0 && s * 2 <= steps)); s += 1 + s / 8) {
      const size_t bytes = s == 1 ? 0 : (size_t)left * s * kTile * tn * sizeof(float);
      if (bytes > budget) break;
      const double us = fixed + (double)((left * s + pairs - 1) / pairs) * (double)((steps + s - 1) / s) * step +
                        (s == 1 ? 0.0 : 3.5 + (double)bytes * 2.0 / 1e7);
      if (us < best_us * 0.98) {
        best_us = us;
        best.tn = tn;
        best.full = (int)(s == 1 ? tiles : tiles - left);
        best.splits = s;
        best.bytes = bytes;
      }
    }
  }
  best.us = best_us;
  return best;
}
inline long long tiles_of(long long n, int tile = kTile) { return (n + tile - 1) / tile; }

// Work units, raster and rest of a launch.  `per_col` rows of B stand behind one
// output column (1, or 2: N rows further on).
inline Shape make_shape(long long M, long long N, long long K, int per_col, const Cut &cut) {
  Shape s = {};
  const int n_tile = cut.tn / per_col;
  s.m_tiles = (int)tiles_of(M);
  s.n_tiles = (int)tiles_of(N, n_tile);
  s.full = cut.full;
  s.splits = cut.splits;
  s.k_steps = (int)((K + kBK - 1) / kBK);
  s.group_m = 8;
  s.b_step = n_tile;
  s.b_half = per_col == 1 ? cut.tn / 2 : (int)N;
  s.err = error_word();
  s.wait_limit = wait_limit_cycles();
  return s;
}
// K-major rows of B in one box (one CTA's share of a tile).
inline int b_box(const Cut &cut) { return cut.tn / 2; }

// `part`: cut.bytes for the partial tiles of a shape that has any.
template <class Epi, int TN, bool A_MN, bool B_MN>
uly_status launch_tn(const CUtensorMap &ta, const CUtensorMap &tb, const Shape &s, const typename Epi::Params &ep,
                     float *part, cudaStream_t stream) {
  static std::atomic<uint64_t> optin{0};
  auto kernel = gemm_pair_sm100_kernel<Epi, TN, A_MN, B_MN>;
  if (!smem_optin(kernel, Layout<TN>::kBytes, optin)) return ULY_ERR_CUDA;
  const int units = units_of(s), pairs = device_sm_count() / 2;
  const int grid = 2 * (units < pairs ? units : pairs);
  CUtensorMap tp = ta;
  if (s.splits > 1 && !make_out_map(&tp, part, TN, (long long)(units - s.full) * kTile, TN, true)) return ULY_ERR_CUDA;
  kernel<<<grid, kThreads, Layout<TN>::kBytes, stream>>>(ta, tb, tp, s, ep);
  note_launches(1);
  return last_launch_status();
}
template <class Epi, bool A_MN, bool B_MN>
uly_status launch(const CUtensorMap &ta, const CUtensorMap &tb, const Shape &s, const Cut &cut,
                  const typename Epi::Params &ep, float *part, cudaStream_t stream) {
  return cut.tn == kTile ? launch_tn<Epi, kTile, A_MN, B_MN>(ta, tb, s, ep, part, stream)
                         : launch_tn<Epi, kNarrow, A_MN, B_MN>(ta, tb, s, ep, part, stream);
}

// ---------------------------------------------------- vectors of 8 columns
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
// Of memory that the kernel does not write (the read-only path must not see it change).
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
  unpack8(__ldg(reinterpret_cast<const uint4 *>(p)), x);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum of the cut tiles' partials, in a fixed order, and Epi::join8(params, row,
// col, z, up) of eight columns (up: those half a tile further on, in a tile whose
// B holds two rows for each column).  2^lanes_log2 lanes share the parts of eight
// columns: one thread for 74 parts waits for memory some 15 times (1 row of 136 columns over
// 105315: 39 us with the product, 27 this way).
template <class Epi, int TN>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ typename Epi::Params p,
                                                   const __grid_constant__ Shape s, const float *__restrict__ part,
                                                   long long M, int N, int lanes_log2) {
  constexpr int cols = Epi::kGated ? TN / 2 : TN, vecs = cols / 8;
  const int tiles = s.m_tiles * s.n_tiles - s.full, lanes = 1 << lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int rows = (int)min((long long)kTile, M);   // a single row of tiles may be short
  const long long all = (long long)tiles * rows * vecs;
  // whole warps go round together
  for (long long i0 = ((long long)blockIdx.x * 256 + (threadIdx.x & ~31)) >> lanes_log2; i0 < all;
       i0 += ((long long)gridDim.x * 256) >> lanes_log2) {
    const long long i = i0 + ((threadIdx.x & 31) >> lanes_log2);
    const int c = (int)(i % vecs) * 8, r = (int)(i / vecs % rows), t = (int)(i / ((long long)vecs * rows));
    int mt, nt;
    place_of(s, s.full + min(t, tiles - 1), mt, nt);
    const long long row = (long long)mt * kTile + r;
    const int col = nt * cols + c;
    const bool ok = i < all && row < M && col < N;
    float z[8] = {}, up[8] = {};
    if (ok) {
      const float *src = part + (((long long)t * s.splits + lane) * kTile + r) * TN + c;
#pragma unroll 4
      for (int k = lane; k < s.splits; k += lanes, src += (long long)lanes * kTile * TN) {
        float v[8];
        load8(src, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
        if (Epi::kGated) {
          load8(src + TN / 2, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) up[e] += v[e];
        }
      }
    }
    for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] += __shfl_xor_sync(0xffffffffu, z[e], off);
        if (Epi::kGated) up[e] += __shfl_xor_sync(0xffffffffu, up[e], off);
      }
    if (ok && lane == 0) Epi::join8(p, row, col, z, up);
  }
}
template <class Epi>
uly_status launch_join(const typename Epi::Params &p, const Shape &s, const Cut &cut, const float *part, long long M,
                       int N, cudaStream_t stream) {
  if (s.splits == 1) return ULY_OK;
  const int lanes_log2 = s.splits > 32 ? 4 : s.splits > 16 ? 3 : s.splits > 8 ? 2 : 0;
  const long long vecs = (long long)(s.m_tiles * s.n_tiles - s.full) * (M < kTile ? M : kTile) *
                         (cut.tn / (Epi::kGated ? 2 : 1)) / 8;
  const long long want = ((vecs << lanes_log2) + 255) / 256, most = (long long)device_sm_count() * 8;
  auto kernel = cut.tn == kTile ? join_kernel<Epi, kTile> : join_kernel<Epi, kNarrow>;
  kernel<<<(unsigned)(want < most ? want : most), 256, 0, stream>>>(p, s, part, M, N, lanes_log2);
  note_launches(1);
  return last_launch_status();
}

// --------------------------------------------------------- plain epilogue
// out = A B^T / max(*over, 1) + add, in bf16 or fp32; N is a multiple of 8.
struct PlainParams {
  CUtensorMap out_map;      // of out (launch_plain fills it in)
  void *out;
  const float *add;         // nullable fp32 [M][N] (may be `out` itself, fp32)
  const long long *over;    // nullable: 1
  long long M;
  int N, out_f32;
};
__device__ __forceinline__ float one_over(const long long *n) {
  return n ? 1.f / (float)max(__ldg(n), 1ll) : 1.f;
}
struct EpiPlain {
  using Params = PlainParams;
  static constexpr bool kGated = false;
  template <int TN>
  static __device__ __forceinline__ Nothing before(const Params &, const Unit &, int, int, int) { return {}; }
  static __device__ __forceinline__ void add8(const Params &p, long long row, int col, float (&z)[8]) {
    float a[8];
    load8(p.add + row * p.N + col, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += a[e];
  }
  static __device__ __forceinline__ void join8(const Params &p, long long row, int col, float (&z)[8],
                                               const float (&)[8]) {
    if (p.over) {
      const float f = one_over(p.over);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] *= f;
    }
    if (p.add) add8(p, row, col, z);
    if (p.out_f32) store8(static_cast<float *>(p.out) + row * p.N + col, z);
    else store8(static_cast<__nv_bfloat16 *>(p.out) + row * p.N + col, z);
  }
  template <int TN>
  static __device__ __forceinline__ void tile(const Params &p, const Unit &w, uint32_t acc, int row, int half,
                                              Nothing &, OutRing &out) {
    const int row0 = row - out.lane;
    const float f = one_over(p.over);
#pragma unroll 1
    for (int c = 0; c < TN / 2; c += 64) {
      const int col0 = w.nt * TN + half * TN / 2 + c;
      uint32_t a[64], v[16];
      tmem_ld64(acc + half * TN / 2 + c, a);
      if (col0 >= p.N || row0 >= p.M) continue;   // the whole warp
      if (p.over)
#pragma unroll
        for (int e = 0; e < 64; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
      if (p.add && row < p.M) {
#pragma unroll
        for (int g = 0; g < 8; ++g)
          if (col0 + 8 * g < p.N) {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = __uint_as_float(a[8 * g + e]);
            add8(p, row, col0 + 8 * g, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[8 * g + e] = __float_as_uint(z[e]);
          }
      }
      __syncwarp();
      const CUtensorMap *map = &p.out_map;
      if (p.out_f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = col0 + 32 * h;
          if (c0 >= p.N) break;
          out.begin();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = a[32 * h + 16 * i + e];
            out.write(i, v);
          }
          out.end(map, c0, row0);
        }
      } else {
        out.begin();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = pack_bf16x2(__uint_as_float(a[32 * i + 2 * e]), __uint_as_float(a[32 * i + 2 * e + 1]));
          out.write(i, v);
        }
        out.end(map, col0, row0);
      }
    }
  }
};

inline Cut plain_cut(long long M, long long N, long long K, size_t budget = SIZE_MAX) {
  return choose_cut(tiles_of(M), tiles_of(N), tiles_of(N, kNarrow), (K + kBK - 1) / kBK, budget);
}
// out[M][N] (+)= A B^T with a plain epilogue, B MN-major; `part` has room for part_bytes.
template <bool A_MN>
uly_status launch_plain(const CUtensorMap &ta, const CUtensorMap &tb, PlainParams p, long long K, float *part,
                        size_t part_bytes, int kernel_id, cudaStream_t stream) {
  if (!make_out_map(&p.out_map, p.out, p.N, p.M, p.N, p.out_f32 != 0)) return ULY_ERR_CUDA;
  const Cut cut = plain_cut(p.M, p.N, K, part_bytes);
  const Shape s = make_shape(p.M, p.N, K, 1, cut);
  prof::Scope scope(kernel_id, stream);
  const uly_status st = launch<EpiPlain, A_MN, true>(ta, tb, s, cut, p, part, stream);
  return st != ULY_OK ? st : launch_join<EpiPlain>(p, s, cut, part, p.M, p.N, stream);
}

}  // namespace gemm
}  // namespace uly
