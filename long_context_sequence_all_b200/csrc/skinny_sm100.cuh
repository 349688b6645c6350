// The products of gemm_sm100.cuh for few tokens (up to 128): bound by the
// weight matrix's bytes, so what counts is that every SM streams its share of
// them from the first microsecond to the last.
//
// The roles are swapped: 128 rows of the weight matrix are the M side of the
// tensor-core product (with N = the tokens, 16 to 128), so a k-step of 64 costs
// 16 KB of weights and little else.  A tile's k-steps are shared by a cluster of
// up to sixteen CTAs, which meet in distributed shared memory: each adds one slice
// of the tile's rows over the cluster in a fixed order and runs the epilogue on
// it.  No partial leaves the chip, no second launch, no counters.  Several CTAs
// share an SM (one loads while another finishes), so no CTA is persistent.
//
// (8 tokens' worth of the pair product's 256-row tiles would leave 97 % of its
// shared memory to zeros, and its cut along K needs a second kernel: one token
// through 2560 -> 2 x 10240 took 38 us that way, 20 us this way; from 200 tokens
// on the pair product is the faster one, 45 against 93 us.)
#pragma once

#include "gemm_sm100.cuh"

namespace uly {
namespace skinny {

using namespace gemm;

constexpr int kRows = 128;               // weight rows of a tile
constexpr int kSkinnyThreads = 128;
constexpr int kMaxTokens = 128;
constexpr int kCluster = 8, kMaxCluster = 16;   // CTAs of a tile; the second for long sums of few tokens
constexpr uint32_t kWBytes = kRows * kBK * 2;   // 16 KB

template <int NT>
struct Shared {   // bytes of one CTA
  static constexpr int kStages = NT == 16 ? 4 : 3;
  static constexpr int kPerSm = NT == 128 ? 2 : 3;   // CTAs an SM has room for
  static constexpr uint32_t kStage = kWBytes + NT * kBK * 2;
  static constexpr uint32_t kOffBar = kStages * kStage;
  static constexpr uint32_t kBytes = kOffBar + 128 + 1024;
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static_assert(NT * kRows * 4 <= (int)kOffBar, "the accumulators are staged over the ring");
};

struct SkinnyShape {
  int ranks, k_steps;
  int w_step, w_half;   // weight rows of tile i: 64 from i * w_step and 64 from i * w_step + w_half
  int *err;
  long long wait_limit;
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// A tile's sums, when every CTA of the cluster has staged its own: element
// (row, token) is the sum over the cluster, in rank order.
template <int MAX>
struct Tile {
  uint32_t part[MAX];   // cluster addresses of [token][row] fp32
  int ranks;
  // rows [row, row + 4), row a multiple of 4
  __device__ __forceinline__ void sum4(int row, int token, float (&v)[4]) const {
    const uint32_t at = (token * kRows + row) * 4;
    float4 a = ld_cluster4(part[0] + at);
#pragma unroll
    for (int r = 1; r < MAX; ++r)
      if (r < ranks) {
        const float4 b = ld_cluster4(part[r] + at);
        a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
      }
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
};

__device__ __forceinline__ void unpack4(const uint2 &u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {   // not written by the kernel
  unpack4(__ldg(reinterpret_cast<const uint2 *>(p)), x);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// This thread's share of a CTA's slice of `cols` output columns of a tile:
// f(first column of four, in the tile; token).  From thread `first` on.
template <class F>
__device__ __forceinline__ void for_slice(int cols, int rank, int ranks, int T, F f, int first = 0) {
  const int quads = cols / 4 / ranks, shift = 31 - __clz(quads);   // powers of two
#pragma unroll 2
  for (int i = threadIdx.x - first; i < quads * T; i += kSkinnyThreads - first)
    f((rank * quads + (i & (quads - 1))) * 4, i >> shift);
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The `ranks` CTAs of a tile are a cluster.
// Epi::Params,
//   Epi::prefetch(params, index, rank, ranks): warps 2 and 3, while the product
//   runs: what finish() reads of memory may be sent for to L2, and
//   Epi::finish(params, tile, index, rank, ranks): all threads of the CTA, its
//   slice of tile `index`.
template <class Epi, int NT, bool W_MN, int MAX>
__global__ void __launch_bounds__(kSkinnyThreads)
    skinny_sm100_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const SkinnyShape sh, const __grid_constant__ typename Epi::Params ep) {
  using S = Shared<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
  enum { B_FULL = 0, B_EMPTY = S::kStages, B_DONE = 2 * S::kStages, B_N = B_DONE + 1 };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffBar + 8 * B_N);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffBar + 8 * B_N + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = sh.ranks, index = blockIdx.x / ranks, rank = blockIdx.x - index * ranks;
  const int k0 = (int)((long long)sh.k_steps * rank / ranks), k1 = (int)((long long)sh.k_steps * (rank + 1) / ranks);

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_N; ++i) mbar_init(bar(i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), S::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    const int w0 = index * sh.w_step;
    int stage = 0;
    uint32_t phase = 1;
    for (int k = k0; k < k1; ++k) {
      if (!mbar_wait(bar(B_EMPTY + stage), phase, abort_flag, sh.err, sh.wait_limit)) break;
      const uint32_t sW = sb + stage * S::kStage, sX = sW + kWBytes;
      mbar_arrive_expect_tx(bar(B_FULL + stage), S::kStage);
      for (int h = 0; h < 2; ++h) {
        if (W_MN) tma_load_2d(sW + h * 8192, &tmW, bar(B_FULL + stage), w0 + h * sh.w_half, k * kBK);
        else tma_load_2d(sW + h * 8192, &tmW, bar(B_FULL + stage), k * kBK, w0 + h * sh.w_half);
      }
      tma_load_2d(sX, &tmX, bar(B_FULL + stage), k * kBK, 0);
      if (++stage == S::kStages) { stage = 0; phase ^= 1; }
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(kRows, NT, W_MN, false);
    int stage = 0;
    uint32_t phase = 0;
    for (int k = k0; k < k1; ++k) {
      if (!mbar_wait(bar(B_FULL + stage), phase, abort_flag, sh.err, sh.wait_limit)) break;
      tc_fence_after();
      const uint32_t sW = sb + stage * S::kStage, sX = sW + kWBytes;
      const uint64_t dw = W_MN ? sdesc_sw128(sW, 8192, 1024) : sdesc_sw128(sW, 16, 1024);
      const uint64_t dx = sdesc_sw128(sX, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < kBK / 16; ++kk)
        mma_bf16_ss(tmem, sdesc_add(dw, kk * (W_MN ? 2048 : 32)), sdesc_add(dx, kk * 32), idesc,
                    (k > k0 || kk > 0) ? 1u : 0u);
      tc_commit(bar(B_EMPTY + stage));
      if (++stage == S::kStages) { stage = 0; phase ^= 1; }
    }
    tc_commit(bar(B_DONE));
  } else if (warp >= 2) {
    Epi::prefetch(ep, index, rank, ranks);
  }
  __syncwarp();
  // Every MMA has completed (so every copy was consumed): the ring's memory is
  // free for the accumulators, [token][row].
  mbar_wait(bar(B_DONE), 0, abort_flag, sh.err, sh.wait_limit);
  __syncthreads();
  if (*abort_flag) {   // copies and MMAs may be in flight: let them finish
    const long long t0 = clock64();
    while (clock64() - t0 < kLandCycles) __nanosleep(1000);
  }
  tc_fence_after();
  {
    float *out = reinterpret_cast<float *>(smem);
    const int row = warp * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < NT; c += 16) {
      uint32_t a[16];
      tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c, a);
#pragma unroll
      for (int e = 0; e < 16; ++e) out[(c + e) * kRows + row] = __uint_as_float(a[e]);
    }
  }
  tc_fence_before();
  if (ranks > 1) cluster_sync();
  else __syncthreads();
  Tile<MAX> tile;
  tile.ranks = ranks;
#pragma unroll
  for (int r = 0; r < MAX; ++r) tile.part[r] = r < ranks ? map_cta(sb, r) : 0;
  Epi::finish(ep, tile, index, rank, ranks);
  if (ranks > 1) cluster_sync();   // the peers have read this CTA's sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// ------------------------------------------------------------------- host

inline int tokens_padded(long long T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

// CTAs that share a tile's k-steps: as many as the SMs have room for at once, of at
// least four k-steps each and up to eight; sixteen of at least eight for up to 32
// tokens (24 x 10240 -> 2560: 18.2 us with eight, 16.6 so; 64 x 8192 -> 2048, whose
// sums over the cluster are longer: 17.0 and 19.4).
inline int cluster_size(long long T, long long tiles, long long k_steps) {
  const long long room = (long long)device_sm_count() * (tokens_padded(T) == 128 ? Shared<128>::kPerSm : Shared<64>::kPerSm);
  int s = 1;
  while (s < kCluster && tiles * s * 2 <= room && k_steps >= 8 * s) s *= 2;
  return s == kCluster && T <= 32 && tiles * kMaxCluster <= room && k_steps >= 8 * kMaxCluster ? kMaxCluster : s;
}
// Opt `kernel` into clusters of more than eight CTAs, once per device.
template <typename Kernel>
inline bool wide_optin(Kernel kernel, std::atomic<uint64_t> &done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const uint64_t bit = uint64_t(1) << dev;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

// About how long the product takes: a CTA 0.35 us a k-step (what its ring holds is
// always under way), all of them together move 5.2 TB/s.
inline double micros(long long T, long long N, long long steps, long long ranks) {
  const double latency = (double)((steps + ranks - 1) / ranks) * 0.35, bytes = (double)N * (double)steps * kBK * 2.0 / 5.2e6;
  return 4.0 + 0.05 * (double)T + (latency > bytes ? latency : bytes);
}
// Whether this kernel or the pair product is the faster way to out[T][N] over K:
// at most sixteen CTAs share a tile's k-steps here; the pair product cuts a tile in
// as many parts as the GPU has pairs.
// 16 tokens over 17192, 296 wide: 15 us here, 18 there; 1 over 105315, 136 wide:
// 62 and 23; 100 over 151936, 2560 wide: 156 and 143.
inline bool faster(long long T, long long N, long long K, size_t part_bytes = SIZE_MAX) {
  if (T > kMaxTokens) return false;
  const long long steps = (K + kBK - 1) / kBK, ranks = cluster_size(T, (N + kRows - 1) / kRows, steps);
  return micros(T, N, steps, ranks) <= plain_cut(T, N, K, part_bytes).us + 7.0;
}

template <class Epi, int NT, bool W_MN, int MAX = kCluster>
uly_status launch_nt(const CUtensorMap &tw, const CUtensorMap &tx, const SkinnyShape &sh, const typename Epi::Params &ep,
                     int tiles, int ranks, cudaStream_t stream) {
  static std::atomic<uint64_t> optin{0}, wide{0};
  auto kernel = skinny_sm100_kernel<Epi, NT, W_MN, MAX>;
  if (!smem_optin(kernel, (int)Shared<NT>::kBytes, optin)) return ULY_ERR_CUDA;
  if (MAX > kCluster && !wide_optin(kernel, wide)) return ULY_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles * ranks);
  cfg.blockDim = dim3(kSkinnyThreads);
  cfg.dynamicSmemBytes = Shared<NT>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, tw, tx, sh, ep) != cudaSuccess) {
    cudaGetLastError();
    return ULY_ERR_CUDA;
  }
  note_launches(1);
  return last_launch_status();
}

// C[tokens][rows of W] of x [tokens][K] (K contiguous) and the weight matrix:
// W_MN false: w [rows][K]; true: w [K][rows].  `tiles` tiles of rows as `sh`
// says; the caller's epilogue stores.
template <class Epi, bool W_MN>
uly_status launch(const void *w, long long w_inner, long long w_rows, const void *x, long long x_stride, long long T,
                  long long K, int tiles, int ranks, int w_step, int w_half, const typename Epi::Params &ep,
                  cudaStream_t stream) {
  const int nt = tokens_padded(T);
  CUtensorMap tw, tx;
  if (!make_map(&tw, w, w_inner, w_rows, w_inner, 64) || !make_map(&tx, x, K, T, x_stride, nt)) return ULY_ERR_CUDA;
  SkinnyShape sh = {};
  sh.ranks = ranks;
  sh.k_steps = (int)((K + kBK - 1) / kBK);
  sh.w_step = w_step;
  sh.w_half = w_half;
  sh.err = error_word();
  sh.wait_limit = wait_limit_cycles();
  if (ranks > kCluster)   // an instance of its own: eight more parts cost the others a microsecond
    return nt == 16 ? launch_nt<Epi, 16, W_MN, kMaxCluster>(tw, tx, sh, ep, tiles, ranks, stream)
                    : launch_nt<Epi, 32, W_MN, kMaxCluster>(tw, tx, sh, ep, tiles, ranks, stream);
  switch (nt) {
    case 16: return launch_nt<Epi, 16, W_MN>(tw, tx, sh, ep, tiles, ranks, stream);
    case 32: return launch_nt<Epi, 32, W_MN>(tw, tx, sh, ep, tiles, ranks, stream);
    case 64: return launch_nt<Epi, 64, W_MN>(tw, tx, sh, ep, tiles, ranks, stream);
    default: return launch_nt<Epi, 128, W_MN>(tw, tx, sh, ep, tiles, ranks, stream);
  }
}

// out[tokens][N] in bf16, the sums over max(*over, 1) (over null: 1).
struct SkinnyPlain {
  struct Params {
    __nv_bfloat16 *out;
    const long long *over;
    int T, N;
  };
  static __device__ __forceinline__ void prefetch(const Params &, int, int, int) {}
  template <class T>
  static __device__ __forceinline__ void finish(const Params &p, const T &tile, int index, int rank, int ranks) {
    const float f = gemm::one_over(p.over);
    for_slice(kRows, rank, ranks, p.T, [&](int row, int t) {
      float v[4];
      tile.sum4(row, t, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      const int col = index * kRows + row;   // N is a multiple of 8
      if (col < p.N) store4(p.out + (long long)t * p.N + col, v);
    });
  }
};

// out[T][N] = x [T][K] w / max(*over, 1), w [K][N].
inline uly_status launch_plain_mn(const void *x, long long x_stride, const void *w, void *out, const long long *over,
                                  long long T, int N, long long K, int kernel_id, cudaStream_t stream) {
  prof::Scope scope(kernel_id, stream);
  const int tiles = (N + kRows - 1) / kRows;
  const SkinnyPlain::Params p = {static_cast<__nv_bfloat16 *>(out), over, (int)T, N};
  return launch<SkinnyPlain, true>(w, N, K, x, x_stride, T, K, tiles, cluster_size(T, tiles, (K + kBK - 1) / kBK), kRows,
                                   64, p, stream);
}

}  // namespace skinny
}  // namespace uly
