// The token-weighted cross-entropy taken straight from the hidden states,
// z = x W^T over the whole vocabulary, without a logits tensor:
//
//   l_t = logsumexp_v(z_tv) - z_t[y_t],  S_r, C_r, L as ulysses_loss_aggregate
//   dx = dz W / C,  dW = dz^T x / C,  dz_tv = softmax(z_t)_v - [v == y_t]
//
// Forward: the product's epilogue keeps, for each 128 columns of a row, their
// maximum and the sum of exp(z - maximum) (fp32); a second kernel folds a
// row's pairs into its logsumexp.  No logit leaves the tensor memory.
//
// Gradient, in pieces of tokens: the logits are formed once.  The epilogue
// stores p = 2^15 exp(z - maximum) in fp16, the maximum that of the row's 128
// columns, so every value is at most 2^15 and keeps 11 significant bits down
// to e^-20 of that maximum (2^-40 of it absolute below).  When the row's pairs
// have given its logsumexp, one pass brings p to
//   dz_tv = softmax_tv - [v == y_t]   in bf16, in place
// (the label's element as expm1(z_y - lse), exact for confident tokens too),
// and dz W and dz^T x are plain products, divided by C in fp32 as they leave
// the tensor memory.  So dz is rounded to bf16 once, 2^-8 relative at most,
// after 2^-11 of the stored exponential.  Where the labels' softmax is small
// their elements, which then are nearly all of a gradient, are close to -1 and
// lose nothing; divided by C first they would all be off by the same part.
//
// Three products of 2 T D V operations, the fewest that do not keep the
// logits in a wider type; bound by the tensor cores, with few tokens by W's
// bytes.  The pass over p moves 4 bytes a logit: about a twentieth of the time
// at D = 2560.  Forming the logits a second time instead would cost a third.
#include <cuda_fp16.h>

#include "skinny_sm100.cuh"
#include "tokenwise.cuh"

namespace uly {

using namespace gemm;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSlot = kHalf;        // columns behind one (maximum, sum) pair
constexpr float kScale = 32768.f;   // of a stored exponential
constexpr long long kPieceBytes = 4ll << 30;    // p of one piece of tokens
constexpr long long kPairBytes = 128ll << 20;   // pairs of one forward piece

struct LossParams {
  CUtensorMap p_map;       // STORE_P: fp16 [rows][ldp]
  const int32_t *labels;   // of the piece's rows
  float2 *pairs;           // [slots][rows_pad]: (maximum, sum of exp(z - maximum)); (-inf, 0) where every z is -inf
  float *target;           // [rows]: z[label]
  long long rows_pad;
  int rows, vocab, ignore_index;
};

template <bool STORE_P>
struct EpiLoss {
  using Params = LossParams;
  template <int TN>
  static __device__ __forceinline__ Nothing before(const Params &, const Unit &, int, int, int) { return {}; }
  template <int TN>
  static __device__ __forceinline__ void tile(const Params &p, const Unit &w, uint32_t acc, int row, int half,
                                              Nothing &, OutRing &out) {
    static_assert(TN / 2 == kSlot, "a warpgroup's columns are one slot");
    const int col0 = w.nt * kTile + half * kSlot;
    const int ncol = min(kSlot, p.vocab - col0);   // columns of the vocabulary here; may be <= 0
    const bool ok = row < p.rows;
    const int row0 = row - out.lane;
    if (ncol <= 0 || row0 >= p.rows) return;       // the whole warp
    const int y = ok ? __ldg(p.labels + row) : p.ignore_index;
    const bool counted = y != p.ignore_index && y >= 0 && y < p.vocab;
    // the row's 128 logits stay in registers from here on
    uint32_t a[kSlot];
    tmem_ld128(acc + half * kSlot, a);
    if (ncol < kSlot) {
#pragma unroll
      for (int e = 0; e < kSlot; ++e)
        if (e >= ncol) a[e] = __float_as_uint(-INFINITY);
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < kSlot; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(a[e]));
    const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    const float ref = m == -INFINITY ? 0.f : m;   // every logit -inf: each term is 0
    if (counted && y >= col0 && y < col0 + kSlot) {
      float t = 0.f;
#pragma unroll
      for (int e = 0; e < kSlot; ++e) t = y == col0 + e ? __uint_as_float(a[e]) : t;
      p.target[row] = t;
    }
    __syncwarp();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kSlot; c += 64) {
      if (c >= ncol) break;
      if (STORE_P) out.begin();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          // the difference first: exact at any size of the logits
          const float q0 = ex2_approx((__uint_as_float(a[c + 32 * h + e]) - ref) * kLog2e);
          const float q1 = ex2_approx((__uint_as_float(a[c + 32 * h + e + 1]) - ref) * kLog2e);
          s[e & 2] += q0;
          s[(e & 2) + 1] += q1;
          if (STORE_P) {
            const __half2 x = __floats2half2_rn(q0 * kScale, q1 * kScale);
            v[e / 2] = *reinterpret_cast<const uint32_t *>(&x);
          }
        }
        if (STORE_P) out.write(h, v);
      }
      if (STORE_P)
        out.end(&p.p_map, col0 + c, row0);
    }
    if (ok) p.pairs[(long long)(w.nt * 2 + half) * p.rows_pad + row] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
  }
};

__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2) {
  // (m, s) stands for s exp(m); an empty pair (s = 0) changes nothing
  if (s2 == 0.f) return;
  if (s == 0.f) { m = m2; s = s2; return; }
  const float mm = fmaxf(m, m2);
  s = s * exp2f((m - mm) * kLog2e) + s2 * exp2f((m2 - mm) * kLog2e);
  m = mm;
}

// Few tokens: the tile's 128 columns of the vocabulary are one slot; a warp a
// token, four columns a lane.
struct SkinnyLossParams {
  LossParams l;
  __half *p;        // null: no exponentials are kept
  long long ldp;
};
struct SkinnyLoss {
  using Params = SkinnyLossParams;
  static __device__ __forceinline__ void prefetch(const Params &, int, int, int) {}
  template <class T>
  static __device__ __forceinline__ void finish(const Params &q, const T &tile, int index, int rank, int ranks) {
    const LossParams &p = q.l;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = index * kSlot + 4 * lane, ncol = p.vocab - index * kSlot;
    // four tokens of a warp at a time: their shuffles overlap; the tile's CTAs share
    // the tokens, a row's slot is one warp's
    for (int t0 = (rank * (skinny::kSkinnyThreads / 32) + warp) * 4; t0 < p.rows;
         t0 += ranks * (skinny::kSkinnyThreads / 8)) {
      float z[4][4], m[4], s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        tile.sum4(4 * lane, t0 + k, z[k]);   // padded tokens are in the tile
        m[k] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * lane + e < ncol) m[k] = fmaxf(m[k], z[k][e]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], off));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = t0 + k;
        const bool ok = t < p.rows;
        const int y = ok ? __ldg(p.labels + t) : p.ignore_index;
        const bool counted = y != p.ignore_index && y >= 0 && y < p.vocab;
        const float ref = m[k] == -INFINITY ? 0.f : m[k];   // every logit -inf: each term is 0
        s[k] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (counted && y == col + e) p.target[t] = z[k][e];
          z[k][e] = 4 * lane + e < ncol ? ex2_approx((z[k][e] - ref) * kLog2e) : 0.f;
          s[k] += z[k][e];
        }
        if (q.p && ok && 4 * lane < ncol) {
          const __half2 a = __floats2half2_rn(z[k][0] * kScale, z[k][1] * kScale);
          const __half2 b = __floats2half2_rn(z[k][2] * kScale, z[k][3] * kScale);
          *reinterpret_cast<uint2 *>(q.p + t * q.ldp + col) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], off);
      if (lane < 4 && t0 + lane < p.rows) {
        const float mk = lane == 0 ? m[0] : lane == 1 ? m[1] : lane == 2 ? m[2] : m[3];
        const float sk = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
        p.pairs[(long long)index * p.rows_pad + t0 + lane] = make_float2(mk, sk);
      }
    }
  }
};

// The shards' losses and valid labels and the fold over the shards by one CTA, for
// up to 8 shards of a modest batch: 32 parts, as many a shard as fit, a warp each
// (fewer warps take several), joined in their order.
constexpr int kCloseShards = 8;
constexpr long long kCloseTokens = 16384;
struct CloseParams {
  const float *row_loss;
  const int32_t *labels;
  long long per;              // tokens of a shard
  int P, vocab, ignore_index;
  float *shard_sum, *loss;
  int64_t *shard_count;
  long long *count;           // nullable
};
__device__ __forceinline__ void close_shards(const CloseParams &p) {
  __shared__ double sh_s[32];
  __shared__ int sh_c[32];
  const int lane = threadIdx.x & 31, each = 32 / p.P;
  for (int v = threadIdx.x >> 5; v < 32; v += blockDim.x / 32) {
    const int r = v / each;
    double a = 0.0;
    int c = 0;
    if (r < p.P) {
      const long long t0 = (long long)r * p.per;
#pragma unroll 4
      for (long long i = (v - r * each) * 32 + lane; i < p.per; i += 32 * each) {
        const int y = __ldg(p.labels + t0 + i);
        if (y != p.ignore_index && y >= 0 && y < p.vocab) {
          a += (double)p.row_loss[t0 + i];
          ++c;
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      a += __shfl_down_sync(0xffffffffu, a, off);
      c += __shfl_down_sync(0xffffffffu, c, off);
    }
    if (lane == 0) { sh_s[v] = a; sh_c[v] = c; }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    long long n = 0;
    for (int k = 0; k < p.P; ++k) {
      double s = 0.0;
      long long m = 0;
      for (int w = 0; w < each; ++w) { s += sh_s[k * each + w]; m += sh_c[k * each + w]; }
      p.shard_sum[k] = (float)s;
      p.shard_count[k] = m;
      all += s;
      n += m;
    }
    *p.loss = (float)(all / (double)n);   // 0/0 -> NaN when no token is valid
    if (p.count) *p.count = n;
  }
}
__global__ void __launch_bounds__(1024) loss_close_kernel(const __grid_constant__ CloseParams p) { close_shards(p); }

// Four rows a CTA: their pairs (one 32-byte sector for a slot of all four) are
// folded in a fixed order into lse and the rows' losses.  GRAD: and each slot's
// factor exp(maximum - lse) of its stored exponentials, [row][slot]: at most about 1,
// as a slot with nothing in it has -inf for its maximum and 0 for its factor.
struct RowsParams {
  const float2 *pairs;
  const float *target;
  const int32_t *labels;
  float *row_loss, *row_lse;  // of the piece's rows
  float *factor;              // [rows][slots]
  long long rows_pad;
  int rows, slots, vocab, ignore_index;
  int *err;
  CloseParams close;
};
constexpr int kRowsCta = 4, kRowThreads = 512;

template <bool GRAD>
__device__ __forceinline__ void rows_of_cta(const RowsParams &p, int row0) {
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float sh_m[kWarps][kRowsCta], sh_s[kWarps][kRowsCta];
  __shared__ float sh_lse[kRowsCta];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nrows = min(kRowsCta, p.rows - row0);
  float m[kRowsCta], s[kRowsCta];
#pragma unroll
  for (int r = 0; r < kRowsCta; ++r) { m[r] = 0.f; s[r] = 0.f; }
  for (int k = threadIdx.x; k < p.slots; k += kRowThreads) {
    // rows past the last one are in the padding of the array: read, not used
    const float4 *v = reinterpret_cast<const float4 *>(p.pairs + (long long)k * p.rows_pad + row0);
    const float4 a = __ldg(v), b = __ldg(v + 1);
    merge(m[0], s[0], a.x, a.y);
    merge(m[1], s[1], a.z, a.w);
    merge(m[2], s[2], b.x, b.y);
    merge(m[3], s[3], b.z, b.w);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int r = 0; r < kRowsCta; ++r) {
      const float m2 = __shfl_down_sync(0xffffffffu, m[r], off), s2 = __shfl_down_sync(0xffffffffu, s[r], off);
      merge(m[r], s[r], m2, s2);
    }
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < kRowsCta; ++r) { sh_m[warp][r] = m[r]; sh_s[warp][r] = s[r]; }
  __syncthreads();
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x;
    float mm = sh_m[0][r], ss = sh_s[0][r];
    for (int k = 1; k < kWarps; ++k) merge(mm, ss, sh_m[k][r], sh_s[k][r]);
    const float lse = mm + logf(ss);
    const int y = __ldg(p.labels + row0 + r);
    const bool counted = y != p.ignore_index && y >= 0 && y < p.vocab;
    if (y != p.ignore_index && !counted) raise_error(p.err, ULY_ERR_LABEL);
    p.row_loss[row0 + r] = counted ? lse - p.target[row0 + r] : 0.f;
    if (GRAD) p.row_lse[row0 + r] = sh_lse[r] = lse;
  }
  if (!GRAD) return;
  __syncthreads();
  for (int k = threadIdx.x; k < p.slots; k += kRowThreads) {
    const float2 *v = p.pairs + (long long)k * p.rows_pad + row0;
    for (int r = 0; r < nrows; ++r)
      p.factor[(long long)(row0 + r) * p.slots + k] = exp2f((v[r].x - sh_lse[r]) * kLog2e) / kScale;
  }
}

template <bool GRAD>
__global__ void __launch_bounds__(kRowThreads) loss_rows_kernel(const __grid_constant__ RowsParams p) {
  rows_of_cta<GRAD>(p, blockIdx.x * kRowsCta);
}
// Few rows, all there are: the CTAs are one cluster, and its first also closes the
// losses (12 tokens of 2536 over 1103: 26.7 -> 24.6 us; a launch of more CTAs costs
// what the second one did).
constexpr int kOneCluster = 4, kOneRows = kOneCluster * kRowsCta;
__global__ void __launch_bounds__(kRowThreads) loss_rows_close_kernel(const __grid_constant__ RowsParams p) {
  if ((int)blockIdx.x * kRowsCta < p.rows) rows_of_cta<false>(p, blockIdx.x * kRowsCta);
  cluster_sync();   // the rows' losses are there for the whole cluster
  if (blockIdx.x == 0) close_shards(p.close);
}

// p becomes dz: kGradCols columns of a CTA's rows.  Those of the first columns also
// copy x, with zeros in the rows that do not count (a row of a padded batch
// may hold anything, and 0 times NaN is not 0).  Where the piece is all there is, a
// row of CTAs more closes the losses, which saves two launches (16 tokens of 296
// over 17192: 55 -> 50 us, 40 -> 36 in a graph).
struct GradParams {
  const float *factor, *row_lse, *target;
  const int32_t *labels;
  uint4 *p;                   // [rows][ldp / 8]: fp16 in, bf16 out
  const uint4 *x;
  uint4 *xk;                  // [rows][ldx / 8]
  long long ldp, ldx;
  int slots, vocab, ignore_index, hidden, rows, closing;
  CloseParams close;          // of the last column of CTAs, if `closing`
};
constexpr int kGradPerSm = 4, kGradThreads = 256, kGradVecs = 4, kGradCols = kGradThreads * kGradVecs * 8;

// A CTA goes down the rows of its columns; a row's values are asked for while the
// row before is worked on, its label two rows ahead.
__global__ void __launch_bounds__(kGradThreads) loss_grad_kernel(const __grid_constant__ GradParams p) {
  const int step = gridDim.x - p.closing;
  if (blockIdx.x == step) {
    if (blockIdx.y == 0) close_shards(p.close);
    return;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int vecs = (p.vocab + 7) / 8, i0 = blockIdx.y * (kGradCols / 8) + threadIdx.x;
  auto label = [&](int row) { return row < p.rows ? __ldg(p.labels + row) : p.ignore_index; };
  auto counts = [&](int y) { return y != p.ignore_index && y >= 0 && y < p.vocab; };
  uint4 next[kGradVecs];
  float fnext[kGradVecs];
  auto ask = [&](int row, int y) {
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const int i = i0 + k * kGradThreads;
      const bool ok = counts(y) && i < vecs;
      next[k] = ok ? __ldcs(p.p + row * (p.ldp / 8) + i) : zero;
      fnext[k] = ok ? __ldg(p.factor + (long long)row * p.slots + i / (kSlot / 8)) : 0.f;
    }
  };
  int y = label(blockIdx.x), y1 = label(blockIdx.x + step);
  ask(blockIdx.x, y);
  for (int row = blockIdx.x; row < p.rows; row += step) {
    const bool counted = counts(y);
    uint4 h[kGradVecs];
    float f[kGradVecs];
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) { h[k] = next[k]; f[k] = fnext[k]; }
    const int y2 = label(row + 2 * step);
    ask(row + step, y1);
    uint4 *o = p.p + row * (p.ldp / 8);
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const int i = i0 + k * kGradThreads;
      if (i >= vecs) break;
      const __half2 *hp = reinterpret_cast<const __half2 *>(&h[k]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = __half22float2(hp[e]);
        v[2 * e] = t.x * f[k];
        v[2 * e + 1] = t.y * f[k];
      }
      if (counted && i == y / 8) {
        // z_y <= lse but for rounding: the label's softmax is at most 1 (or NaN, which stays)
        const float d = p.target[row] - p.row_lse[row];
        const float dy = expm1f(d > 0.f ? 0.f : d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e == y % 8) v[e] = dy;
      }
      o[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    if (blockIdx.y == 0) {
      const int xv = p.hidden / 8;
      for (int i = threadIdx.x; i < xv; i += kGradThreads)
        p.xk[row * (p.ldx / 8) + i] = counted ? __ldg(p.x + (long long)row * xv + i) : zero;
    }
    y = y1;
    y1 = y2;
  }
}

// Shard r's losses and valid labels, one CTA a shard, in a fixed order.
__global__ void __launch_bounds__(256) shard_sum_kernel(const float *__restrict__ row_loss,
                                                        const int32_t *__restrict__ labels, long long per, int vocab,
                                                        int ignore_index, double *__restrict__ psum,
                                                        long long *__restrict__ pcnt) {
  __shared__ double sh_s[256];
  __shared__ long long sh_c[256];
  const long long t0 = (long long)blockIdx.x * per;
  double a = 0.0;
  long long c = 0;
  for (long long i = threadIdx.x; i < per; i += blockDim.x) {
    const int y = __ldg(labels + t0 + i);
    if (y != ignore_index && y >= 0 && y < vocab) {
      a += (double)row_loss[t0 + i];
      ++c;
    }
  }
  sh_s[threadIdx.x] = a;
  sh_c[threadIdx.x] = c;
  __syncthreads();
  for (int w = blockDim.x / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) {
      sh_s[threadIdx.x] += sh_s[threadIdx.x + w];
      sh_c[threadIdx.x] += sh_c[threadIdx.x + w];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    psum[blockIdx.x] = sh_s[0];
    pcnt[blockIdx.x] = sh_c[0];
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
long long round_up(long long v, long long m) { return (v + m - 1) / m * m; }

// Tokens of a piece: all of them where `row_bytes` of scratch a token allow.
long long piece_of(long long tokens, long long row_bytes, long long budget) {
  long long t = budget / row_bytes / kTile * kTile;
  if (t < kTile) t = kTile;
  return t < tokens ? t : (tokens > 0 ? tokens : 1);
}

struct Plan {
  long long piece, rows_pad, ldp, ldx;   // ldp, ldx: row strides of p and of the copy of x
  int slots;
  bool dw_acc;   // dW of several pieces is summed in an fp32 array of the workspace
  size_t psum, pcnt, count, row_loss, row_lse, target, pairs, factor, p, xk, part, acc, bytes;   // offsets, total
  size_t part_bytes;
};

Plan make_plan(int P, long long T, int D, int V, bool grad, int dw_dtype, long long piece_tokens) {
  Plan q = {};
  q.slots = (V + kTile - 1) / kTile * 2;
  q.ldp = round_up(V, kRowAlign);
  q.ldx = round_up(D, kRowAlign);
  q.piece = piece_tokens > 0 ? (piece_tokens < T ? piece_tokens : (T > 0 ? T : 1))
            : grad           ? piece_of(T, q.ldp * 2, kPieceBytes)
                             : piece_of(T, (long long)q.slots * 8, kPairBytes);
  q.rows_pad = round_up(q.piece, 32);
  size_t at = 0;
  auto take = [&](size_t n) { const size_t o = at; at += up256(n); return o; };
  q.psum = take((size_t)P * sizeof(double));
  q.pcnt = take((size_t)P * sizeof(long long));
  q.count = take(sizeof(long long));
  q.row_loss = take((size_t)T * sizeof(float));
  q.target = take((size_t)q.piece * sizeof(float));
  q.pairs = take((size_t)q.slots * q.rows_pad * sizeof(float2));
  if (grad) {
    q.dw_acc = q.piece < T && dw_dtype == ULY_BF16;
    q.row_lse = take((size_t)q.piece * sizeof(float));
    q.factor = take((size_t)q.piece * q.slots * sizeof(float));
    q.p = take((size_t)q.piece * q.ldp * 2);
    q.xk = take((size_t)q.piece * q.ldx * 2);
    const size_t a = plain_cut(q.piece, D, V).bytes, b = plain_cut(V, D, q.piece).bytes;
    q.part_bytes = a > b ? a : b;
    q.part = take(q.part_bytes);
    q.acc = take(q.dw_acc ? (size_t)V * D * sizeof(float) : 0);
  }
  q.bytes = at;
  return q;
}

template <typename T>
T *at(void *ws, size_t off) { return reinterpret_cast<T *>(static_cast<char *>(ws) + off); }

// Whole tiles of 256 columns: the epilogue needs the finished sums of its slots.
Cut whole(long long rows, long long V) {
  Cut c;
  c.full = (int)(tiles_of(rows) * tiles_of(V));
  return c;
}

// Whether the weights' side of few rows' logits is the M side: up to 64 rows always,
// bound by w's bytes (64 to 128 rows: 165 against 191 us over 151936 x 2560 for the
// pair product); up to 128 where the vocabulary gives few tiles, whose k-steps only
// that way are shared by several SMs (100 x 2536 over 1103: 33 us
// on the pair product, 23 this way).
bool few_rows(long long rows, long long steps, long long slots) {
  if (rows > skinny::kMaxTokens) return false;
  if (rows <= 64) return true;
  const long long ranks = skinny::cluster_size(rows, slots, steps), pairs = device_sm_count() / 2;
  const long long turns = (tiles_of(rows) * ((slots + 1) / 2) + pairs - 1) / pairs;
  return skinny::micros(rows, slots * kSlot, steps, ranks) < (double)(turns * steps) * 0.3 + 8.0;
}

// The pairs, targets and (grad) exponentials of a piece's rows.
template <bool GRAD>
uly_status logits_pass(const __nv_bfloat16 *x, const void *w, int D, LossParams &p, void *pp, long long ldp,
                       cudaStream_t stream) {
  prof::Scope scope(prof::K_LINEAR_LOSS, stream);
  const int rows = p.rows, V = p.vocab;
  const long long steps = (D + kBK - 1) / kBK, slots = (V + kSlot - 1) / kSlot;
  if (few_rows(rows, steps, slots)) {
    SkinnyLossParams s = {p, GRAD ? static_cast<__half *>(pp) : nullptr, ldp};
    return skinny::launch<SkinnyLoss, false>(w, D, V, x, D, rows, D, (int)slots, skinny::cluster_size(rows, slots, steps),
                                             kSlot, 64, s, stream);
  }
  CUtensorMap tx, tw;
  if (!make_map(&tw, w, D, V, D, kHalf) || !make_map(&tx, x, D, rows, D, kHalf) ||
      (GRAD && !make_out_map(&p.p_map, pp, V, rows, ldp)))
    return ULY_ERR_CUDA;
  return launch_tn<EpiLoss<GRAD>, kTile, false, false>(tx, tw, make_shape(rows, V, D, 1, whole(rows, V)), p, nullptr, stream);
}

RowsParams rows_of(const Plan &q, const LossParams &p, void *ws, long long t0) {
  RowsParams r = {};
  r.pairs = p.pairs; r.target = p.target; r.labels = p.labels;
  r.row_loss = at<float>(ws, q.row_loss) + t0;
  r.rows_pad = q.rows_pad;
  r.rows = p.rows; r.slots = (p.vocab + kSlot - 1) / kSlot; r.vocab = p.vocab; r.ignore_index = p.ignore_index;
  r.err = error_word();
  return r;
}

bool one_close(int P, long long T) { return P <= kCloseShards && T <= kCloseTokens; }

CloseParams close_of(const Plan &q, int P, long long T, int V, const int32_t *labels, int ignore_index,
                     float *shard_sum, int64_t *shard_count, float *loss, void *ws) {
  CloseParams c = {};
  c.row_loss = at<float>(ws, q.row_loss);
  c.labels = labels;
  c.per = T / P;
  c.P = P; c.vocab = V; c.ignore_index = ignore_index;
  c.shard_sum = shard_sum; c.shard_count = shard_count; c.loss = loss;
  return c;
}

uly_status rows_close(const RowsParams &r, cudaStream_t stream) {
  unsigned ctas = 1;
  while (ctas < kOneCluster && (int)ctas * kRowsCta < r.rows) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, loss_rows_close_kernel, r) != cudaSuccess) {
    cudaGetLastError();
    return ULY_ERR_CUDA;
  }
  note_launches(1);
  return last_launch_status();
}

uly_status finish(const Plan &q, const CloseParams &c, long long T, void *ws, cudaStream_t stream) {
  if (one_close(c.P, T)) {
    prof::Scope scope(prof::K_LOSS_FINALIZE, stream);
    loss_close_kernel<<<1, 1024, 0, stream>>>(c);
    note_launches(1);
    return last_launch_status();
  }
  shard_sum_kernel<<<c.P, 256, 0, stream>>>(c.row_loss, c.labels, c.per, c.vocab, c.ignore_index,
                                            at<double>(ws, q.psum), at<long long>(ws, q.pcnt));
  note_launches(1);
  loss_finalize_launch(at<double>(ws, q.psum), at<long long>(ws, q.pcnt), c.P, 1, c.shard_sum, c.shard_count, c.loss,
                       stream);
  return last_launch_status();
}

}  // namespace

size_t linear_loss_workspace_bytes(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab) {
  return make_plan(P, tokens, hidden, vocab, false, ULY_F32, 0).bytes;
}

uly_status linear_loss_launch(int32_t P, int64_t tokens, int32_t D, int32_t V, const void *x, const void *w,
                              const int32_t *labels, int32_t ignore_index, float *shard_sum, int64_t *shard_count,
                              float *loss, void *ws, cudaStream_t stream) {
  const Plan q = make_plan(P, tokens, D, V, false, ULY_F32, 0);
  const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16 *>(x);
  const CloseParams close = close_of(q, P, tokens, V, labels, ignore_index, shard_sum, shard_count, loss, ws);
  for (long long t0 = 0; t0 < tokens; t0 += q.piece) {
    const int rows = (int)(tokens - t0 < q.piece ? tokens - t0 : q.piece);
    LossParams p = {};
    p.labels = labels + t0;
    p.pairs = at<float2>(ws, q.pairs);
    p.target = at<float>(ws, q.target);
    p.rows_pad = q.rows_pad;
    p.rows = rows; p.vocab = V; p.ignore_index = ignore_index;
    const uly_status st = logits_pass<false>(xb + t0 * D, w, D, p, nullptr, 0, stream);
    if (st != ULY_OK) return st;
    RowsParams r = rows_of(q, p, ws, t0);
    prof::Scope scope(prof::K_LINEAR_LOSS_ROWS, stream);
    if (tokens <= kOneRows && q.piece >= tokens && one_close(P, tokens)) {
      r.close = close;
      return rows_close(r, stream);
    }
    loss_rows_kernel<false><<<(rows + kRowsCta - 1) / kRowsCta, kRowThreads, 0, stream>>>(r);
    note_launches(1);
    if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
  }
  return finish(q, close, tokens, ws, stream);
}

size_t linear_loss_bwd_workspace_bytes(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab, int32_t dw_dtype,
                                       int64_t piece_tokens) {
  return make_plan(P, tokens, hidden, vocab, true, dw_dtype, piece_tokens).bytes;
}

uly_status linear_loss_bwd_launch(int32_t P, int64_t tokens, int32_t D, int32_t V, const void *x, const void *w,
                                  const int32_t *labels, int32_t ignore_index, void *dx, void *dw, int32_t dw_dtype,
                                  int64_t piece_tokens, float *shard_sum, int64_t *shard_count, float *loss, void *ws,
                                  cudaStream_t stream) {
  const Plan q = make_plan(P, tokens, D, V, true, dw_dtype, piece_tokens);
  const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16 *>(x);
  __nv_bfloat16 *dxb = static_cast<__nv_bfloat16 *>(dx);
  long long *count = at<long long>(ws, q.count);
  if (tokens == 0)
    if (cudaMemsetAsync(dw, 0, (size_t)V * D * (dw_dtype == ULY_F32 ? 4 : 2), stream) != cudaSuccess)
      return ULY_ERR_CUDA;
  CloseParams close = close_of(q, P, tokens, V, labels, ignore_index, shard_sum, shard_count, loss, ws);
  const bool closed = tokens > 0 && q.piece >= tokens && one_close(P, tokens);   // by the gradient pass
  if (closed) close.count = count;
  else loss_count_launch(labels, tokens, V, ignore_index, count, stream);
  CUtensorMap tw_mn, tz, tz_mn, tk_mn;
  if (!make_map(&tw_mn, w, D, V, D, 64)) return ULY_ERR_CUDA;
  for (long long t0 = 0; t0 < tokens; t0 += q.piece) {
    const int rows = (int)(tokens - t0 < q.piece ? tokens - t0 : q.piece);
    void *pp = at<char>(ws, q.p), *xk = at<char>(ws, q.xk);
    LossParams p = {};
    if (!make_map(&tz, pp, V, rows, q.ldp, kHalf) || !make_map(&tz_mn, pp, V, rows, q.ldp, 64) ||
        !make_map(&tk_mn, xk, D, rows, q.ldx, 64))
      return ULY_ERR_CUDA;
    p.labels = labels + t0;
    p.pairs = at<float2>(ws, q.pairs);
    p.target = at<float>(ws, q.target);
    p.rows_pad = q.rows_pad;
    p.rows = rows; p.vocab = V; p.ignore_index = ignore_index;
    uly_status st = logits_pass<true>(xb + t0 * D, w, D, p, pp, q.ldp, stream);
    if (st != ULY_OK) return st;
    RowsParams r = rows_of(q, p, ws, t0);
    r.row_lse = at<float>(ws, q.row_lse);
    r.factor = at<float>(ws, q.factor);
    GradParams g = {};
    g.factor = r.factor; g.row_lse = r.row_lse; g.target = r.target; g.labels = r.labels;
    g.p = static_cast<uint4 *>(pp);
    g.x = reinterpret_cast<const uint4 *>(xb + t0 * D);
    g.xk = static_cast<uint4 *>(xk);
    g.ldp = q.ldp; g.ldx = q.ldx; g.slots = r.slots; g.vocab = V; g.ignore_index = ignore_index; g.hidden = D; g.rows = rows; g.closing = closed;
    g.close = close;
    {
      prof::Scope scope(prof::K_LINEAR_LOSS_ROWS, stream);
      loss_rows_kernel<true><<<(rows + kRowsCta - 1) / kRowsCta, kRowThreads, 0, stream>>>(r);
      const long long cols = (V + kGradCols - 1) / kGradCols;
      const long long ctas = ((long long)device_sm_count() * kGradPerSm + cols - 1) / cols;
      loss_grad_kernel<<<dim3((unsigned)((rows < ctas ? rows : ctas) + closed), (unsigned)cols), kGradThreads, 0, stream>>>(g);
      note_launches(2);
      if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
    }
    // dx = dz W
    PlainParams o = {};
    o.out = dxb + t0 * D;
    o.over = count;
    o.M = rows; o.N = D;
    float *part = at<float>(ws, q.part);
    st = skinny::faster(rows, D, V, q.part_bytes)
             ? skinny::launch_plain_mn(pp, q.ldp, w, o.out, count, rows, D, V, prof::K_LINEAR_LOSS_DX, stream)
             : launch_plain<false>(tz, tw_mn, o, V, part, q.part_bytes, prof::K_LINEAR_LOSS_DX, stream);
    if (st != ULY_OK) return st;
    // dW (+)= dz^T x; the last piece writes the caller's type
    const bool last = t0 + rows >= tokens;
    o = PlainParams{};
    o.over = count;
    o.M = V; o.N = D;
    float *acc = q.dw_acc ? at<float>(ws, q.acc) : static_cast<float *>(dw);
    o.add = t0 > 0 ? acc : nullptr;
    o.out = last ? dw : acc;
    o.out_f32 = !last || dw_dtype == ULY_F32;
    st = launch_plain<true>(tz_mn, tk_mn, o, rows, part, q.part_bytes, prof::K_LINEAR_LOSS_DW, stream);
    if (st != ULY_OK) return st;
  }
  return closed ? ULY_OK : finish(q, close, tokens, ws, stream);
}

}  // namespace uly
