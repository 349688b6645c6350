// The token-weighted cross-entropy taken straight from the hidden states,
// z = x W^T over the whole vocabulary, without a logits tensor:
//
//   l_t = logsumexp_v(z_tv) - z_t[y_t],  S_r, C_r, L as ulysses_loss_aggregate
//   dx = dz W,  dW = dz^T x,  dz_tv = (softmax(z_t)_v - [v == y_t]) / C
//
// Forward: the product's epilogue keeps, for each 128 columns of a row, their
// maximum and the sum of exp(z - maximum) (fp32); a second kernel folds a
// row's pairs into its logsumexp.  No logit leaves the tensor memory.
//
// Gradient, in pieces of tokens: the logits are formed once.  The epilogue
// stores p_tv = exp(z_tv - c_t) in bf16 against a reference c_t of the row (the
// largest logit of the first 256 columns, a small product of its own).  bf16
// has fp32's exponents, so p keeps its 8 significant bits wherever it lies
// between e^-80 and e^40, and no second pass over it is needed: with
// g_t = exp(c_t - lse_t) / C,
//   dz_tv = g_t (p_tv - [v == y_t] exp(lse_t - c_t)),
// the label's element of p is replaced once lse is known (as
// exp(lse - c) expm1(z_y - lse), exact for confident tokens too), dx takes g_t
// in its product's epilogue and dW takes it through x' = g_t x (bf16).  A row
// with a logit more than 40 above c_t stores those 128 columns against their
// own maximum instead and is brought to c_t = lse_t when its logsumexp is
// known (a pass over that row alone).
// Roundings to bf16: p, x', dx, (dW); each at most half a step, 2^-8 relative.
//
// Three products of 2 T D V operations, the fewest that do not keep the
// logits of all tokens in a wider type; bound by the tensor cores, with few
// tokens by W's bytes.
#include "gemm_sm100.cuh"
#include "tokenwise.cuh"

namespace uly {

using namespace gemm;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxAbove = 40.f;   // p up to e^40; sums over any vocabulary stay far inside fp32
constexpr int kSlot = kHalf;        // columns behind one (reference, sum) pair
constexpr int kProbe = kTile;       // columns the row references are taken from
constexpr long long kPieceBytes = 4ll << 30;    // p of one piece of tokens
constexpr long long kPairBytes = 128ll << 20;   // pairs of one forward piece

struct LossParams {
  const int32_t *labels;   // of the piece's rows
  float2 *pairs;           // [slots][rows_pad]: (reference, sum of exp(z - reference))
  float *target;           // [rows]: z[label]
  const float *ref;        // STORE_P: [rows] row references
  __nv_bfloat16 *p;        // STORE_P: [rows][ldp]
  long long ldp, rows_pad;
  int rows, vocab, ignore_index;
};

template <bool STORE_P>
struct EpiLoss {
  using Params = LossParams;
  static __device__ __forceinline__ void tile(const Params &p, const Unit &w, uint32_t acc, int row, int half) {
    const int col0 = w.nt * kTile + half * kSlot;
    const int ncol = min(kSlot, p.vocab - col0);   // columns of the vocabulary here; may be <= 0
    const bool ok = row < p.rows;
    const int y = ok ? __ldg(p.labels + row) : p.ignore_index;
    const bool counted = y != p.ignore_index && y >= 0 && y < p.vocab;
    float m = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kSlot; c += 32) {
      uint32_t a[32];
      tmem_ld32(acc + half * kSlot + c, a);
      if (c + 32 <= ncol) {
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, __uint_as_float(a[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c + e < ncol) m = fmaxf(m, __uint_as_float(a[e]));
      }
    }
    float ref = m == -INFINITY ? 0.f : m;   // every logit -inf: each term is 0
    if (STORE_P && ok) {
      const float r = __ldg(p.ref + row);
      if (m - r <= kMaxAbove) ref = r;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c = 0; c < kSlot; c += 32) {
      uint32_t a[32];
      tmem_ld32(acc + half * kSlot + c, a);
      if (counted && y >= col0 + c && y < col0 + c + 32) {
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) t = y == col0 + c + e ? __uint_as_float(a[e]) : t;
        p.target[row] = t;
      }
      if (c < ncol) {
        float q[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          q[e] = ex2_approx((__uint_as_float(a[e]) - ref) * kLog2e);   // the difference first: exact at any size
          if (c + 32 > ncol && c + e >= ncol) q[e] = 0.f;
          s[e & 3] += q[e];
        }
        if (STORE_P && ok) {
          __nv_bfloat16 *o = p.p + row * p.ldp + col0 + c;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (c + 8 * g < ncol) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = counted ? q[8 * g + e] : 0.f;
              store8(o + 8 * g, v);
            }
          }
        }
      }
      __syncwarp();
    }
    if (ok && ncol > 0)
      p.pairs[(long long)(w.nt * 2 + half) * p.rows_pad + row] = make_float2(ref, (s[0] + s[1]) + (s[2] + s[3]));
  }
};

// Row references from the probe's pairs: the larger of its (at most two) maxima.
__global__ void __launch_bounds__(256) row_ref_kernel(const float2 *__restrict__ pairs, long long rows_pad, int slots,
                                                      int rows, float *__restrict__ ref) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  float m = pairs[r].x;
  if (slots > 1) m = fmaxf(m, pairs[rows_pad + r].x);
  ref[r] = m;
}

// 32 rows a CTA, lane = row: the warps fold strips of a row's pairs, joined in
// a fixed order, into lse and the row's loss.  GRAD: also the row's factor
// g = exp(ref - lse) / C, the label's element of p, x' = g x, and rows with a
// slot kept against its own maximum brought to the one reference lse.
struct RowsParams {
  const float2 *pairs;
  const float *target, *ref;
  const int32_t *labels;
  float *row_loss;            // of the piece's rows
  const long long *count;
  float *g;
  __nv_bfloat16 *p, *xg;
  const __nv_bfloat16 *x;
  long long ldp, rows_pad;
  int rows, slots, vocab, ignore_index, hidden;
  int *err;
};
constexpr int kRowWarps = 16;

template <bool GRAD>
__global__ void __launch_bounds__(32 * kRowWarps) loss_rows_kernel(const RowsParams p) {
  __shared__ float sh_m[kRowWarps][32], sh_s[kRowWarps][32];
  __shared__ float sh_g[32], sh_lse[32];
  __shared__ int sh_odd[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * 32, row = row0 + lane;
  const bool ok = row < p.rows;
  const float ref = GRAD && ok ? p.ref[row] : 0.f;
  const int y = ok ? __ldg(p.labels + row) : p.ignore_index;
  const bool counted = y != p.ignore_index && y >= 0 && y < p.vocab;
  float m = -INFINITY, s = 0.f;
  bool odd = false;
  if (threadIdx.x < 32) sh_odd[threadIdx.x] = 0;
  if (ok) {
    for (int k = warp; k < p.slots; k += kRowWarps) {
      const float2 v = __ldg(p.pairs + (long long)k * p.rows_pad + row);
      if (GRAD && counted && v.x != ref) odd = true;
      if (v.y == 0.f) continue;
      const float mm = fmaxf(m, v.x);
      s = s * exp2f((m - mm) * kLog2e) + v.y * exp2f((v.x - mm) * kLog2e);
      m = mm;
    }
  }
  sh_m[warp][lane] = m;
  sh_s[warp][lane] = s;
  __syncthreads();
  if (odd) sh_odd[lane] = 1;
  if (warp == 0) {
    for (int k = 1; k < kRowWarps; ++k) {
      const float m2 = sh_m[k][lane], s2 = sh_s[k][lane];
      if (s2 == 0.f) continue;
      const float mm = fmaxf(m, m2);
      s = s * exp2f((m - mm) * kLog2e) + s2 * exp2f((m2 - mm) * kLog2e);
      m = mm;
    }
    const float lse = m + logf(s);
    if (ok) {
      if (y != p.ignore_index && !counted) raise_error(p.err, ULY_ERR_LABEL);
      p.row_loss[row] = counted ? lse - p.target[row] : 0.f;
    }
    sh_lse[lane] = counted ? lse : 0.f;
    sh_g[lane] = 0.f;
  }
  if (!GRAD) return;
  __syncthreads();
  // a row that has columns against another reference: all of them against lse
  for (int r = 0; r < 32; ++r) {
    if (!sh_odd[r] || row0 + r >= p.rows) continue;
    const float to = sh_lse[r];
    __nv_bfloat16 *pr = p.p + (long long)(row0 + r) * p.ldp;
    for (int v = threadIdx.x; v < p.vocab; v += blockDim.x) {
      const float from = __ldg(p.pairs + (long long)(v / kSlot) * p.rows_pad + row0 + r).x;
      pr[v] = __float2bfloat16_rn(__bfloat162float(pr[v]) * exp2f((from - to) * kLog2e));
    }
  }
  __syncthreads();
  if (warp == 0 && ok) {
    float g = 0.f;
    if (counted) {
      const float lse = sh_lse[lane], base = sh_odd[lane] ? lse : ref;
      const double inv = 1.0 / (double)*p.count;
      g = (float)inv * expf(base - lse);
      // z_y <= lse but for rounding: the label's softmax is at most 1
      p.p[(long long)row * p.ldp + y] =
          __float2bfloat16_rn(expf(lse - base) * expm1f(fminf(p.target[row] - lse, 0.f)));
    }
    p.g[row] = g;
    sh_g[lane] = g;
  }
  __syncthreads();
  const int vecs = p.hidden / 8, nrows = min(32, p.rows - row0);
  for (int i = threadIdx.x; i < nrows * vecs; i += blockDim.x) {
    const int r = i / vecs;
    const long long at = (long long)(row0 + r) * p.hidden + (i - r * vecs) * 8;
    const float g = sh_g[r];
    float v[8];
    load8(p.x + at, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = g == 0.f ? 0.f : v[e] * g;   // an ignored row may hold anything
    store8(p.xg + at, v);
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
  long long piece, rows_pad, ldp;
  int slots, dx_splits, dw_splits;
  bool dw_acc;   // dW of several pieces is summed in an fp32 array of the workspace
  size_t psum, pcnt, count, row_loss, target, pairs, ref, g, p, xg, part, acc, bytes;   // offsets, total
};

Plan make_plan(int P, long long T, int D, int V, bool grad, int dw_dtype, long long piece_tokens) {
  Plan q = {};
  q.slots = (V + kTile - 1) / kTile * 2;
  q.ldp = round_up(V, 8);
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
    const int sms = device_sm_count();
    auto tiles = [](long long v) { return (v + kTile - 1) / kTile; };
    q.dx_splits = choose_splits(q.piece, D, tiles(q.piece), tiles(D), (V + kBK - 1) / kBK, sms);
    q.dw_splits = choose_splits(V, D, tiles(V), tiles(D), (q.piece + kBK - 1) / kBK, sms);
    q.dw_acc = q.piece < T && dw_dtype == ULY_BF16;
    q.ref = take((size_t)q.piece * sizeof(float));
    q.g = take((size_t)q.piece * sizeof(float));
    q.p = take((size_t)q.piece * q.ldp * 2);
    q.xg = take((size_t)q.piece * D * 2);
    const size_t a = part_bytes(q.piece, D, q.dx_splits), b = part_bytes(V, D, q.dw_splits);
    q.part = take(a > b ? a : b);
    q.acc = take(q.dw_acc ? (size_t)V * D * sizeof(float) : 0);
  }
  q.bytes = at;
  return q;
}

template <typename T>
T *at(void *ws, size_t off) { return reinterpret_cast<T *>(static_cast<char *>(ws) + off); }

uly_status finish(const Plan &q, int P, long long T, int V, const int32_t *labels, int ignore_index, float *shard_sum,
                  int64_t *shard_count, float *loss, void *ws, cudaStream_t stream) {
  shard_sum_kernel<<<P, 256, 0, stream>>>(at<float>(ws, q.row_loss), labels, T / P, V, ignore_index,
                                          at<double>(ws, q.psum), at<long long>(ws, q.pcnt));
  note_launches(1);
  loss_finalize_launch(at<double>(ws, q.psum), at<long long>(ws, q.pcnt), P, 1, shard_sum, shard_count, loss, stream);
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
  CUtensorMap ta, tb;
  if (!make_map(&tb, w, D, V, D, kHalf)) return ULY_ERR_CUDA;
  for (long long t0 = 0; t0 < tokens; t0 += q.piece) {
    const int rows = (int)(tokens - t0 < q.piece ? tokens - t0 : q.piece);
    if (!make_map(&ta, xb + t0 * D, D, rows, D, kHalf)) return ULY_ERR_CUDA;
    LossParams p = {};
    p.labels = labels + t0;
    p.pairs = at<float2>(ws, q.pairs);
    p.target = at<float>(ws, q.target);
    p.rows_pad = q.rows_pad;
    p.rows = rows; p.vocab = V; p.ignore_index = ignore_index;
    {
      prof::Scope scope(prof::K_LINEAR_LOSS, stream);
      const uly_status st = launch<EpiLoss<false>, false, false>(ta, tb, make_shape(rows, V, D, kTile, 1), p, stream);
      if (st != ULY_OK) return st;
    }
    RowsParams r = {};
    r.pairs = p.pairs; r.target = p.target; r.labels = p.labels;
    r.row_loss = at<float>(ws, q.row_loss) + t0;
    r.rows_pad = q.rows_pad; r.rows = rows; r.slots = (V + kSlot - 1) / kSlot; r.vocab = V; r.ignore_index = ignore_index;
    r.err = error_word();
    prof::Scope scope(prof::K_LINEAR_LOSS_ROWS, stream);
    loss_rows_kernel<false><<<(rows + 31) / 32, 32 * kRowWarps, 0, stream>>>(r);
    note_launches(1);
    if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
  }
  return finish(q, P, tokens, V, labels, ignore_index, shard_sum, shard_count, loss, ws, stream);
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
  loss_count_launch(labels, tokens, V, ignore_index, count, stream);
  CUtensorMap tw, tw_mn, tx, tp, tp_mn, tg_mn;
  if (!make_map(&tw, w, D, V, D, kHalf) || !make_map(&tw_mn, w, D, V, D, 64)) return ULY_ERR_CUDA;
  for (long long t0 = 0; t0 < tokens; t0 += q.piece) {
    const int rows = (int)(tokens - t0 < q.piece ? tokens - t0 : q.piece);
    __nv_bfloat16 *pp = at<__nv_bfloat16>(ws, q.p), *xg = at<__nv_bfloat16>(ws, q.xg);
    if (!make_map(&tx, xb + t0 * D, D, rows, D, kHalf) || !make_map(&tp, pp, V, rows, q.ldp, kHalf) ||
        !make_map(&tp_mn, pp, V, rows, q.ldp, 64) || !make_map(&tg_mn, xg, D, rows, D, 64))
      return ULY_ERR_CUDA;
    LossParams p = {};
    p.labels = labels + t0;
    p.pairs = at<float2>(ws, q.pairs);
    p.target = at<float>(ws, q.target);
    p.rows_pad = q.rows_pad;
    p.rows = rows; p.ignore_index = ignore_index;
    float *ref = at<float>(ws, q.ref);
    {
      prof::Scope scope(prof::K_LINEAR_LOSS, stream);
      // the row references: the same product over the first columns of the vocabulary
      p.vocab = V < kProbe ? V : kProbe;
      uly_status st = launch<EpiLoss<false>, false, false>(tx, tw, make_shape(rows, p.vocab, D, kTile, 1), p, stream);
      if (st != ULY_OK) return st;
      row_ref_kernel<<<(rows + 255) / 256, 256, 0, stream>>>(p.pairs, q.rows_pad, p.vocab > kSlot ? 2 : 1, rows, ref);
      note_launches(1);
      p.vocab = V;
      p.ref = ref;
      p.p = pp;
      p.ldp = q.ldp;
      st = launch<EpiLoss<true>, false, false>(tx, tw, make_shape(rows, V, D, kTile, 1), p, stream);
      if (st != ULY_OK) return st;
    }
    RowsParams r = {};
    r.pairs = p.pairs; r.target = p.target; r.ref = ref; r.labels = p.labels;
    r.row_loss = at<float>(ws, q.row_loss) + t0;
    r.count = count;
    r.g = at<float>(ws, q.g);
    r.p = pp; r.xg = xg; r.x = xb + t0 * D;
    r.ldp = q.ldp; r.rows_pad = q.rows_pad;
    r.rows = rows; r.slots = (V + kSlot - 1) / kSlot; r.vocab = V; r.ignore_index = ignore_index; r.hidden = D;
    r.err = error_word();
    {
      prof::Scope scope(prof::K_LINEAR_LOSS_ROWS, stream);
      loss_rows_kernel<true><<<(rows + 31) / 32, 32 * kRowWarps, 0, stream>>>(r);
      note_launches(1);
      if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
    }
    // dx = g (p W)
    PlainParams o = {};
    o.out = dxb + t0 * D;
    o.row_scale = r.g;
    o.M = rows; o.N = D;
    float *part = at<float>(ws, q.part);
    uly_status st = launch_plain<false, true>(tp, tw_mn, o, V, q.dx_splits, part, prof::K_LINEAR_LOSS_DX, stream);
    if (st != ULY_OK) return st;
    // dW (+)= p^T x'; the last piece writes the caller's type
    const bool last = t0 + rows >= tokens;
    o = PlainParams{};
    o.M = V; o.N = D;
    float *acc = q.dw_acc ? at<float>(ws, q.acc) : static_cast<float *>(dw);
    o.add = t0 > 0 ? acc : nullptr;
    o.out = last ? dw : acc;
    o.out_f32 = !last || dw_dtype == ULY_F32;
    st = launch_plain<true, true>(tp_mn, tg_mn, o, rows, q.dw_splits, part, prof::K_LINEAR_LOSS_DW, stream);
    if (st != ULY_OK) return st;
  }
  return finish(q, P, tokens, V, labels, ignore_index, shard_sum, shard_count, loss, ws, stream);
}

}  // namespace uly
