// The linear product of a rank's tokens with its epilogue, and its gradients:
//
//   z = x W^T + bias        y = act(z) + residual
//
// act: identity, gelu (tanh form), silu, or swiglu, where W holds the gate's
// rows and then the other factor's, y = silu(z_gate) z_up: a tile takes the
// same 128 features of both, so the two halves of an accumulator row meet in
// one thread.  y comes from the fp32 z; y and the optionally kept z are rounded
// to bf16 once each.
//
// Backward: dz = dy act'(z) is formed once (bf16, the products' operand type;
// the bias gradient takes it in fp32 before that rounding), then dx = dz W and
// dW = dz^T x on the tensor cores, dW with both operands MN-major.
//
// Bound by the tensor cores from a few hundred tokens on, by W's bytes below.
#include "skinny_sm100.cuh"
#include "tokenwise.cuh"

namespace uly {

using namespace gemm;

namespace {

// 1 / (1 + e^-v): e^-v overflows to infinity for large negative v, and the
// quotient is then 0.
__device__ __forceinline__ float sigmoid_fast(float v) {
  return __fdividef(1.f, 1.f + ex2_approx(v * -1.4426950408889634f));
}

// gelu, tanh form: 0.5 z (1 + tanh(t)) = z sigmoid(2t), t = sqrt(2/pi)(z + 0.044715 z^3).
constexpr float kGelu2c = 1.5957691216057308f, kGelu3 = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_of(float z, float up) {
  if (ACT == ULY_ACT_SILU) return z * sigmoid_fast(z);
  if (ACT == ULY_ACT_SWIGLU) return z * sigmoid_fast(z) * up;
  if (ACT == ULY_ACT_GELU) {
    const float c = fminf(fmaxf(z, -20.f), 20.f);   // beyond, sigmoid(2t) is 0 or 1 and z^3 could overflow
    return z * sigmoid_fast(kGelu2c * fmaf(kGelu3 * c * c, c, c));
  }
  return z;
}

// act'(z); swiglu: the derivatives by the gate (times up) and by up.
template <int ACT>
__device__ __forceinline__ float dact_of(float z) {
  if (ACT == ULY_ACT_GELU) {
    const float c = fminf(fmaxf(z, -20.f), 20.f);
    const float s = sigmoid_fast(kGelu2c * fmaf(kGelu3 * c * c, c, c));
    return fmaf(z * (s * (1.f - s)) * kGelu2c, fmaf(3.f * kGelu3 * c, c, 1.f), s);
  }
  const float s = sigmoid_fast(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

struct LinearParams {
  CUtensorMap y_map, pre_map, up_map;     // y, and the parts of pre (up: swiglu)
  const __nv_bfloat16 *bias, *residual;   // nullable; the residual may be y itself: no read-only loads of it
  __nv_bfloat16 *y, *pre;                 // pre nullable: z [M][NZ]
  long long M;
  int N, NZ;                              // output features, rows of W
};

template <int ACT>
struct EpiLinear {
  using Params = LinearParams;
  static constexpr bool kGated = ACT == ULY_ACT_SWIGLU;

  static __device__ __forceinline__ void add_bias(const Params &p, int col, float (&z)[8], float (&up)[8]) {
    if (!p.bias) return;
    float b[8];
    load8(p.bias + col, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += b[e];
    if (kGated) {
      load8(p.bias + p.N + col, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) up[e] += b[e];
    }
  }
  static __device__ __forceinline__ void join8(const Params &p, long long row, int col, float (&z)[8],
                                               float (&up)[8]) {
    uint4 r = make_uint4(0, 0, 0, 0);   // asked for before pre is stored
    if (p.residual) r = *reinterpret_cast<const uint4 *>(p.residual + row * p.N + col);
    add_bias(p, col, z, up);
    if (p.pre) {
      store8(p.pre + row * p.NZ + col, z);
      if (kGated) store8(p.pre + row * p.NZ + p.N + col, up);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = act_of<ACT>(z[e], up[e]);
    if (p.residual) {
      float x[8];
      unpack8(r, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] += x[e];
    }
    store8(p.y + row * p.N + col, z);
  }

  // A warp's 32 rows x 64 columns of the residual, read along the rows while the
  // tile's product or the step before is under way.  (Each lane's own row, 16 bytes
  // at a time, looks up 32 lines an instruction.  8192 x 64 -> 8192 that way and in
  // steps of 32 columns: 86 us with a residual, 47 without; this way 64 and 28.)
  struct Ahead {
    uint4 v[8];
    __device__ __forceinline__ void load(const Params &p, long long row0, int col0, int lane) {
      const int col = col0 + 8 * (lane & 7);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const long long row = row0 + 4 * i + (lane >> 3);
        if (row < p.M && col < p.N) v[i] = *reinterpret_cast<const uint4 *>(p.residual + row * p.N + col);
      }
    }
  };
  // Columns of one warp, from column first() of the output on.  A narrow gated
  // tile has 64: one warpgroup writes y, the other pre.
  template <int TN>
  static constexpr int kTileCols = kGated ? TN / 2 : TN;
  template <int TN>
  static constexpr bool kRoles = kTileCols<TN> == 64;
  template <int TN>
  static constexpr int kCols = kRoles<TN> ? 64 : kTileCols<TN> / 2;
  template <int TN>
  static __device__ __forceinline__ int first(const Unit &w, int half) {
    return w.nt * kTileCols<TN> + (kRoles<TN> ? 0 : half * kCols<TN>);
  }
  template <int TN>
  static __device__ __forceinline__ Ahead before(const Params &p, const Unit &w, int row0, int half, int lane) {
    Ahead next = {};
    if (p.residual && (!kRoles<TN> || half == 0)) next.load(p, row0, first<TN>(w, half), lane);
    return next;
  }
  static __device__ __forceinline__ void bias32(const Params &p, int col, int shift, uint32_t *a) {
    if (!p.bias) return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (col + 8 * g < p.N) {
        float b[8];
        load8(p.bias + shift + col + 8 * g, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[8 * g + e] = __float_as_uint(__uint_as_float(a[8 * g + e]) + b[e]);
      }
  }
  static __device__ __forceinline__ void send64(const CUtensorMap *map, const uint32_t (&a)[64], int col0, int row0,
                                                OutRing &out) {
    out.begin();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        v[e] = pack_bf16x2(__uint_as_float(a[32 * h + 2 * e]), __uint_as_float(a[32 * h + 2 * e + 1]));
      out.write(h, v);
    }
    out.end(map, col0, row0);
  }

  template <int TN>
  static __device__ __forceinline__ void tile(const Params &p, const Unit &w, uint32_t acc, int row, int half,
                                              Ahead &next, OutRing &out) {
    constexpr int cols = kCols<TN>;
    const int row0 = row - out.lane, col_first = first<TN>(w, half);
    const bool do_y = !kRoles<TN> || half == 0, do_pre = p.pre && (!kRoles<TN> || half == 1);
    if (row0 >= p.M) return;   // the whole warp, here and below
    if (!kRoles<TN>) acc += half * cols;
#pragma unroll 1
    for (int c = 0; c < cols; c += 64) {
      const int col0 = col_first + c;
      if (col0 >= p.N) return;
      uint32_t a[64];
      if (kGated) {
        if (do_pre)
#pragma unroll 1
          for (int up = 0; up < 2; ++up) {
            tmem_ld64(acc + c + up * (TN / 2), a);
            bias32(p, col0, up * p.N, a);
            bias32(p, col0 + 32, up * p.N, a + 32);
            send64(up ? &p.up_map : &p.pre_map, a, col0, row0, out);
          }
      } else {
        tmem_ld64(acc + c, a);
        bias32(p, col0, 0, a);
        bias32(p, col0 + 32, 0, a + 32);
        if (do_pre) send64(&p.pre_map, a, col0, row0, out);
      }
      if (!do_y) continue;
      out.begin();
      if (p.residual) {
        out.stage(next.v);
        if (c + 64 < cols) next.load(p, row0, col0 + 64, out.lane);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[kGated ? 64 : 1];
        if constexpr (kGated) {
          tmem_ld32x2(acc + c + 32 * h, acc + c + TN / 2 + 32 * h, b);
          bias32(p, col0 + 32 * h, 0, b);
          bias32(p, col0 + 32 * h, p.N, b + 32);
        }
        uint32_t v[16], r[16];
        if (p.residual) out.read(h, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float y[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (kGated) y[i] = act_of<ACT>(__uint_as_float(b[2 * e + i]), __uint_as_float(b[32 + 2 * e + i]));
            else y[i] = act_of<ACT>(__uint_as_float(a[32 * h + 2 * e + i]), 0.f);
          }
          if (p.residual) {
            y[0] += __uint_as_float(r[e] << 16);
            y[1] += __uint_as_float(r[e] & 0xffff0000u);
          }
          v[e] = pack_bf16x2(y[0], y[1]);
        }
        out.write(h, v);
      }
      out.end(&p.y_map, col0, row0);
    }
  }
};

// Few tokens: this CTA's slice of a tile's features, four of a token a thread.
template <int ACT>
struct SkinnyLinear {
  using Params = LinearParams;
  static constexpr bool kGated = ACT == ULY_ACT_SWIGLU;
  static constexpr int kCols = kGated ? 64 : 128;
  // (128 x 2560 -> 10240 with a residual: 31 us without, 28 so.)
  static __device__ __forceinline__ void prefetch(const Params &p, int index, int rank, int ranks) {
    if (!p.residual) return;
    skinny::for_slice(kCols, rank, ranks, (int)p.M, [&](int row, int t) {
      const int col = index * kCols + row;
      if (col < p.N) skinny::prefetch_l2(p.residual + (long long)t * p.N + col);
    }, 64);
  }
  template <class T>
  static __device__ __forceinline__ void finish(const Params &p, const T &tile, int index, int rank, int ranks) {
    skinny::for_slice(kCols, rank, ranks, (int)p.M, [&](int row, int t) {
      const int col = index * kCols + row;   // N is a multiple of 8
      if (col >= p.N) return;
      float z[4], up[4] = {}, b[4];
      tile.sum4(row, t, z);
      if (kGated) tile.sum4(64 + row, t, up);
      if (p.bias) {
        skinny::load4(p.bias + col, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] += b[e];
        if (kGated) {
          skinny::load4(p.bias + p.N + col, b);
#pragma unroll
          for (int e = 0; e < 4; ++e) up[e] += b[e];
        }
      }
      if (p.pre) {
        skinny::store4(p.pre + (long long)t * p.NZ + col, z);
        if (kGated) skinny::store4(p.pre + (long long)t * p.NZ + p.N + col, up);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = act_of<ACT>(z[e], up[e]);
      if (p.residual) {
        skinny::unpack4(*reinterpret_cast<const uint2 *>(p.residual + (long long)t * p.N + col), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] += b[e];
      }
      skinny::store4(p.y + (long long)t * p.N + col, z);
    });
  }
};

template <int ACT>
uly_status run_skinny(const void *x, const void *w, const LinearParams &p, int K, cudaStream_t stream) {
  prof::Scope scope(prof::K_LINEAR, stream);
  constexpr int cols = SkinnyLinear<ACT>::kCols;
  const int tiles = (p.N + cols - 1) / cols;
  return skinny::launch<SkinnyLinear<ACT>, false>(w, K, p.NZ, x, K, p.M, K, tiles,
                                                  skinny::cluster_size(p.M, tiles, (K + kBK - 1) / kBK), cols,
                                                  cols == 64 ? p.N : 64, p, stream);
}

int gated(int act) { return act == ULY_ACT_SWIGLU ? 2 : 1; }

Cut linear_cut(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  return choose_cut(tiles_of(tokens), tiles_of(out, kTile / gated(act)), tiles_of(out, kNarrow / gated(act)),
                    (in + kBK - 1) / kBK);
}

template <int ACT>
uly_status run_linear(const void *x, const void *w, LinearParams p, int K, float *part, cudaStream_t stream) {
  const Cut cut = linear_cut(p.M, K, p.N, ACT);
  using Epi = EpiLinear<ACT>;
  CUtensorMap ta, tb;
  if (!make_map(&ta, x, K, p.M, K, kHalf) || !make_map(&tb, w, K, p.NZ, K, b_box(cut)) ||
      !make_out_map(&p.y_map, p.y, p.N, p.M, p.N) || (p.pre && !make_out_map(&p.pre_map, p.pre, p.N, p.M, p.NZ)) ||
      (p.pre && p.NZ > p.N && !make_out_map(&p.up_map, p.pre + p.N, p.N, p.M, p.NZ)))
    return ULY_ERR_CUDA;
  const Shape s = make_shape(p.M, p.N, K, gated(ACT), cut);
  prof::Scope scope(prof::K_LINEAR, stream);
  const uly_status st = launch<Epi, false, false>(ta, tb, s, cut, p, part, stream);
  return st != ULY_OK ? st : launch_join<Epi>(p, s, cut, part, p.M, p.N, stream);
}

// ------------------------------------------------------------ dz and dbias
// dz[t][c] for 8 columns a thread; rows of one CTA's strip summed per column
// into a partial of the bias gradient (fp32, before dz is rounded).
struct DzParams {
  const __nv_bfloat16 *pre, *dy;   // pre null: act none, dz = dy (only the sums are formed)
  __nv_bfloat16 *dz;
  float *part;                     // [gridDim.y][NZ]; null without a bias gradient
  long long M;
  int N, NZ, rows_per_cta;
  long long ld;                    // row stride of dz
};

template <int ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const DzParams p) {
  constexpr bool kGated = ACT == ULY_ACT_SWIGLU;
  const int strip = threadIdx.x >> 5, col = (blockIdx.x * 32 + (threadIdx.x & 31)) * 8;
  const bool mine = col < p.N;
  float s0[8] = {}, s1[8] = {};
  const long long r0 = (long long)blockIdx.y * p.rows_per_cta;
  const long long r1 = r0 + p.rows_per_cta < p.M ? r0 + p.rows_per_cta : p.M;
#pragma unroll 2
  for (long long r = mine ? r0 + strip : r1; r < r1; r += 8) {
    float d[8], z[8];
    load8(p.dy + r * p.N + col, d);
    if (ACT == ULY_ACT_NONE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s0[e] += d[e];
      continue;
    }
    load8(p.pre + r * p.NZ + col, z);
    if (kGated) {
      float up[8], a[8], b[8];
      load8(p.pre + r * p.NZ + p.N + col, up);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = sigmoid_fast(z[e]);
        b[e] = d[e] * (z[e] * s);
        a[e] = d[e] * up[e] * (s * fmaf(z[e], 1.f - s, 1.f));
        s0[e] += a[e];
        s1[e] += b[e];
      }
      store8(p.dz + r * p.ld + col, a);
      store8(p.dz + r * p.ld + p.N + col, b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= dact_of<ACT>(z[e]);
        s0[e] += d[e];
      }
      store8(p.dz + r * p.ld + col, d);
    }
  }
  if (p.part) {   // the strips' sums, in their order
    __shared__ __align__(16) float sh[8][256];
    const int c = blockIdx.x * 256 + threadIdx.x;
    float *o = p.part + (long long)blockIdx.y * p.NZ + c;
#pragma unroll
    for (int h = 0; h < (kGated ? 2 : 1); ++h) {
      if (h) __syncthreads();
      store8(&sh[strip][(threadIdx.x & 31) * 8], h ? s1 : s0);
      __syncthreads();
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a += sh[e][threadIdx.x];
      if (c < p.N) o[h ? p.N : 0] = a;
    }
  }
}

// Up to so many rows one CTA a column of them forms the bias gradient alone (2
// tokens of 2392 -> 936, the whole backward: 24.6 -> 20.7 us).
constexpr int kOneCtaRows = 64;
// CTAs along the tokens: about eight an SM in all, of at least 64 rows, or of 16
// where that leaves SMs without one (391 x 808: 10.2 -> 4.9 us).
int dz_row_ctas(int64_t tokens, int32_t out) {
  const long long cols = (out / 8 + 31) / 32;
  const long long sms = device_sm_count();
  long long ctas = sms * 8 / cols, most = (tokens + 63) / 64;
  if (most * cols < sms) {
    most = (tokens + 15) / 16;
    if (most * cols > sms) most = (sms + cols - 1) / cols;
  }
  if (ctas > most) ctas = most;
  return (int)(ctas < 1 ? 1 : ctas);
}

// Workspace of the backward: dz, the bias gradient's partials, a cut product's
// partials (the two products run one after the other and share them).
struct BwdPlan {
  int nz, row_ctas;
  long long ld;   // row stride of dz (dy itself without an activation)
  size_t off_bias, off_part, part, bytes;
};
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
BwdPlan bwd_plan(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  BwdPlan q;
  q.nz = out * gated(act);
  q.row_ctas = dz_row_ctas(tokens, out);
  q.ld = act == ULY_ACT_NONE ? q.nz : (q.nz + kRowAlign - 1) / kRowAlign * kRowAlign;
  q.off_bias = act == ULY_ACT_NONE ? 0 : up256((size_t)tokens * q.ld * 2);
  q.off_part = q.off_bias + up256((size_t)q.row_ctas * q.nz * sizeof(float));
  const size_t a = plain_cut(tokens, in, q.nz).bytes, b = plain_cut(q.nz, in, tokens).bytes;
  q.part = a > b ? a : b;
  q.bytes = q.off_part + up256(q.part);
  return q;
}


// Few tokens: the weights' bytes bound the product and the skinny kernel streams
// them best.
bool few_tokens(int64_t tokens) { return tokens <= skinny::kMaxTokens; }

template <int ACT>
uly_status linear_of(const void *x, const void *w, const LinearParams &p, int K, void *workspace, cudaStream_t stream) {
  if (few_tokens(p.M)) return run_skinny<ACT>(x, w, p, K, stream);
  return run_linear<ACT>(x, w, p, K, static_cast<float *>(workspace), stream);
}

}  // namespace

size_t linear_workspace_bytes(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  if (few_tokens(tokens)) return 0;
  return linear_cut(tokens, in, out, act).bytes;
}

uly_status linear_launch(int64_t tokens, int32_t in, int32_t out, int32_t act, const void *x, const void *w,
                         const void *bias, const void *residual, void *y, void *pre, void *workspace,
                         cudaStream_t stream) {
  LinearParams p = {};
  p.bias = static_cast<const __nv_bfloat16 *>(bias);
  p.residual = static_cast<const __nv_bfloat16 *>(residual);
  p.y = static_cast<__nv_bfloat16 *>(y);
  p.pre = static_cast<__nv_bfloat16 *>(pre);
  p.M = tokens; p.N = out; p.NZ = out * gated(act);
  switch (act) {
    case ULY_ACT_GELU: return linear_of<ULY_ACT_GELU>(x, w, p, in, workspace, stream);
    case ULY_ACT_SILU: return linear_of<ULY_ACT_SILU>(x, w, p, in, workspace, stream);
    case ULY_ACT_SWIGLU: return linear_of<ULY_ACT_SWIGLU>(x, w, p, in, workspace, stream);
    default: return linear_of<ULY_ACT_NONE>(x, w, p, in, workspace, stream);
  }
}

size_t linear_bwd_workspace_bytes(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  return bwd_plan(tokens, in, out, act).bytes;
}

uly_status linear_bwd_launch(int64_t tokens, int32_t in, int32_t out, int32_t act, const void *x, const void *w,
                             const void *pre, const void *dy, void *dx, void *dw, int32_t dw_dtype, float *dbias,
                             void *workspace, cudaStream_t stream) {
  const BwdPlan q = bwd_plan(tokens, in, out, act);
  char *ws = static_cast<char *>(workspace);
  float *bias_part = reinterpret_cast<float *>(ws + q.off_bias), *part = reinterpret_cast<float *>(ws + q.off_part);
  const void *dz = act == ULY_ACT_NONE ? dy : workspace;
  if (dbias || (act != ULY_ACT_NONE && (dx || dw))) {
    DzParams p = {};
    p.pre = static_cast<const __nv_bfloat16 *>(pre);
    p.dy = static_cast<const __nv_bfloat16 *>(dy);
    p.dz = static_cast<__nv_bfloat16 *>(workspace);
    // few tokens' sums by one CTA of rows: no partials, no second launch
    const int row_ctas = dbias && tokens <= kOneCtaRows ? 1 : q.row_ctas;
    p.part = !dbias ? nullptr : row_ctas == 1 ? dbias : bias_part;
    p.M = tokens; p.N = out; p.NZ = q.nz; p.ld = q.ld;
    p.rows_per_cta = (int)((tokens + row_ctas - 1) / row_ctas);
    const dim3 grid((out / 8 + 31) / 32, row_ctas);
    prof::Scope scope(prof::K_LINEAR_DZ, stream);
    switch (act) {
      case ULY_ACT_GELU: linear_dz_kernel<ULY_ACT_GELU><<<grid, 256, 0, stream>>>(p); break;
      case ULY_ACT_SILU: linear_dz_kernel<ULY_ACT_SILU><<<grid, 256, 0, stream>>>(p); break;
      case ULY_ACT_SWIGLU: linear_dz_kernel<ULY_ACT_SWIGLU><<<grid, 256, 0, stream>>>(p); break;
      default: linear_dz_kernel<ULY_ACT_NONE><<<grid, 256, 0, stream>>>(p);
    }
    note_launches(1);
    scope.end();
    if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
    if (dbias && row_ctas > 1) {
      const uly_status st = fold_columns_launch(bias_part, 1, row_ctas, q.nz, dbias, stream);
      if (st != ULY_OK) return st;
    }
  }
  CUtensorMap ta, tb;
  if (dx && skinny::faster(tokens, in, q.nz, q.part)) {   // dx[tokens][in] = dz[tokens][nz] W[nz][in]
    const uly_status st = skinny::launch_plain_mn(dz, q.ld, w, dx, nullptr, tokens, in, q.nz, prof::K_LINEAR_DX, stream);
    if (st != ULY_OK) return st;
  } else if (dx) {
    if (!make_map(&ta, dz, q.nz, tokens, q.ld, kHalf) || !make_map(&tb, w, in, q.nz, in, 64)) return ULY_ERR_CUDA;
    PlainParams p = {};
    p.out = dx; p.M = tokens; p.N = in;
    const uly_status st = launch_plain<false>(ta, tb, p, q.nz, part, q.part, prof::K_LINEAR_DX, stream);
    if (st != ULY_OK) return st;
  }
  if (dw) {   // dW[nz][in] = dz^T x
    if (!make_map(&ta, dz, q.nz, tokens, q.ld, 64) || !make_map(&tb, x, in, tokens, in, 64)) return ULY_ERR_CUDA;
    PlainParams p = {};
    p.out = dw; p.out_f32 = dw_dtype == ULY_F32; p.M = q.nz; p.N = in;
    return launch_plain<true>(ta, tb, p, tokens, part, q.part, prof::K_LINEAR_DW, stream);
  }
  return ULY_OK;
}

}  // namespace uly
