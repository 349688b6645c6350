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
  const __nv_bfloat16 *bias, *residual;   // nullable
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
    add_bias(p, col, z, up);
    if (p.pre) {
      store8(p.pre + row * p.NZ + col, z);
      if (kGated) store8(p.pre + row * p.NZ + p.N + col, up);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = act_of<ACT>(z[e], up[e]);
    if (p.residual) {
      float r[8];
      load8(p.residual + row * p.N + col, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] += r[e];
    }
    store8(p.y + row * p.N + col, z);
  }

  // A row's next 32 columns of the residual: asked for a turn of the loop ahead.
  struct Ahead {
    uint4 v[4];
    __device__ __forceinline__ void load(const Params &p, int row, int col, bool ok) {
      if (p.residual && ok)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (col + 8 * g < p.N) v[g] = __ldg(reinterpret_cast<const uint4 *>(p.residual + (long long)row * p.N + col) + g);
    }
    __device__ __forceinline__ void add(const Params &p, int g, float (&z)[8]) const {
      if (!p.residual) return;
      const uint32_t w[4] = {v[g].x, v[g].y, v[g].z, v[g].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[2 * e] += __uint_as_float(w[e] << 16);
        z[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  };

  template <int TN>
  static constexpr bool kWide = TN / (kGated ? 4 : 2) % 64 == 0;   // y_map's boxes, without pre

  template <int TN>
  static __device__ __forceinline__ void tile(const Params &p, const Unit &w, uint32_t acc, int row, int half,
                                              OutRing &out) {
    constexpr int cols = kGated ? TN / 4 : TN / 2;   // output columns of one warpgroup
    const bool ok = row < p.M;
    const int row0 = row - out.lane, first = w.nt * 2 * cols + half * cols;
    Ahead next = {};
    next.load(p, row, first, ok);
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
      const int c0 = half * cols + c, col0 = first + c;
      uint32_t a[kGated ? 64 : 32];
      if constexpr (kGated) tmem_ld32x2(acc + c0, acc + TN / 2 + c0, a);
      else tmem_ld32(acc + c0, a);
      if (col0 >= p.N || row0 >= p.M) continue;   // the whole warp
      const Ahead res = next;
      if (c + 32 < cols) next.load(p, row, col0 + 32, ok);
      uint32_t vy[16], vz[16], vu[kGated ? 16 : 1];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = col0 + 8 * g;
        float z[8], up[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[e] = __uint_as_float(a[8 * g + e]);
          up[e] = kGated ? __uint_as_float(a[(kGated ? 32 : 0) + 8 * g + e]) : 0.f;
        }
        if (col < p.N) add_bias(p, col, z, up);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          vz[4 * g + e] = pack_bf16x2(z[2 * e], z[2 * e + 1]);
          if constexpr (kGated) vu[4 * g + e] = pack_bf16x2(up[2 * e], up[2 * e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = act_of<ACT>(z[e], up[e]);
        res.add(p, g, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) vy[4 * g + e] = pack_bf16x2(z[2 * e], z[2 * e + 1]);
      }
      __syncwarp();
      if (kWide<TN> && !p.pre) {   // two steps a store
        const int h = c >> 5 & 1;
        if (h == 0) out.begin();
        out.write_wide(h, vy);
        if (h == 1 || col0 + 32 >= p.N) out.end_wide(&p.y_map, col0 - 32 * h, row0);
        continue;
      }
      out.begin();
      out.write(0, vy);
      if (p.pre) out.write(1, vz);
      out.end(&p.y_map, col0, p.pre ? &p.pre_map : nullptr, col0, row0);
      if constexpr (kGated) {
        if (p.pre) {
          out.begin();
          out.write(0, vu);
          out.end(&p.up_map, col0, nullptr, 0, row0);
        }
      }
    }
  }
};

// Few tokens: this CTA's slice of a tile's features, four of a token a thread.
template <int ACT>
struct SkinnyLinear {
  using Params = LinearParams;
  static constexpr bool kGated = ACT == ULY_ACT_SWIGLU;
  static constexpr int kCols = kGated ? 64 : 128;
  static __device__ __forceinline__ void finish(const Params &p, const skinny::Tile &tile, int index, int rank,
                                                int ranks) {
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
        skinny::load4(p.residual + (long long)t * p.N + col, b);
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
  const bool wide = !p.pre && (cut.tn == kTile ? Epi::template kWide<kTile> : Epi::template kWide<kNarrow>);
  CUtensorMap ta, tb;
  if (!make_map(&ta, x, K, p.M, K, kHalf) || !make_map(&tb, w, K, p.NZ, K, b_box(cut)) ||
      !(wide ? make_wide_map : make_out_map)(&p.y_map, p.y, p.N, p.M, p.N, false) || (p.pre && !make_out_map(&p.pre_map, p.pre, p.N, p.M, p.NZ)) ||
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
  float *part;                     // [gridDim.y * 8][NZ]; null without a bias gradient
  long long M;
  int N, NZ, rows_per_cta;
};

template <int ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const DzParams p) {
  constexpr bool kGated = ACT == ULY_ACT_SWIGLU;
  const int strip = threadIdx.x >> 5, col = (blockIdx.x * 32 + (threadIdx.x & 31)) * 8;
  if (col >= p.N) return;
  float s0[8] = {}, s1[8] = {};
  const long long r0 = (long long)blockIdx.y * p.rows_per_cta;
  const long long r1 = r0 + p.rows_per_cta < p.M ? r0 + p.rows_per_cta : p.M;
#pragma unroll 2
  for (long long r = r0 + strip; r < r1; r += 8) {
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
      store8(p.dz + r * p.NZ + col, a);
      store8(p.dz + r * p.NZ + p.N + col, b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= dact_of<ACT>(z[e]);
        s0[e] += d[e];
      }
      store8(p.dz + r * p.NZ + col, d);
    }
  }
  if (p.part) {
    float *o = p.part + ((long long)blockIdx.y * 8 + strip) * p.NZ + col;
    store8(o, s0);
    if (kGated) store8(o + p.N, s1);
  }
}

// CTAs along the tokens: about eight an SM in all, no shorter than 64 rows.
int dz_row_ctas(int64_t tokens, int32_t out) {
  const long long cols = (out / 8 + 31) / 32;
  long long ctas = (long long)device_sm_count() * 8 / cols, most = (tokens + 63) / 64;
  if (ctas > most) ctas = most;
  return (int)(ctas < 1 ? 1 : ctas);
}

// Workspace of the backward: dz, the bias gradient's partials, a cut product's
// partials (the two products run one after the other and share them).
struct BwdPlan {
  int nz, row_ctas;
  size_t off_bias, off_part, part, bytes;
};
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
BwdPlan bwd_plan(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  BwdPlan q;
  q.nz = out * gated(act);
  q.row_ctas = dz_row_ctas(tokens, out);
  q.off_bias = act == ULY_ACT_NONE ? 0 : up256((size_t)tokens * q.nz * 2);
  q.off_part = q.off_bias + up256((size_t)q.row_ctas * 8 * q.nz * sizeof(float));
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
    p.part = dbias ? bias_part : nullptr;
    p.M = tokens; p.N = out; p.NZ = q.nz;
    p.rows_per_cta = (int)((tokens + q.row_ctas - 1) / q.row_ctas);
    const dim3 grid((out / 8 + 31) / 32, q.row_ctas);
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
    if (dbias) {
      const uly_status st = fold_columns_launch(bias_part, 1, (long long)q.row_ctas * 8, q.nz, dbias, stream);
      if (st != ULY_OK) return st;
    }
  }
  CUtensorMap ta, tb;
  if (dx && skinny::faster(tokens, in, q.nz, q.part)) {   // dx[tokens][in] = dz[tokens][nz] W[nz][in]
    const uly_status st = skinny::launch_plain_mn(dz, q.nz, w, dx, nullptr, tokens, in, q.nz, prof::K_LINEAR_DX, stream);
    if (st != ULY_OK) return st;
  } else if (dx) {
    if (!make_map(&ta, dz, q.nz, tokens, q.nz, kHalf) || !make_map(&tb, w, in, q.nz, in, 64)) return ULY_ERR_CUDA;
    PlainParams p = {};
    p.out = dx; p.M = tokens; p.N = in;
    const uly_status st = launch_plain<false>(ta, tb, p, q.nz, part, q.part, prof::K_LINEAR_DX, stream);
    if (st != ULY_OK) return st;
  }
  if (dw) {   // dW[nz][in] = dz^T x
    if (!make_map(&ta, dz, q.nz, tokens, q.nz, 64) || !make_map(&tb, x, in, tokens, in, 64)) return ULY_ERR_CUDA;
    PlainParams p = {};
    p.out = dw; p.out_f32 = dw_dtype == ULY_F32; p.M = q.nz; p.N = in;
    return launch_plain<true>(ta, tb, p, tokens, part, q.part, prof::K_LINEAR_DW, stream);
  }
  return ULY_OK;
}

}  // namespace uly
