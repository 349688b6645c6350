// Norms around a residual branch, fused with its gate and the residual
// stream's scale (the token-wise step between two blocks of a layer; every
// logical rank's tokens are independent, so the seq layout is walked as rows):
//
//   N(v; w)_j = w_j v_j / sqrt(mean_j v_j^2 + eps)
//   r = res_scale x + gate * N(h; w_post)        u = N(r; w_pre)
//
// One row per group of threads, one 16-byte vector of it per thread (rows over
// 512 vectors: several), so every tensor is read once and written once: bound
// by memory traffic.  Sums are fp32; u is taken from the fp32 r, and r and u
// are rounded once.
//
// Backward, from the stored r (its own sum of squares is formed again beside
// the other row sum, so no statistics are kept between the passes).  With
// rn = r / rms(r), hn = h / rms(h), a = du * w_pre:
//   dR = dr + (a - rn mean(a rn)) / rms(r)       dx = res_scale dR
//   dw_pre = sum_t du rn                         dN = gate dR
//   dgate = sum dR N(h)   (over what the gate is broadcast along)
//   b = dN * w_post, dh = (b - hn mean(b hn)) / rms(h),  dw_post = sum_t dN hn
// The column sums stay in fp32 registers over all rows of a CTA; each CTA
// writes one partial per column and a second kernel folds the partials in a
// fixed order, so every output is bitwise repeatable.
#include "common.cuh"
#include "prof.cuh"
#include "tokenwise.cuh"

namespace uly {

namespace {

template <typename T>
struct Vec;   // one 16-byte vector
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(h[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    return u;
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

constexpr int kMaxGroup = 512;   // threads of one row
constexpr int kMaxVecs = 8;      // vectors of one thread

// Sums of K values over the threads of each group (group g = threads
// [g*tpr, (g+1)*tpr), tpr a multiple of 32); every thread gets its group's.
// Two buffers taken in turn, so one barrier a call is enough.
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int tpr, float (*sh)[K], int &turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, wpg = tpr >> 5, first = warp / wpg * wpg;
  float (*buf)[K] = sh + 32 * turn;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < wpg; ++w)   // fixed order, the same in every thread
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += buf[first + w][k];
}

struct NormParams {
  const void *x, *h, *gate, *w_post, *w_pre;
  void *r, *u;
  long long rows;
  int vecs, tpr, gate_mode, B, s;
  float res_scale, eps, inv_d;
};

// Row of the gate that token `t` of the seq layout uses.
__device__ __forceinline__ long long gate_row(int mode, long long t, int B, int s) {
  return mode == ULY_GATE_TOKEN ? t : mode == ULY_GATE_SEQUENCE ? (t / s) % B : 0;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kMaxGroup) residual_norm_kernel(const NormParams p) {
  constexpr int E = Vec<T>::N;
  __shared__ float sh[64][1];
  int turn = 0;
  const int grp = threadIdx.x / p.tpr, l = threadIdx.x - grp * p.tpr, rpb = blockDim.x / p.tpr;
  for (long long t0 = (long long)blockIdx.x * rpb; t0 < p.rows; t0 += (long long)gridDim.x * rpb) {
    const long long t = t0 + grp;
    const bool row_ok = t < p.rows;
    const long long base = t * p.vecs;
    const long long gbase = row_ok ? gate_row(p.gate_mode, t, p.B, p.s) * p.vecs : 0;
    uint4 xv[NV], hv[NV], gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * p.tpr;
      const bool ok = row_ok && v < p.vecs;
      xv[i] = ok ? __ldcs(static_cast<const uint4 *>(p.x) + base + v) : make_uint4(0, 0, 0, 0);
      hv[i] = ok && p.h ? __ldcs(static_cast<const uint4 *>(p.h) + base + v) : make_uint4(0, 0, 0, 0);
      if (p.gate_mode != ULY_GATE_NONE)
        gv[i] = ok ? __ldg(static_cast<const uint4 *>(p.gate) + gbase + v) : make_uint4(0, 0, 0, 0);
    }
    float hscale = 1.f;
    if (p.w_post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float h[E];
        Vec<T>::unpack(hv[i], h);
#pragma unroll
        for (int e = 0; e < E; ++e) ss[0] = fmaf(h[e], h[e], ss[0]);
      }
      group_sum<1>(ss, p.tpr, sh, turn);
      hscale = rsqrtf(ss[0] * p.inv_d + p.eps);
    }
    float r[NV][E];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * p.tpr;
      float h[E], x[E];
      Vec<T>::unpack(hv[i], h);
      Vec<T>::unpack(xv[i], x);
      if (p.w_post && v < p.vecs) {
        float w[E];
        Vec<T>::unpack(__ldg(static_cast<const uint4 *>(p.w_post) + v), w);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] *= hscale * w[e];
      }
      if (p.gate_mode != ULY_GATE_NONE) {
        float g[E];
        Vec<T>::unpack(gv[i], g);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[i][e] = p.h ? fmaf(p.res_scale, x[e], h[e]) : p.res_scale * x[e];
        ss[0] = fmaf(r[i][e], r[i][e], ss[0]);
      }
      if (p.r && row_ok && v < p.vecs) static_cast<uint4 *>(p.r)[base + v] = Vec<T>::pack(r[i]);
    }
    if (!p.u) continue;
    group_sum<1>(ss, p.tpr, sh, turn);
    const float rscale = rsqrtf(ss[0] * p.inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * p.tpr;
      if (!row_ok || v >= p.vecs) continue;
      float w[E], u[E];
      Vec<T>::unpack(__ldg(static_cast<const uint4 *>(p.w_pre) + v), w);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = r[i][e] * rscale * w[e];
      static_cast<uint4 *>(p.u)[base + v] = Vec<T>::pack(u);
    }
  }
}

struct NormBwdParams {
  const void *r, *h, *dr, *du, *gate, *w_post, *w_pre;
  void *dx, *dh, *dgate_tok;
  float *part_pre, *part_post;   // [groups of all CTAs][vecs * E]; null where not asked for
  float *part_gate;              // [units][groups of a CTA][vecs * E]
  long long rows_per_b;          // tokens of one gate row (P * s, or all of them)
  int vecs, tpr, gate_mode, B, s, bs;   // bs = gate rows that units walk (B for sequence gates, else 1)
  int upb;                       // units (runs of tokens) per gate row
  float res_scale, eps, inv_d;
};

template <typename T, int NV>
__global__ void __launch_bounds__(kMaxGroup) residual_norm_bwd_kernel(const NormBwdParams p) {
  constexpr int E = Vec<T>::N;
  __shared__ float sh3[64][3], sh1[64][1];
  int turn3 = 0, turn1 = 0;
  const int grp = threadIdx.x / p.tpr, l = threadIdx.x - grp * p.tpr, rpb = blockDim.x / p.tpr;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float a_pre[NV][E] = {}, a_post[NV][E] = {}, a_gate[NV][E] = {};
  const int units = p.bs * p.upb;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int b = unit / p.upb, part = unit - b * p.upb;
    const long long q0 = p.rows_per_b * part / p.upb, q1 = p.rows_per_b * (part + 1) / p.upb;
    for (long long q = q0; q < q1; q += rpb) {
      const bool row_ok = q + grp < q1;
      long long t = row_ok ? q + grp : q;
      if (p.bs > 1) {   // token q of sequence b: rank q / s, position q % s
        const long long rk = t / p.s;
        t = (rk * p.B + b) * p.s + (t - rk * p.s);
      }
      const long long base = t * p.vecs;
      const long long gbase = gate_row(p.gate_mode, t, p.B, p.s) * p.vecs;
      uint4 rv[NV], hv[NV], dv[NV], uv[NV], gv[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = l + i * p.tpr;
        const bool ok = row_ok && v < p.vecs;
        rv[i] = ok && p.r ? __ldcs(static_cast<const uint4 *>(p.r) + base + v) : zero;
        uv[i] = ok && p.du ? __ldcs(static_cast<const uint4 *>(p.du) + base + v) : zero;
        hv[i] = ok && p.h ? __ldcs(static_cast<const uint4 *>(p.h) + base + v) : zero;
        dv[i] = ok && p.dr ? __ldcs(static_cast<const uint4 *>(p.dr) + base + v) : zero;
        if (p.gate_mode != ULY_GATE_NONE) gv[i] = ok ? __ldg(static_cast<const uint4 *>(p.gate) + gbase + v) : zero;
      }
      // sums of r^2, du w_pre r and h^2 together
      float s3[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = l + i * p.tpr;
        float r[E], h[E];
        Vec<T>::unpack(rv[i], r);
        Vec<T>::unpack(hv[i], h);
#pragma unroll
        for (int e = 0; e < E; ++e) s3[2] = fmaf(h[e], h[e], s3[2]);
        if (p.du && v < p.vecs) {
          float u[E], w[E];
          Vec<T>::unpack(uv[i], u);
          Vec<T>::unpack(__ldg(static_cast<const uint4 *>(p.w_pre) + v), w);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            s3[0] = fmaf(r[e], r[e], s3[0]);
            s3[1] = fmaf(u[e] * w[e], r[e], s3[1]);
          }
        }
      }
      group_sum<3>(s3, p.tpr, sh3, turn3);
      const float ir = rsqrtf(s3[0] * p.inv_d + p.eps);
      const float c1 = s3[1] * ir * ir * p.inv_d;      // mean(a rn) / rms(r), so that a rn-term is c1 * r
      const float ih = p.w_post ? rsqrtf(s3[2] * p.inv_d + p.eps) : 1.f;
      float s1[1] = {0.f};
      float dn[NV][E];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = l + i * p.tpr;
        const bool ok = row_ok && v < p.vecs;
        float r[E], d[E], h[E], w[E];
        Vec<T>::unpack(dv[i], d);
        if (p.du && v < p.vecs) {
          float u[E];
          Vec<T>::unpack(rv[i], r);
          Vec<T>::unpack(uv[i], u);
          Vec<T>::unpack(__ldg(static_cast<const uint4 *>(p.w_pre) + v), w);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            d[e] += ir * (u[e] * w[e] - c1 * r[e]);
            if (ok) a_pre[i][e] = fmaf(u[e] * ir, r[e], a_pre[i][e]);
          }
        }
        if (p.dx && ok) {
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = p.res_scale * d[e];
          static_cast<uint4 *>(p.dx)[base + v] = Vec<T>::pack(o);
        }
        Vec<T>::unpack(hv[i], h);
        if (p.w_post && v < p.vecs) {
          Vec<T>::unpack(__ldg(static_cast<const uint4 *>(p.w_post) + v), w);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) w[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) dn[i][e] = d[e];
        if (p.gate_mode != ULY_GATE_NONE) {
          float g[E], o[E];
          Vec<T>::unpack(gv[i], g);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            o[e] = d[e] * (h[e] * ih * w[e]);   // dR N(h)
            dn[i][e] = d[e] * g[e];
          }
          if (p.gate_mode == ULY_GATE_TOKEN) {
            if (p.dgate_tok && ok) static_cast<uint4 *>(p.dgate_tok)[base + v] = Vec<T>::pack(o);
          } else if (ok) {
#pragma unroll
            for (int e = 0; e < E; ++e) a_gate[i][e] += o[e];
          }
        }
        if (p.w_post && ok) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float hn = h[e] * ih;
            a_post[i][e] = fmaf(dn[i][e], hn, a_post[i][e]);
            dn[i][e] *= w[e];
            s1[0] = fmaf(dn[i][e], hn, s1[0]);
          }
        }
      }
      if (!p.dh) continue;
      float c2 = 0.f;
      if (p.w_post) {
        group_sum<1>(s1, p.tpr, sh1, turn1);
        c2 = s1[0] * p.inv_d;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = l + i * p.tpr;
        if (!row_ok || v >= p.vecs) continue;
        float h[E], o[E];
        Vec<T>::unpack(hv[i], h);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = p.w_post ? ih * (dn[i][e] - c2 * (h[e] * ih)) : dn[i][e];
        static_cast<uint4 *>(p.dh)[base + v] = Vec<T>::pack(o);
      }
    }
    if (p.part_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = l + i * p.tpr;
        if (v < p.vecs) {
          float *o = p.part_gate + (((long long)unit * rpb + grp) * p.vecs + v) * E;
#pragma unroll
          for (int e = 0; e < E; ++e) { o[e] = a_gate[i][e]; a_gate[i][e] = 0.f; }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = l + i * p.tpr;
    if (v >= p.vecs) continue;
    const long long at = (((long long)blockIdx.x * rpb + grp) * p.vecs + v) * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (p.part_pre) p.part_pre[at + e] = a_pre[i][e];
      if (p.part_post) p.part_post[at + e] = a_post[i][e];
    }
  }
}

// Threads of a row, vectors of a thread and rows of a CTA for rows of `vecs`
// vectors: one vector a thread up to 512 (2560 bf16: 320 threads), CTAs of
// about 256 threads or one row.
struct RowShape {
  int tpr, nv, rpb;
};
RowShape row_shape(int vecs) {
  RowShape r;
  r.nv = (vecs + kMaxGroup - 1) / kMaxGroup;
  const int per = (vecs + r.nv - 1) / r.nv;
  r.tpr = (per + 31) / 32 * 32;
  r.rpb = r.tpr >= 256 ? 1 : 256 / r.tpr;
  return r;
}

template <typename T>
using FwdKernel = void (*)(NormParams);
template <typename T>
FwdKernel<T> fwd_kernel(int nv) {
  switch (nv) {
    case 1: return residual_norm_kernel<T, 1>;
    case 2: return residual_norm_kernel<T, 2>;
    case 3: case 4: return residual_norm_kernel<T, 4>;
    default: return residual_norm_kernel<T, 8>;
  }
}
using BwdKernel = void (*)(NormBwdParams);
template <typename T>
BwdKernel bwd_kernel(int nv) {
  switch (nv) {
    case 1: return residual_norm_bwd_kernel<T, 1>;
    case 2: return residual_norm_bwd_kernel<T, 2>;
    case 3: case 4: return residual_norm_bwd_kernel<T, 4>;
    default: return residual_norm_bwd_kernel<T, 8>;
  }
}

// How the backward walks the tokens: `bs` gate rows, each cut into `upb` runs
// of tokens, on `grid` CTAs.  About four CTAs an SM keep enough loads in
// flight; the runs are no shorter than a CTA's rows.
struct BwdPlan {
  RowShape rs;
  int bs, upb, grid;
  size_t off_pre, off_post, off_gate, bytes;
};
BwdPlan bwd_plan(int B, long long n, int vecs, int E, int gate_mode, bool pre, bool post, bool gate) {
  BwdPlan q;
  q.rs = row_shape(vecs);
  q.bs = gate_mode == ULY_GATE_SEQUENCE ? B : 1;
  const long long rows = gate_mode == ULY_GATE_SEQUENCE ? n : (long long)B * n;
  const int per_sm = q.rs.tpr * q.rs.rpb <= 320 ? 4 : 2;
  const long long want = (long long)device_sm_count() * per_sm;
  long long upb = want / q.bs, most = (rows + q.rs.rpb - 1) / q.rs.rpb;
  if (upb < 1) upb = 1;
  if (upb > most) upb = most;
  q.upb = (int)upb;
  const long long units = (long long)q.bs * q.upb;
  q.grid = (int)(units < want ? units : want);
  const size_t col = (size_t)vecs * E * sizeof(float) * q.rs.rpb;
  q.off_pre = 0;
  q.off_post = q.off_pre + (pre ? col * q.grid : 0);
  q.off_gate = q.off_post + (post ? col * q.grid : 0);
  q.bytes = q.off_gate + (gate && (gate_mode == ULY_GATE_CHANNEL || gate_mode == ULY_GATE_SEQUENCE) ? col * units : 0);
  return q;
}

}  // namespace

// dst[k][c] = sum over i < parts of src[k][i][c], in a fixed order: 32 columns
// a CTA, 8 strips of partials folded through shared memory.
__global__ void __launch_bounds__(256) fold_columns_kernel(const float *__restrict__ src, long long parts, int cols,
                                                           float *__restrict__ dst) {
  __shared__ float sh[8][33];
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float *s = src + (long long)blockIdx.y * parts * cols;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < cols) {
    long long i = strip;
    for (; i + 24 < parts; i += 32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] += __ldcs(s + (i + 8 * k) * cols + c);
    }
    for (int k = 0; i < parts; i += 8, ++k) a[k & 3] += __ldcs(s + i * cols + c);
  }
  sh[strip][lane] = (a[0] + a[1]) + (a[2] + a[3]);
  __syncthreads();
  if (strip == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += sh[k][lane];
    dst[(long long)blockIdx.y * cols + c] = v;
  }
}

uly_status fold_columns_launch(const float *src, int rows, long long parts, int cols, float *dst,
                               cudaStream_t stream) {
  prof::Scope scope(prof::K_FOLD_COLUMNS, stream);
  for (int r0 = 0; r0 < rows; r0 += 65535) {
    const int n = rows - r0 < 65535 ? rows - r0 : 65535;
    fold_columns_kernel<<<dim3((cols + 31) / 32, n), 256, 0, stream>>>(src + (long long)r0 * parts * cols, parts,
                                                                      cols, dst + (long long)r0 * cols);
    note_launches(1);
  }
  return last_launch_status();
}

bool residual_norm_supported(int vecs) { return vecs <= kMaxGroup * kMaxVecs; }

uly_status residual_norm_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *x,
                                const void *h, const void *gate, int32_t gate_mode, const void *w_post,
                                const void *w_pre, float res_scale, float eps, void *r, void *u,
                                cudaStream_t stream) {
  NormParams p = {};
  p.x = x; p.h = h; p.gate = gate; p.w_post = w_post; p.w_pre = w_pre; p.r = r; p.u = u;
  p.rows = (long long)B * n;
  p.vecs = hidden * (dtype == ULY_BF16 ? 2 : 4) / 16;
  p.gate_mode = gate_mode; p.B = B; p.s = n / P;
  p.res_scale = res_scale; p.eps = eps; p.inv_d = 1.0f / hidden;
  const RowShape rs = row_shape(p.vecs);
  p.tpr = rs.tpr;
  long long blocks = (p.rows + rs.rpb - 1) / rs.rpb;
  if (blocks > (1LL << 30)) blocks = 1LL << 30;
  prof::Scope scope(prof::K_RESIDUAL_NORM, stream);
  if (dtype == ULY_BF16)
    fwd_kernel<__nv_bfloat16>(rs.nv)<<<(unsigned)blocks, rs.tpr * rs.rpb, 0, stream>>>(p);
  else
    fwd_kernel<float>(rs.nv)<<<(unsigned)blocks, rs.tpr * rs.rpb, 0, stream>>>(p);
  note_launches(1);
  return last_launch_status();
}

size_t residual_norm_bwd_workspace_bytes(int32_t B, int32_t n, int32_t hidden, int32_t dtype, int32_t gate_mode) {
  const int e = dtype == ULY_BF16 ? 8 : 4;
  return bwd_plan(B, n, hidden / e, e, gate_mode, true, true, true).bytes;
}

uly_status residual_norm_bwd_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *r,
                                    const void *h, const void *dr, const void *du, const void *gate,
                                    int32_t gate_mode, const void *w_post, const void *w_pre, float res_scale,
                                    float eps, void *dx, void *dh, float *dw_post, float *dw_pre, void *dgate,
                                    void *workspace, cudaStream_t stream) {
  const int E = dtype == ULY_BF16 ? 8 : 4, vecs = hidden / E;
  const bool shared_gate = gate_mode == ULY_GATE_CHANNEL || gate_mode == ULY_GATE_SEQUENCE;
  const BwdPlan q = bwd_plan(B, n, vecs, E, gate_mode, dw_pre != nullptr, dw_post != nullptr, dgate != nullptr);
  char *ws = static_cast<char *>(workspace);
  NormBwdParams p = {};
  p.r = r; p.h = h; p.dr = dr; p.du = du; p.gate = gate; p.w_post = w_post; p.w_pre = w_pre;
  p.dx = dx; p.dh = dh;
  p.dgate_tok = gate_mode == ULY_GATE_TOKEN ? dgate : nullptr;
  p.part_pre = dw_pre ? reinterpret_cast<float *>(ws + q.off_pre) : nullptr;
  p.part_post = dw_post ? reinterpret_cast<float *>(ws + q.off_post) : nullptr;
  p.part_gate = shared_gate && dgate ? reinterpret_cast<float *>(ws + q.off_gate) : nullptr;
  p.rows_per_b = q.bs > 1 ? n : (long long)B * n;
  p.vecs = vecs; p.tpr = q.rs.tpr; p.gate_mode = gate_mode; p.B = B; p.s = n / P;
  p.bs = q.bs; p.upb = q.upb;
  p.res_scale = res_scale; p.eps = eps; p.inv_d = 1.0f / hidden;
  {
    prof::Scope scope(prof::K_RESIDUAL_NORM_BWD, stream);
    const int threads = q.rs.tpr * q.rs.rpb;
    if (dtype == ULY_BF16) bwd_kernel<__nv_bfloat16>(q.rs.nv)<<<q.grid, threads, 0, stream>>>(p);
    else bwd_kernel<float>(q.rs.nv)<<<q.grid, threads, 0, stream>>>(p);
    note_launches(1);
    if (last_launch_status() != ULY_OK) return ULY_ERR_CUDA;
  }
  uly_status st = ULY_OK;
  const long long parts = (long long)q.grid * q.rs.rpb;
  if (dw_pre) st = fold_columns_launch(p.part_pre, 1, parts, hidden, dw_pre, stream);
  if (st == ULY_OK && dw_post) st = fold_columns_launch(p.part_post, 1, parts, hidden, dw_post, stream);
  if (st == ULY_OK && p.part_gate)
    st = fold_columns_launch(p.part_gate, q.bs, (long long)q.upb * q.rs.rpb, hidden, static_cast<float *>(dgate),
                             stream);
  return st;
}

}  // namespace uly
