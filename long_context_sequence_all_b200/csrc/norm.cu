// Norms around a residual branch, fused with its gate and the residual
// stream's scale (the token-wise step between two blocks of a layer; every
// logical rank's tokens are independent, so the seq layout is walked as rows):
//
//   N(v; w)_j = w_j v_j / sqrt(mean_j v_j^2 + eps)
//   r = res_scale x + gate * N(h; w_post)        u = N(r; w_pre)
//
// Every tensor is read once and written once; bound by memory traffic.  Sums
// are fp32; u is taken from the fp32 r, and r and u are rounded once.
//
// Backward, from the stored r (its own sum of squares is formed again beside
// the other row sum, so no statistics are kept between the passes).  With
// rn = r / rms(r), hn = h / rms(h), a = du * w_pre:
//   dR = dr + (a - rn mean(a rn)) / rms(r)       dx = res_scale dR
//   dw_pre = sum_t du rn                         dN = gate dR
//   dgate = sum dR N(h)   (over what the gate is broadcast along)
//   b = dN * w_post, dh = (b - hn mean(b hn)) / rms(h),  dw_post = sum_t dN hn
// A gate shared by the tokens of a run is a factor of that run's sums, so with
// A = sum_t dR hn over the run, dw_post = sum gate A and dgate = w_post A: two
// column sums (A and dw_pre's) stay in fp32 registers over all rows of a group.
// A CTA's groups add theirs in shared memory and write one partial per column and
// run, and a second kernel folds the partials, all in a fixed order, so every
// output is bitwise repeatable.
//
// How: persistent teams of a warp or of several.  A team's rows arrive by bulk
// copies in a ring of shared-memory stages, so the loads run ahead of the two row
// sums (each a barrier of the team).  The CTA's teams share the weights, and a
// gate that all tokens share, in shared memory (where two stages fit beside them):
// from L1, which the streams keep emptying, their latency was the forward's
// largest stall.  A thread takes up to five 16-byte vectors of a
// row (backward: two, its column sums take the registers; up to four of the rows of
// more than 1024 vectors, which 512 threads share).  Short rows share a
// warp, a power of two of lanes each, and arrive several at a time (253074 x 160:
// 142 us with one row a warp, 65 us so); of long ones few warps share a row: at
// 2560 bf16 columns two warps (backward: five) instead of ten, which had left both
// directions waiting for barriers and shuffles at 3.2 and 2.6 TB/s.  Arithmetic
// runs on pairs of fp32 values.
// 65536 x 2560 bf16 with a channel gate: forward 251 us (5.4 TB/s of its 1.34
// GB), backward 416 us (4.8 TB/s of 2.01 GB) + 9 us of folding.  The forward is
// near the memory's rate (a copy: 6.5 TB/s); the backward issues about 4100
// instructions a row and its two row sums, one after the other, leave their latency
// in the open (with a gate of every token it moves a third more in 460 us).
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "prof.cuh"
#include "sm100.cuh"
#include "tokenwise.cuh"

namespace uly {

namespace {

// Two fp32 values in one 64-bit register pair.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ float sum2(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

template <typename T>
struct Vec;   // one 16-byte vector as N pairs
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, F2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = f2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const F2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      split(x[e], lo, hi);
      w[e] = sm100::pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void unpack(const uint4 &u, F2 (&x)[2]) {
    x[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const F2 (&x)[2]) {
    float a, b, c, d;
    split(x[0], a, b);
    split(x[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
};

constexpr int kMaxLanes = 512;                 // threads of one row
constexpr int kMaxVecs = 2048;                 // vectors of one row (32 KB)
constexpr int kMaxTeams = 10;                  // teams of a CTA
constexpr int kWarpTeams = 4;                  // ... where a team is one warp
constexpr int kMaxStages = 4;
constexpr uint32_t kRingBytes = 200 * 1024;    // shared memory the stages (and weights) of an SM's CTAs may take

// Sums of K values over a row's threads: `lanes` of a warp (a power of two), or a
// team of several warps (then also a barrier of it: named barrier team + 1; two
// buffers taken in turn, so one barrier a call is enough).
template <bool WARP, bool STAGED>
__device__ __forceinline__ void team_barrier(int team, int lanes) {
  if (WARP) __syncwarp();
  else if (!STAGED) __syncthreads();   // the CTA's only team
  else sm100::named_bar_sync(team + 1, lanes);
}
template <int K, bool WARP, bool STAGED>
__device__ __forceinline__ void row_sum(float (&v)[K], int lanes, int team, float (*sh)[K], int &turn) {
  if (WARP) {
    for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    return;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  const int warp = threadIdx.x >> 5, warps = STAGED ? lanes >> 5 : blockDim.x >> 5, first = STAGED ? team * warps : 0;
  float (*buf)[K] = sh + 32 * turn;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
  team_barrier<WARP, STAGED>(team, lanes);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < warps; ++w)   // fixed order, the same in every thread
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += buf[first + w][k];
}

// Tensors whose rows a stage holds, one after the other.
struct RingSrc {
  const void *p[5];
  int n;
  void add(const void *q, int &slot) {
    slot = q ? n : -1;
    if (q) p[n++] = q;
  }
};

struct RingShape {
  int slots, stages;   // tensors of a stage, stages of a team
  int lanes;           // threads of a row: of a warp, or a whole team of warps
  int *err;
  long long wait_limit;
};

// Vectors that all rows share.
struct Shared3 {
  const uint4 *p[3];   // nullable
};

// A team's ring of stages, each of `rows` rows of every tensor, and this
// thread's place in it: thread `l` of `lanes` of row `sub` of a stage.
// STAGED: the vectors all rows share are brought into shared memory first.
template <bool WARP, bool STAGED>
struct Ring {
  uint8_t *base;
  uint64_t *bars;
  uint32_t row_bytes, slot_bytes, stage_bytes;
  int stages, at;        // at: the stage the next rows are taken from
  uint32_t phase;        // of `at`'s barrier
  volatile int *abort;   // a thread of the CTA has given up a wait
  int l, lanes, sub, rows;

  int team;
  uint8_t *mem;

  __device__ __forceinline__ Ring(uint8_t *smem, uint64_t *barriers, volatile int *abort_flag, int vecs, const RingShape &s,
                                  const Shared3 &all) {
    const int lane = threadIdx.x & 31;
    lanes = WARP || STAGED ? s.lanes : blockDim.x;
    team = WARP ? threadIdx.x >> 5 : STAGED ? threadIdx.x / s.lanes : 0;
    rows = WARP ? 32 / s.lanes : 1;
    l = WARP ? lane & (s.lanes - 1) : STAGED ? threadIdx.x - team * s.lanes : threadIdx.x;
    sub = WARP ? lane / s.lanes : 0;
    row_bytes = (uint32_t)vecs * 16;
    slot_bytes = row_bytes * rows;
    stage_bytes = slot_bytes * s.slots;
    stages = s.stages;
    mem = smem;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (STAGED && all.p[k]) share(k, all.p[k], vecs);
    base = first_stage() + (size_t)team * stages * stage_bytes;
    bars = barriers + team * kMaxStages;
    at = 0;
    phase = 0;
    abort = abort_flag;
    if (l == 0 && sub == 0)
      for (int i = 0; i < stages; ++i) sm100::mbar_init(sm100::smem_u32(&bars[i]), 1);
    if (threadIdx.x == 0) *abort = 0;
    sm100::fence_mbar_init();
    __syncthreads();
  }
  // The CTA: vector `k` of those that all rows share.
  __device__ __forceinline__ void share(int k, const uint4 *v, int vecs) const {
    for (int i = threadIdx.x; i < vecs; i += blockDim.x) reinterpret_cast<uint4 *>(mem + k * row_bytes)[i] = __ldg(v + i);
  }
  // the first team's stages, the others' behind them
  __device__ __forceinline__ uint8_t *first_stage() const { return mem + (STAGED ? 3 * row_bytes : 0); }
  // vector i * lanes + l of those that all rows share
  __device__ __forceinline__ uint4 common(const Shared3 &all, int k, int at) const {
    return STAGED ? reinterpret_cast<const uint4 *>(mem + k * row_bytes)[l + at] : __ldg(all.p[k] + l + at);
  }
  __device__ __forceinline__ void barrier() const { team_barrier<WARP, STAGED>(team, lanes); }
  __device__ __forceinline__ uint32_t slot(int st, int k) const {
    return sm100::smem_u32(base + st * stage_bytes + k * slot_bytes);
  }
  // The team: `n` rows of every tensor from token `t` on, into stage `st`.
  __device__ __forceinline__ void issue(const RingSrc &src, long long t, int n, int st) const {
    if (l != 0 || sub != 0 || *abort) return;
    const uint32_t bar = sm100::smem_u32(&bars[st]);
    sm100::mbar_arrive_expect_tx(bar, src.n * n * row_bytes);
    for (int k = 0; k < src.n; ++k)
      sm100::bulk_load(slot(st, k), static_cast<const uint8_t *>(src.p[k]) + t * row_bytes, n * row_bytes, bar);
  }
  // The same for rows that do not follow one another: `t` is this thread's row.
  __device__ __forceinline__ void issue_each(const RingSrc &src, long long t, int n, int st) const {
    if (WARP ? __any_sync(0xffffffffu, *abort) : *abort) return;   // all lanes or none
    const uint32_t bar = sm100::smem_u32(&bars[st]);
    if (l == 0 && sub == 0) sm100::mbar_arrive_expect_tx(bar, src.n * n * row_bytes);
    if (WARP) __syncwarp();
    if (l == 0 && sub < n)
      for (int k = 0; k < src.n; ++k)
        sm100::bulk_load(slot(st, k) + sub * row_bytes, static_cast<const uint8_t *>(src.p[k]) + t * row_bytes, row_bytes,
                         bar);
  }
  // Giving up raises the error.  The barriers of the team are met all the same, so
  // its rows are then computed from what is there, but nothing more is sent for: a
  // stage is only filled again by a thread that saw it full.
  __device__ __forceinline__ void wait(const RingShape &s) const {
    sm100::mbar_wait(sm100::smem_u32(&bars[at]), phase, abort, s.err, s.wait_limit);
  }
  // this thread's first vector of its row of tensor `k`
  __device__ __forceinline__ const uint4 *row(int k) const {
    return reinterpret_cast<const uint4 *>(base + at * stage_bytes + k * slot_bytes + sub * row_bytes) + l;
  }
  __device__ __forceinline__ void next() {
    if (++at == stages) { at = 0; phase ^= 1; }
  }
  // After a wait that gave up the copies may still be in flight: let them land
  // before the CTA's shared memory is given away.
  __device__ __forceinline__ void end() const {
    __syncthreads();
    if (!*abort) return;
    const long long t0 = clock64();
    while (clock64() - t0 < (1 << 20)) __nanosleep(1000);
  }
};

struct NormParams {
  RingSrc src;
  RingShape ring;
  int sx, sh, sg;   // stage slots of x, h and a token's gate (-1: none)
  Shared3 all;      // w_post, w_pre, a gate that all tokens share
  const uint4 *gate;
  uint4 *r, *u;
  int rows, vecs, gate_mode, B, s;
  float res_scale, eps, inv_d;
};

// Thread `l` of a row's `tpr` takes its vectors l, l + tpr, ...: NV of them, of
// which only the last can lie behind the row's end.
template <typename T, int NV, bool WARP, bool STAGED>
__global__ void __launch_bounds__(!WARP ? 640 : NV <= 2 ? 1024 : 512, 1) residual_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = Vec<T>::N;
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ uint64_t bars[kMaxTeams * kMaxStages];
  __shared__ int abort_flag;
  __shared__ float sh[2 * 32][1];
  int turn = 0;
  Ring<WARP, STAGED> ring(stage_mem, bars, &abort_flag, p.vecs, p.ring, p.all);
  const int l = ring.l, tpr = ring.lanes, rows = p.rows;
  const int teams = WARP ? kWarpTeams : STAGED ? blockDim.x / tpr : 1;
  const long long first = ((long long)blockIdx.x * teams + ring.team) * ring.rows;
  const long long step = (long long)gridDim.x * teams * ring.rows;
  const bool tail = l + (NV - 1) * tpr < p.vecs;   // this thread's last vector exists
  const bool branch = p.sh >= 0, post = p.all.p[0] != nullptr, gated = p.gate_mode != ULY_GATE_NONE;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto issue = [&](long long t, int st) {
    if (t < rows) ring.issue(p.src, t, (int)min((long long)ring.rows, rows - t), st);
  };
  for (int k = 0; k < ring.stages; ++k) issue(first + k * step, k);
  int done = -1;   // stage whose rows every thread has finished with, after the team's next barrier
  for (long long t0 = first; t0 < rows; t0 += step, ring.next()) {
    if (ring.stages == 1 && done >= 0) {   // no stage to run ahead into
      ring.barrier();
      issue(t0, 0);
    }
    ring.wait(p.ring);
    const long long t = t0 + ring.sub;
    const bool row_ok = !WARP || t < rows;
    const bool own_gate = p.sg >= 0, all_gate = p.gate_mode == ULY_GATE_CHANNEL;
    const uint4 *gv = p.gate + l;   // of this token's sequence
    if (p.gate_mode == ULY_GATE_SEQUENCE) gv += (long long)((int)t / p.s % p.B) * p.vecs;
    F2 r[NV][E], q = f2(0.f);
    if (branch) {
      const uint4 *hv = ring.row(p.sh);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Vec<T>::unpack(i < NV - 1 || tail ? hv[i * tpr] : zero, r[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) q = fma(r[i][e], r[i][e], q);
      }
    }
    float ss[1] = {sum2(q)};
    if (post || !WARP) row_sum<1, WARP, STAGED>(ss, tpr, ring.team, sh, turn);   // its barrier also frees the previous stage
    if (WARP) __syncwarp();
    if (done >= 0 && ring.stages > 1) issue(t0 + (ring.stages - 1) * step, done);
    const F2 hs = f2(post ? rsqrtf(ss[0] * p.inv_d + p.eps) : 1.f), a = f2(p.res_scale);
    const uint4 *xv = ring.row(p.sx);
    uint4 *rv = p.r + t * p.vecs + l;
    q = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool ok = i < NV - 1 || tail;
      F2 x[E];
      Vec<T>::unpack(ok ? xv[i * tpr] : zero, x);
      if (branch) {
        if (post) {
          F2 w[E];
          Vec<T>::unpack(ok ? ring.common(p.all, 0, i * tpr) : zero, w);
#pragma unroll
          for (int e = 0; e < E; ++e) r[i][e] = mul(r[i][e], mul(hs, w[e]));
        }
        if (gated) {
          F2 g[E];
          Vec<T>::unpack(!ok ? zero : all_gate ? ring.common(p.all, 2, i * tpr) : own_gate ? ring.row(p.sg)[i * tpr] : __ldg(gv + i * tpr), g);
#pragma unroll
          for (int e = 0; e < E; ++e) r[i][e] = mul(r[i][e], g[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[i][e] = fma(a, x[e], r[i][e]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) r[i][e] = mul(a, x[e]);
      }
      if (p.r && ok && row_ok) rv[i * tpr] = Vec<T>::pack(r[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) q = fma(r[i][e], r[i][e], q);
    }
    done = ring.at;
    if (!p.u) continue;
    ss[0] = sum2(q);
    row_sum<1, WARP, STAGED>(ss, tpr, ring.team, sh, turn);
    const F2 rs = f2(rsqrtf(ss[0] * p.inv_d + p.eps));
    uint4 *uv = p.u + t * p.vecs + l;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i < NV - 1 || tail) && row_ok) {
        F2 w[E];
        Vec<T>::unpack(ring.common(p.all, 1, i * tpr), w);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = mul(r[i][e], mul(rs, w[e]));
        uv[i * tpr] = Vec<T>::pack(w);
      }
    }
  }
  ring.end();
}

struct NormBwdParams {
  RingSrc src;
  RingShape ring;
  int sr, su, sh, sd, sg;        // stage slots of r, du, h, dr and a token's gate
  Shared3 all;                   // w_post, w_pre, a gate that all tokens share
  const uint4 *gate;
  uint4 *dx, *dh, *dgate_tok;
  float *part_pre;               // [CTAs][vecs * 2 E]: sums of du rn; null where not asked for
  float *part_a;                 // [units][vecs * 2 E]: sums of dR hn (token gates: of dN hn)
  int rows_per_b;                // tokens of one gate row (P * s, or all of them)
  int vecs, gate_mode, B, s;
  int bs, upb;                   // gate rows that units walk (B for sequence gates, else 1); units (runs of tokens) each
  float res_scale, eps, inv_d;
};

template <typename T, int NV, bool WARP, bool STAGED>
__global__ void __maxnreg__(sizeof(T) == 4 && NV == 2 && !WARP ? 96 : 128) residual_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int E = Vec<T>::N;
  constexpr bool kUnitGate = STAGED && !WARP;   // a unit's gate is staged beside the weights
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ uint64_t bars[kMaxTeams * kMaxStages];
  __shared__ int abort_flag;
  __shared__ float sh3[2 * 32][3], sh1[2 * 32][1];
  int turn3 = 0, turn1 = 0;
  Ring<WARP, STAGED> ring(stage_mem, bars, &abort_flag, p.vecs, p.ring, p.all);
  const int l = ring.l, tpr = ring.lanes, team = ring.team, teams = WARP ? kWarpTeams : STAGED ? blockDim.x / tpr : 1;
  const int G = teams * ring.rows;   // tokens of a turn of the CTA's teams
  const bool tail = l + (NV - 1) * tpr < p.vecs;   // this thread's last vector exists
  const bool post = p.all.p[0] != nullptr, gated = p.gate_mode != ULY_GATE_NONE;
  const bool all_gate = p.gate_mode == ULY_GATE_CHANNEL;
  F2 a_pre[NV][E], a_a[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) a_pre[i][e] = a_a[i][e] = f2(0.f);
  // Column sums of a CTA's rows: lanes of the same columns, then its teams in order,
  // through the memory of the stages, which all are done with.
  auto store_sums = [&](F2 (&v)[NV][E], float *part, long long index) {
    F2 *o = reinterpret_cast<F2 *>(part) + index * p.vecs * E;
    F2 *buf = teams > 1 ? reinterpret_cast<F2 *>(ring.first_stage()) + team * p.vecs * E : o;
    if (teams > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (WARP)
          for (int off = tpr; off < 32; off <<= 1) {
            F2 w;
            w.v = __shfl_xor_sync(0xffffffffu, v[i][e].v, off);
            v[i][e] = add(v[i][e], w);
          }
        if ((i < NV - 1 || tail) && ring.sub == 0) buf[(l + (long long)i * tpr) * E + e] = v[i][e];
        v[i][e] = f2(0.f);
      }
    if (teams > 1) {
      __syncthreads();
      const F2 *all = reinterpret_cast<const F2 *>(ring.first_stage());
      for (int c = threadIdx.x; c < p.vecs * E; c += blockDim.x) {
        F2 a = all[c];
        for (int t = 1; t < teams; ++t) a = add(a, all[t * p.vecs * E + c]);
        o[c] = a;
      }
      sm100::fence_proxy_async_smem();   // bulk copies may follow
      __syncthreads();
    }
  };
  const int units = p.bs * p.upb;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int b = unit / p.upb, part = unit - b * p.upb;
    const int q0 = (int)((long long)p.rows_per_b * part / p.upb) + team * ring.rows;
    const int q1 = (int)((long long)p.rows_per_b * (part + 1) / p.upb);
    // token k of gate row b: rank k / s, position k % s
    auto token = [&](int k) { return p.bs == 1 ? k : k + (k / p.s * (p.B - 1) + b) * p.s; };
    auto issue = [&](int k, int st) {
      if (k >= q1) return;
      const int n = min(ring.rows, q1 - k);
      if (p.bs == 1 || !WARP) ring.issue(p.src, token(k), n, st);
      else ring.issue_each(p.src, token(min(k + ring.sub, q1 - 1)), n, st);
    };
    const uint4 *seq_gate = p.gate + (long long)b * p.vecs + l;   // a channel gate's b is 0
    if (WARP || unit != blockIdx.x) ring.barrier();   // every thread is done with the last unit's stages
    {
      int st = ring.at;
      for (int k = 0; k < ring.stages; ++k) {
        issue(q0 + k * G, st);
        if (++st == ring.stages) st = 0;
      }
    }
    if (kUnitGate && p.gate_mode == ULY_GATE_SEQUENCE) {   // the gate of the unit's tokens
      __syncthreads();
      ring.share(2, p.gate + (long long)b * p.vecs, p.vecs);
      __syncthreads();
    }
    int done = -1;
    int pos = p.bs == 1 ? 0 : (q0 + ring.sub) % p.s, t = token(q0 + ring.sub);
    for (int k = q0; k < q1; k += G, ring.next()) {
      const long long base = (long long)t * p.vecs + l;
      const bool row_ok = !WARP || k + ring.sub < q1;
      const bool ok_tail = tail && row_ok;
      if (ring.stages == 1 && done >= 0) {   // no stage to run ahead into
        ring.barrier();
        issue(k, 0);
      }
      ring.wait(p.ring);
      F2 rr = f2(0.f), ar = f2(0.f), hh = f2(0.f);   // sums of r^2, du w_pre r and h^2, taken together
      const uint4 *rv = ring.row(p.sr), *uv = ring.row(p.su), *hv = ring.row(p.sh), *dv = ring.row(p.sd);
      F2 hn[NV][E];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * tpr;
        if (i < NV - 1 ? row_ok : ok_tail) {
          if (p.sh >= 0) {
            Vec<T>::unpack(hv[v], hn[i]);
            if (post) {
#pragma unroll
              for (int e = 0; e < E; ++e) hh = fma(hn[i][e], hn[i][e], hh);
            }
          }
          if (p.su >= 0) {
            F2 r[E], u[E], w[E];
            Vec<T>::unpack(rv[v], r);
            Vec<T>::unpack(uv[v], u);
            Vec<T>::unpack(ring.common(p.all, 1, v), w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              rr = fma(r[e], r[e], rr);
              ar = fma(mul(u[e], w[e]), r[e], ar);
            }
          }
        }
      }
      float s3[3] = {sum2(rr), sum2(ar), sum2(hh)};
      row_sum<3, WARP, STAGED>(s3, tpr, team, sh3, turn3);   // its barrier also frees the previous stage
      if (WARP) __syncwarp();
      if (done >= 0 && ring.stages > 1) issue(k + (ring.stages - 1) * G, done);
      const float irs = rsqrtf(s3[0] * p.inv_d + p.eps);
      const F2 ir = f2(irs), nc1 = f2(-s3[1] * irs * irs * p.inv_d);   // -mean(a rn) / rms(r)
      const float ihs = post ? rsqrtf(s3[2] * p.inv_d + p.eps) : 1.f;
      const F2 ih = f2(ihs), a = f2(p.res_scale);
      F2 s1p = f2(0.f), dn[NV][E];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * tpr;
        if (i < NV - 1 ? row_ok : ok_tail) {
          F2 (&d)[E] = dn[i];
          if (p.sd >= 0) {
            Vec<T>::unpack(dv[v], d);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = f2(0.f);
          }
          if (p.su >= 0) {
            F2 r[E], u[E], w[E];
            Vec<T>::unpack(rv[v], r);
            Vec<T>::unpack(uv[v], u);
            Vec<T>::unpack(ring.common(p.all, 1, v), w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              d[e] = fma(ir, fma(nc1, r[e], mul(u[e], w[e])), d[e]);
              a_pre[i][e] = fma(mul(u[e], ir), r[e], a_pre[i][e]);
            }
          }
          if (p.dx) {
            F2 o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = mul(a, d[e]);
            p.dx[base + v] = Vec<T>::pack(o);
          }
          if (p.sh >= 0) {
            F2 w[E];
            if (post) {
              Vec<T>::unpack(ring.common(p.all, 0, v), w);
#pragma unroll
              for (int e = 0; e < E; ++e) hn[i][e] = mul(hn[i][e], ih);
            }
            if (p.sg < 0) {
#pragma unroll
              for (int e = 0; e < E; ++e) a_a[i][e] = fma(d[e], hn[i][e], a_a[i][e]);
            }
            if (gated) {
              F2 g[E];
              Vec<T>::unpack(p.sg >= 0 ? ring.row(p.sg)[v]
                             : STAGED && all_gate || kUnitGate ? ring.common(p.all, 2, v) : __ldg(seq_gate + v), g);
              if (p.sg >= 0) {
                if (p.dgate_tok) {
                  F2 o[E];
#pragma unroll
                  for (int e = 0; e < E; ++e) o[e] = mul(d[e], post ? mul(hn[i][e], w[e]) : hn[i][e]);   // dR N(h)
                  p.dgate_tok[base + v] = Vec<T>::pack(o);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) a_a[i][e] = fma(mul(d[e], g[e]), hn[i][e], a_a[i][e]);
              }
#pragma unroll
              for (int e = 0; e < E; ++e) d[e] = mul(d[e], g[e]);
            }
            if (post) {
#pragma unroll
              for (int e = 0; e < E; ++e) {
                d[e] = mul(d[e], w[e]);
                s1p = fma(d[e], hn[i][e], s1p);
              }
            }
          }
        }
      }
      done = ring.at;
      if (p.bs > 1) {   // the group's next token
        for (pos += G, t += G; pos >= p.s; pos -= p.s) t += (p.B - 1) * p.s;
      } else {
        t += G;
      }
      if (!p.dh) continue;
      F2 nc2 = f2(0.f);
      if (post) {
        float s1[1] = {sum2(s1p)};
        row_sum<1, WARP, STAGED>(s1, tpr, team, sh1, turn1);
        nc2 = f2(-s1[0] * p.inv_d);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i < NV - 1 ? row_ok : ok_tail) {
          if (post) {
#pragma unroll
            for (int e = 0; e < E; ++e) dn[i][e] = mul(ih, fma(nc2, hn[i][e], dn[i][e]));
          }
          p.dh[base + i * tpr] = Vec<T>::pack(dn[i]);
        }
      }
    }
    if (p.part_a) store_sums(a_a, p.part_a, unit);
  }
  if (p.part_pre) store_sums(a_pre, p.part_pre, blockIdx.x);
  ring.end();
}

// ------------------------------------------------------------------- host

// Teams and stages for rows of `vecs` vectors: lanes of a warp (a power of two)
// while `nv` vectors a lane cover a row, several teams of one warp a CTA and
// several CTAs an SM; else teams of the fewest warps that do, one CTA an SM with
// the weights staged or (`apart`, and where two stages do not fit beside them) CTAs
// of one team.  As many as the registers allow and two stages each (one only where
// a single team's do not fit); `slots` tensors a stage.
struct RowShape {
  int lanes, nv, teams, rows;   // threads of a row, vectors of each; teams of a CTA, rows of a team
  int threads, per_sm, stages;
  bool staged;                  // the weights in shared memory
  uint32_t smem;
};
constexpr RowShape row_shape(int vecs, int slots, int nv, bool backward, bool f32, bool apart = false) {
  RowShape r = {};
  auto need = [&](int lanes) { return (vecs + lanes - 1) / lanes; };
  const bool warp = vecs <= 32 * nv;
  if (warp) {
    r.lanes = 1;
    while (need(r.lanes) > nv) r.lanes *= 2;
  } else {
    r.lanes = (need(nv) + 31) / 32 * 32;
    if (r.lanes > kMaxLanes) r.lanes = kMaxLanes;
  }
  r.nv = need(r.lanes);
  r.rows = warp ? 32 / r.lanes : 1;
  // threads an SM holds by the kernels' registers: up to 128; forward 100 where a
  // team is several warps and 64 up to two vectors a thread; backward 96 for two
  // fp32 vectors where a team is several warps
  const int room = backward ? (f32 && r.nv == 2 && !warp ? 640 : 512) : r.nv <= 2 ? 1024 : warp ? 512 : 640;
  const int team = warp ? 32 : r.lanes;
  const uint32_t row = (uint32_t)vecs * 16, stage = row * slots * r.rows;
  int teams = room / team;   // of an SM
  if (!warp && teams > kMaxTeams) teams = kMaxTeams;
  if (teams < 1) teams = 1;
  auto bytes = [&](int t, int stages) { return t * stages * stage + 3 * row * (warp ? (t + kWarpTeams - 1) / kWarpTeams : 1); };
  while (teams > 1 && bytes(teams, 2) > kRingBytes) --teams;
  if (warp && teams > kWarpTeams) teams = teams / kWarpTeams * kWarpTeams;
  // the backward's three and four bf16 vectors need its 128 registers for themselves:
  // their weights come from L1
  r.staged = (warp || !apart) && !(backward && !f32 && r.nv > 2) && bytes(teams, 2) <= kRingBytes;
  const uint32_t beside = r.staged ? 0 : 3 * row;   // what bytes() counts too much
  r.stages = 1;
  while (r.stages < kMaxStages && bytes(teams, r.stages + 1) - beside <= kRingBytes) ++r.stages;
  r.teams = warp ? kWarpTeams : apart ? 1 : teams;
  r.per_sm = warp ? (teams > kWarpTeams ? teams / kWarpTeams : 1) : apart ? teams : 1;
  r.threads = r.teams * team;
  r.smem = bytes(r.teams, r.stages) - beside;
  return r;
}
constexpr int kFwdVecs = 5, kBwdVecs = 2;

template <typename Params>
struct Entry {
  void (*kernel)(Params);
  std::atomic<uint64_t> optin{0};
};
// The kernel for `nv` vectors a thread, opted into its shared memory.
template <typename Params>
uly_status run(Entry<Params> &e, int grid, int threads, uint32_t smem, const Params &p, cudaStream_t stream) {
  if (!smem_optin(e.kernel, (int)kRingBytes, e.optin)) return ULY_ERR_CUDA;
  e.kernel<<<grid, threads, smem, stream>>>(p);
  note_launches(1);
  return last_launch_status();
}
// The kernels there are, and that row_shape() chooses each of them and no other.
constexpr bool fwd_kernel(const RowShape &r) {
  return r.lanes <= 32 ? r.staged && r.nv <= 5 : r.staged ? r.nv >= 3 && r.nv <= 5 : r.nv == 5;
}
constexpr bool bwd_kernel(const RowShape &r, bool f32) {
  return r.lanes <= 32 ? r.staged && r.nv <= 2 : r.staged ? r.nv >= 2 && r.nv <= (f32 ? 3 : 2) : r.nv >= 2 && r.nv <= 4;
}
constexpr bool kernels_fit_shapes(bool backward, bool f32) {
  unsigned chosen = 0, there = 0;
  auto bit = [](const RowShape &r) { return 1u << ((r.lanes <= 32 ? 0 : r.staged ? 8 : 16) + r.nv); };
  for (int vecs = 1; vecs <= kMaxVecs; ++vecs)
    for (int slots = backward ? 4 : 1; slots <= (backward ? 5 : 3); ++slots)
      for (int apart = 0; apart <= (backward && !f32); ++apart) {
        const RowShape r = row_shape(vecs, slots, backward ? kBwdVecs : kFwdVecs, backward, f32, apart);
        if (!(backward ? bwd_kernel(r, f32) : fwd_kernel(r))) return false;
        chosen |= bit(r);
      }
  for (int lanes = 32; lanes <= 64; lanes += 32)
    for (int staged = 0; staged <= 1; ++staged)
      for (int nv = 1; nv <= 5; ++nv) {
        RowShape r = {};
        r.lanes = lanes, r.staged = staged, r.nv = nv;
        if (backward ? bwd_kernel(r, f32) : fwd_kernel(r)) there |= bit(r);
      }
  return chosen == there;
}
static_assert(kernels_fit_shapes(false, false) && kernels_fit_shapes(false, true), "forward kernels");
static_assert(kernels_fit_shapes(true, false) && kernels_fit_shapes(true, true), "backward kernels");

template <typename T>
Entry<NormParams> &fwd_entry(const RowShape &r) {
  static Entry<NormParams> warp[5] = {{residual_norm_kernel<T, 1, true, true>}, {residual_norm_kernel<T, 2, true, true>},
                                      {residual_norm_kernel<T, 3, true, true>}, {residual_norm_kernel<T, 4, true, true>},
                                      {residual_norm_kernel<T, 5, true, true>}};
  static Entry<NormParams> cta[3] = {{residual_norm_kernel<T, 3, false, true>}, {residual_norm_kernel<T, 4, false, true>},
                                     {residual_norm_kernel<T, 5, false, true>}};
  static Entry<NormParams> wide = {residual_norm_kernel<T, 5, false, false>};
  return r.lanes <= 32 ? warp[r.nv - 1] : r.staged ? cta[r.nv - 3] : wide;
}
template <typename T>
Entry<NormBwdParams> &bwd_entry(const RowShape &r) {
  static Entry<NormBwdParams> warp[2] = {{residual_norm_bwd_kernel<T, 1, true, true>},
                                         {residual_norm_bwd_kernel<T, 2, true, true>}};
  static Entry<NormBwdParams> wide[3] = {{residual_norm_bwd_kernel<T, 2, false, false>},
                                         {residual_norm_bwd_kernel<T, 3, false, false>},
                                         {residual_norm_bwd_kernel<T, 4, false, false>}};
  if (r.lanes <= 32) return warp[r.nv - 1];
  if (r.staged) {
    static Entry<NormBwdParams> cta = {residual_norm_bwd_kernel<T, 2, false, true>};
    if constexpr (sizeof(T) == 4) {
      static Entry<NormBwdParams> cta3 = {residual_norm_bwd_kernel<T, 3, false, true>};
      if (r.nv == 3) return cta3;
    }
    return cta;
  }
  return wide[r.nv - 2];
}

// How the backward walks the tokens: `bs` gate rows, each cut into `upb` runs
// of tokens, on `grid` CTAs.  The same whichever tensors a call has.
struct BwdPlan {
  RowShape rs;
  int slots, bs, upb, grid;
  size_t off_pre, off_a, bytes;
};
BwdPlan bwd_plan(int B, long long n, int hidden, int e, int gate_mode) {
  BwdPlan q;
  q.slots = gate_mode == ULY_GATE_TOKEN ? 5 : 4;
  q.bs = gate_mode == ULY_GATE_SEQUENCE ? B : 1;
  const long long rows = gate_mode == ULY_GATE_SEQUENCE ? n : (long long)B * n;
  // Turns of the CTAs that take most: a unit costs its rows and about two more.
  auto plan = [&](bool apart) {
    q.rs = row_shape(hidden / e, q.slots, kBwdVecs, true, e == 4, apart);
    const long long want = (long long)device_sm_count() * q.rs.per_sm, turn = q.rs.teams * q.rs.rows;
    long long upb = want / q.bs, most = (rows + turn - 1) / turn;
    if (upb < 1) upb = 1;
    if (upb > most) upb = most;
    q.upb = (int)upb;
    const long long units = (long long)q.bs * q.upb, each = (rows + upb - 1) / upb;
    q.grid = (int)(units < want ? units : want);
    return (double)((units + q.grid - 1) / q.grid) * (double)((each + turn - 1) / turn + 2);
  };
  // bf16 teams of several warps: in one CTA an SM they share the weights and a unit's
  // gate in shared memory; CTAs of their own balance short units better and start
  // sooner, which counts up to some three rows an SM.  (In one CTA and apart, us:
  // 65536 x 2560 with a channel gate 419 and 452, 19531 x 4096 205 and 273; 2000
  // sequences of 8 x 2560 with their gates 270 and 227, 1000 of 50 419 and 500; 20
  // rows of 2560 16.7 and 13.6, 700 20.8 and 23.3.)
  const double together = plan(false);
  if (e == 8 && q.rs.lanes > 32 && q.rs.staged) {
    const bool few = q.bs * rows <= 3ll * device_sm_count();
    if (plan(true) > 0.9 * together && !few) plan(false);
  }
  const size_t col = (size_t)hidden * sizeof(float);
  q.off_pre = 0;
  q.off_a = q.off_pre + col * q.grid;
  q.bytes = q.off_a + col * q.bs * q.upb;
  return q;
}

// Column sums to fold, k < rows:
//   dst[k][c] = mul[c] sum over i < parts of weight[i / per_weight][c] src[k][i][c]
// (mul, weight: nullable vectors of the operators' own type).
struct FoldJob {
  const float *src;
  float *dst;
  long long parts;
  int rows;
  const void *mul, *weight;
  int per_weight;
};
struct FoldJobs {
  FoldJob job[3];
  int n, cols, bf16;
};
constexpr int kStrips = 16;

__device__ __forceinline__ float vector_at(const void *p, long long i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Grid rows a job takes: one for each of its rows, or, where these have few
// partials (a gate of every one of 2000 sequences, whose tokens one run takes), one
// for as many as there are strips (2000 x 8 x 512: 162 -> 27 us).
__host__ __device__ __forceinline__ int fold_units(const FoldJob &f, int ranks) {
  return f.parts < kStrips ? (f.rows + kStrips * ranks - 1) / (kStrips * ranks) : f.rows;
}

// Units of all jobs along grid.y, 32 columns a CTA; strips of partials are added
// in a fixed order and joined through shared memory.  The CTAs of a cluster (along
// grid.z) share the partials of a column: short rows have few columns and many
// partials.
constexpr int kFoldCluster = 8;
template <bool CLUSTER>
__global__ void __launch_bounds__(32 * kStrips) fold_columns_kernel(const __grid_constant__ FoldJobs jobs) {
  namespace cg = cooperative_groups;
  __shared__ float sh[kStrips][33], cta[32];
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5, cols = jobs.cols;
  const int ranks = CLUSTER ? gridDim.z : 1, rank = CLUSTER ? blockIdx.z : 0, stride = kStrips * ranks;
  int total = 0;
  for (int j = 0; j < jobs.n; ++j) total += fold_units(jobs.job[j], ranks);
  for (int unit = blockIdx.y; unit < total; unit += gridDim.y) {
    int k = unit, j = 0;
    while (k >= fold_units(jobs.job[j], ranks)) k -= fold_units(jobs.job[j++], ranks);
    const FoldJob &f = jobs.job[j];
    const long long parts = f.parts;
    const int c = blockIdx.x * 32 + lane;
    if (parts < kStrips) {   // a row a strip
      k = (k * ranks + rank) * kStrips + strip;
      if (k < f.rows && c < cols) {
        const float *s = f.src + (long long)k * parts * cols + c;
        float v = 0.f;
        for (int i = 0; i < (int)parts; ++i, s += cols)
          v += f.weight ? *s * vector_at(f.weight, (long long)(i / f.per_weight) * cols + c, jobs.bf16) : *s;
        if (f.mul) v *= vector_at(f.mul, c, jobs.bf16);
        f.dst[(long long)k * cols + c] = v;
      }
      continue;
    }
    const float *s = f.src + (long long)k * parts * cols;
    float a[8] = {};
    if (c < cols) {
      long long i = rank * kStrips + strip;
      if (f.weight) {
        for (; i + 3 * stride < parts; i += 4 * stride) {
          float v[4], w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = __ldcs(s + (i + e * stride) * cols + c);
            w[e] = vector_at(f.weight, (i + e * stride) / f.per_weight * cols + c, jobs.bf16);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = fmaf(v[e], w[e], a[e]);
        }
        for (; i < parts; i += stride)
          a[0] = fmaf(__ldcs(s + i * cols + c), vector_at(f.weight, i / f.per_weight * cols + c, jobs.bf16), a[0]);
      } else {
        for (; i + 7 * stride < parts; i += 8 * stride) {
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] += __ldcs(s + (i + stride * e) * cols + c);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e, i += stride)
          if (i < parts) a[e] += __ldcs(s + i * cols + c);
      }
    }
    sh[strip][lane] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    __syncthreads();
    float v = 0.f;
    if (strip == 0) {
#pragma unroll
      for (int e = 0; e < kStrips; ++e) v += sh[e][lane];
    }
    if (CLUSTER) {
      cg::cluster_group cluster = cg::this_cluster();
      if (strip == 0) cta[lane] = v;
      cluster.sync();
      if (strip == 0 && rank == 0)
        for (int r = 1; r < ranks; ++r) v += cluster.map_shared_rank(cta, r)[lane];
    }
    if (strip == 0 && rank == 0 && c < cols) {
      if (f.mul) v *= vector_at(f.mul, c, jobs.bf16);
      f.dst[(long long)k * cols + c] = v;
    }
    if (CLUSTER) cg::this_cluster().sync();
    else __syncthreads();
  }
}

uly_status fold_launch(const FoldJobs &jobs, cudaStream_t stream) {
  const long long cols = (jobs.cols + 31) / 32;
  long long rows = 0, many = 0, parts = 0;   // many: rows of many partials
  for (int j = 0; j < jobs.n; ++j) {
    rows += jobs.job[j].rows;
    if (jobs.job[j].parts >= kStrips) many += jobs.job[j].rows;
    if (jobs.job[j].parts > parts) parts = jobs.job[j].parts;
  }
  if (rows == 0) return ULY_OK;
  // where the SMs have room and a thread would have more than 32 partials (weighted
  // ones, 2 x 3 x 9000 x 256 with sequence gates: 13.9 us alone, 10.7 in clusters;
  // 444 of 1028 columns: 8.6 and 9.8)
  unsigned ranks = 1;
  if (parts > 32 * kStrips)
    while (ranks < kFoldCluster && cols * many * ranks <= device_sm_count()) ranks *= 2;
  long long units = 0;
  for (int j = 0; j < jobs.n; ++j) units += fold_units(jobs.job[j], (int)ranks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cols, (unsigned)(units < 65535 ? units : 65535), ranks);
  cfg.blockDim = dim3(32 * kStrips);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = ranks;
  cfg.attrs = &attr;
  cfg.numAttrs = ranks > 1;
  prof::Scope scope(prof::K_FOLD_COLUMNS, stream);
  if (cudaLaunchKernelEx(&cfg, ranks > 1 ? fold_columns_kernel<true> : fold_columns_kernel<false>, jobs) != cudaSuccess) {
    cudaGetLastError();
    return ULY_ERR_CUDA;
  }
  note_launches(1);
  return last_launch_status();
}

}  // namespace

uly_status fold_columns_launch(const float *src, int rows, long long parts, int cols, float *dst,
                               cudaStream_t stream) {
  FoldJobs jobs = {};
  jobs.job[0] = {src, dst, parts, rows, nullptr, nullptr, 1};
  jobs.n = 1;
  jobs.cols = cols;
  return fold_launch(jobs, stream);
}

bool residual_norm_supported(int vecs) { return vecs <= kMaxVecs; }

uly_status residual_norm_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *x,
                                const void *h, const void *gate, int32_t gate_mode, const void *w_post,
                                const void *w_pre, float res_scale, float eps, void *r, void *u,
                                cudaStream_t stream) {
  const bool bf = dtype == ULY_BF16;
  NormParams p = {};
  p.src.add(x, p.sx);
  p.src.add(h, p.sh);
  p.src.add(gate_mode == ULY_GATE_TOKEN ? gate : nullptr, p.sg);
  p.gate = static_cast<const uint4 *>(gate);
  p.all = {{static_cast<const uint4 *>(w_post), static_cast<const uint4 *>(w_pre),
            gate_mode == ULY_GATE_CHANNEL ? p.gate : nullptr}};
  p.r = static_cast<uint4 *>(r);
  p.u = static_cast<uint4 *>(u);
  p.rows = B * n;
  p.vecs = hidden / (bf ? 8 : 4);
  p.gate_mode = gate_mode; p.B = B; p.s = n / P;
  p.res_scale = res_scale; p.eps = eps; p.inv_d = 1.0f / hidden;
  const RowShape rs = row_shape(p.vecs, p.src.n, kFwdVecs, false, !bf);
  p.ring = {p.src.n, rs.stages, rs.lanes, error_word(), wait_limit_cycles()};
  const long long want = (long long)device_sm_count() * rs.per_sm, turn = rs.teams * rs.rows, ctas = (p.rows + turn - 1) / turn;
  const int grid = (int)(ctas < want ? ctas : want);
  prof::Scope scope(prof::K_RESIDUAL_NORM, stream);
  return run(bf ? fwd_entry<__nv_bfloat16>(rs) : fwd_entry<float>(rs), grid, rs.threads, rs.smem, p, stream);
}

size_t residual_norm_bwd_workspace_bytes(int32_t B, int32_t n, int32_t hidden, int32_t dtype, int32_t gate_mode) {
  return bwd_plan(B, n, hidden, dtype == ULY_BF16 ? 8 : 4, gate_mode).bytes;
}

uly_status residual_norm_bwd_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *r,
                                    const void *h, const void *dr, const void *du, const void *gate,
                                    int32_t gate_mode, const void *w_post, const void *w_pre, float res_scale,
                                    float eps, void *dx, void *dh, float *dw_post, float *dw_pre, void *dgate,
                                    void *workspace, cudaStream_t stream) {
  const bool bf = dtype == ULY_BF16;
  const bool shared_gate = gate_mode == ULY_GATE_CHANNEL || gate_mode == ULY_GATE_SEQUENCE;
  const BwdPlan q = bwd_plan(B, n, hidden, bf ? 8 : 4, gate_mode);
  char *ws = static_cast<char *>(workspace);
  NormBwdParams p = {};
  p.src.add(r, p.sr);
  p.src.add(du, p.su);
  p.src.add(h, p.sh);
  p.src.add(dr, p.sd);
  p.src.add(gate_mode == ULY_GATE_TOKEN ? gate : nullptr, p.sg);
  p.ring = {q.slots, q.rs.stages, q.rs.lanes, error_word(), wait_limit_cycles()};
  p.gate = static_cast<const uint4 *>(gate);
  p.all = {{static_cast<const uint4 *>(w_post), static_cast<const uint4 *>(w_pre),
            gate_mode == ULY_GATE_CHANNEL ? p.gate : nullptr}};
  p.dx = static_cast<uint4 *>(dx);
  p.dh = static_cast<uint4 *>(dh);
  p.dgate_tok = gate_mode == ULY_GATE_TOKEN ? static_cast<uint4 *>(dgate) : nullptr;
  p.part_pre = dw_pre ? reinterpret_cast<float *>(ws + q.off_pre) : nullptr;
  p.part_a = dw_post || (shared_gate && dgate) ? reinterpret_cast<float *>(ws + q.off_a) : nullptr;
  p.rows_per_b = gate_mode == ULY_GATE_SEQUENCE ? n : B * n;
  p.vecs = hidden / (bf ? 8 : 4);
  p.gate_mode = gate_mode; p.B = B; p.s = n / P;
  p.bs = q.bs; p.upb = q.upb;
  p.res_scale = res_scale; p.eps = eps; p.inv_d = 1.0f / hidden;
  {
    prof::Scope scope(prof::K_RESIDUAL_NORM_BWD, stream);
    const uly_status st = run(bf ? bwd_entry<__nv_bfloat16>(q.rs) : bwd_entry<float>(q.rs), q.grid,
                              q.rs.threads, q.rs.smem, p, stream);
    if (st != ULY_OK) return st;
  }
  const int run = q.upb;   // partials of one gate row
  FoldJobs jobs = {};
  jobs.cols = hidden;
  jobs.bf16 = bf;
  if (dw_pre) jobs.job[jobs.n++] = {p.part_pre, dw_pre, (long long)q.grid, 1, nullptr, nullptr, 1};
  if (dw_post) {
    FoldJob &f = jobs.job[jobs.n++];
    f = {p.part_a, dw_post, (long long)q.bs * run, 1, nullptr, nullptr, run};
    if (gate_mode == ULY_GATE_CHANNEL) f.mul = gate;
    if (gate_mode == ULY_GATE_SEQUENCE) (q.bs > 1 ? f.weight : f.mul) = gate;
  }
  if (shared_gate && dgate)
    jobs.job[jobs.n++] = {p.part_a, static_cast<float *>(dgate), run, q.bs, w_post, nullptr, 1};
  return fold_launch(jobs, stream);
}

}  // namespace uly
