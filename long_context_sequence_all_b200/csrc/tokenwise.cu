// C ABI of the token-wise operators: argument validation and dispatch.
// Declarations and the contract of every entry point are in include/ulysses.h.
#include <cmath>
#include <initializer_list>

#include "common.cuh"
#include "tokenwise.cuh"

namespace {

using namespace uly;

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

bool all_aligned(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!aligned16(p)) return false;
  return true;
}

// A buffer of a call: null or empty ones overlap nothing.
struct Span {
  const void *p;
  size_t bytes;
};
bool meet(const Span &a, const Span &b) {
  return a.p && b.p && a.bytes && b.bytes && overlap(a.p, a.bytes, b.p, b.bytes);
}
// No output may overlap an input or another output.
bool outputs_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *a = outs.begin(); a != outs.end(); ++a) {
    for (const Span &b : ins)
      if (meet(*a, b)) return false;
    for (const Span *b = a + 1; b != outs.end(); ++b)
      if (meet(*a, *b)) return false;
  }
  return true;
}
// The input, unless the output is that very buffer (element-wise in place).
Span unless_same(const Span &in, const void *out) { return in.p == out ? Span{nullptr, 0} : in; }

constexpr long long kMaxRows = 0x7fffffffLL - 4096;

bool known_act(int act) { return act >= ULY_ACT_NONE && act <= ULY_ACT_SWIGLU; }

uly_status linear_shape(int64_t tokens, int32_t in, int32_t out, int32_t act) {
  if (tokens < 0 || tokens > kMaxRows || in <= 0 || out <= 0) return ULY_ERR_SHAPE;
  if (!known_act(act)) return ULY_ERR_UNSUPPORTED;
  if (in % 8 || out % 8) return ULY_ERR_ALIGN;
  if (out > kMaxRows / 2 || in > kMaxRows) return ULY_ERR_SHAPE;
  auto tiles = [](long long v) { return (v + 127) / 128; };
  // 32-bit work units: a tile each, fewer than (SM pairs)^2 more where the last turn's
  // are cut, and eight rows of tiles at a time in the raster
  const long long most = 0x7fffffffLL / 32;
  if (tiles(tokens) * tiles(out) > most || tiles(tokens) * tiles(in) > most || 2 * tiles(out) * tiles(in) > most)
    return ULY_ERR_SHAPE;
  return ULY_OK;
}

uly_status norm_shape(int32_t batch, int32_t seq_len, int32_t world, int32_t hidden, int32_t dtype,
                      int32_t gate_mode) {
  if (dtype != ULY_BF16 && dtype != ULY_F32) return ULY_ERR_DTYPE;
  if (batch <= 0 || seq_len <= 0 || world <= 0 || hidden <= 0 || seq_len % world) return ULY_ERR_SHAPE;
  if ((long long)batch * seq_len > kMaxRows) return ULY_ERR_SHAPE;
  if (gate_mode < ULY_GATE_NONE || gate_mode > ULY_GATE_TOKEN) return ULY_ERR_UNSUPPORTED;
  const int e = dtype == ULY_BF16 ? 8 : 4;
  if (hidden % e) return ULY_ERR_ALIGN;
  if (!residual_norm_supported(hidden / e)) return ULY_ERR_UNSUPPORTED;
  return ULY_OK;
}

size_t gate_elems(int32_t mode, int32_t batch, int32_t seq_len, int32_t hidden) {
  switch (mode) {
    case ULY_GATE_CHANNEL: return (size_t)hidden;
    case ULY_GATE_SEQUENCE: return (size_t)batch * hidden;
    case ULY_GATE_TOKEN: return (size_t)batch * seq_len * hidden;
    default: return 0;
  }
}

uly_status loss_shape(int32_t world, int64_t tokens, int32_t hidden, int32_t vocab) {
  if (world <= 0 || world > 65535 || tokens < 0 || tokens > kMaxRows || hidden <= 0 || vocab <= 0 || tokens % world)
    return ULY_ERR_SHAPE;
  if (hidden % 8) return ULY_ERR_ALIGN;
  auto tiles = [](long long v) { return (v + 255) / 256; };
  const long long most = 0x7fffffffLL / 32;
  if (vocab > (1 << 28) || hidden > kMaxRows || tiles(tokens) * tiles(vocab) > most ||
      tiles(tokens) * tiles(hidden) > most || tiles(vocab) * tiles(hidden) > most)
    return ULY_ERR_SHAPE;
  return ULY_OK;
}

}  // namespace

extern "C" {

uly_status ulysses_linear_workspace_size(int64_t tokens, int32_t in_features, int32_t out_features,
                                         int32_t activation, size_t *bytes) {
  if (!bytes) return ULY_ERR_NULL;
  const uly_status st = linear_shape(tokens, in_features, out_features, activation);
  if (st != ULY_OK) return st;
  *bytes = align256(linear_workspace_bytes(tokens, in_features, out_features, activation));
  return ULY_OK;
}

uly_status ulysses_linear(int64_t tokens, int32_t in_features, int32_t out_features, int32_t activation,
                          const void *x, const void *w, const void *bias, const void *residual, void *y, void *pre,
                          void *workspace, size_t workspace_bytes, void *stream) {
  uly_status st = linear_shape(tokens, in_features, out_features, activation);
  if (st != ULY_OK) return st;
  if (tokens == 0) return ULY_OK;
  if (!x || !w || !y) return ULY_ERR_NULL;
  size_t need = 0;
  ulysses_linear_workspace_size(tokens, in_features, out_features, activation, &need);
  if (need && (!workspace || workspace_bytes < need)) return ULY_ERR_WORKSPACE;
  if (!all_aligned({x, w, bias, residual, y, pre, need ? workspace : nullptr})) return ULY_ERR_ALIGN;
  const size_t nz = (size_t)out_features * (activation == ULY_ACT_SWIGLU ? 2 : 1);
  const size_t yb = (size_t)tokens * out_features * 2;
  if (!outputs_apart({{y, yb}, {pre, (size_t)tokens * nz * 2}, {workspace, need}},
                     {{x, (size_t)tokens * in_features * 2}, {w, nz * in_features * 2}, {bias, nz * 2}}) ||
      meet({y, yb}, unless_same({residual, yb}, y)) || meet({pre, (size_t)tokens * nz * 2}, {residual, yb}) ||
      meet({workspace, need}, {residual, yb}))
    return ULY_ERR_ALIAS;
  return linear_launch(tokens, in_features, out_features, activation, x, w, bias, residual, y, pre, workspace,
                       static_cast<cudaStream_t>(stream));
}

uly_status ulysses_linear_bwd_workspace_size(int64_t tokens, int32_t in_features, int32_t out_features,
                                             int32_t activation, size_t *bytes) {
  if (!bytes) return ULY_ERR_NULL;
  const uly_status st = linear_shape(tokens, in_features, out_features, activation);
  if (st != ULY_OK) return st;
  *bytes = align256(linear_bwd_workspace_bytes(tokens, in_features, out_features, activation));
  return ULY_OK;
}

uly_status ulysses_linear_bwd(int64_t tokens, int32_t in_features, int32_t out_features, int32_t activation,
                              const void *x, const void *w, const void *pre, const void *dy, void *dx, void *dw,
                              int32_t dw_dtype, float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
  uly_status st = linear_shape(tokens, in_features, out_features, activation);
  if (st != ULY_OK) return st;
  if (!dx && !dw && !dbias && tokens > 0) return ULY_ERR_NULL;
  if (dw && dw_dtype != ULY_F32 && dw_dtype != ULY_BF16) return ULY_ERR_DTYPE;
  const size_t nz = (size_t)out_features * (activation == ULY_ACT_SWIGLU ? 2 : 1);
  const size_t dwb = nz * in_features * (dw_dtype == ULY_F32 ? 4 : 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (!all_aligned({dw, dbias})) return ULY_ERR_ALIGN;
    if ((dw && cudaMemsetAsync(dw, 0, dwb, s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, nz * sizeof(float), s) != cudaSuccess))
      return ULY_ERR_CUDA;
    return ULY_OK;
  }
  if (!dy || (dx && !w) || (dw && !x) || (activation != ULY_ACT_NONE && !pre)) return ULY_ERR_NULL;
  if (activation == ULY_ACT_NONE) pre = nullptr;
  size_t need = 0;
  ulysses_linear_bwd_workspace_size(tokens, in_features, out_features, activation, &need);
  if (need && (!workspace || workspace_bytes < need)) return ULY_ERR_WORKSPACE;
  if (!all_aligned({x, w, pre, dy, dx, dw, dbias, need ? workspace : nullptr})) return ULY_ERR_ALIGN;
  const size_t xb = (size_t)tokens * in_features * 2;
  if (!outputs_apart({{dx, xb}, {dw, dwb}, {dbias, nz * sizeof(float)}, {workspace, need}},
                     {{dw ? x : nullptr, xb}, {dx ? w : nullptr, nz * in_features * 2},
                      {pre, (size_t)tokens * nz * 2}, {dy, (size_t)tokens * out_features * 2}}))
    return ULY_ERR_ALIAS;
  return linear_bwd_launch(tokens, in_features, out_features, activation, x, w, pre, dy, dx, dw, dw_dtype, dbias,
                           workspace, s);
}

uly_status ulysses_residual_norm(int32_t batch, int32_t seq_len, int32_t world, int32_t hidden, int32_t dtype,
                                 const void *x, const void *h, const void *gate, int32_t gate_mode,
                                 const void *w_post, const void *w_pre, float res_scale, float eps, void *r, void *u,
                                 void *stream) {
  const uly_status st = norm_shape(batch, seq_len, world, hidden, dtype, gate_mode);
  if (st != ULY_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(res_scale)) return ULY_ERR_SHAPE;
  if (!x || (!r && !u) || (u && !w_pre) || (gate_mode != ULY_GATE_NONE && !gate)) return ULY_ERR_NULL;
  if (!h && (gate_mode != ULY_GATE_NONE || w_post)) return ULY_ERR_NULL;
  if (!u) w_pre = nullptr;
  if (gate_mode == ULY_GATE_NONE) gate = nullptr;
  if (!all_aligned({x, h, gate, w_post, w_pre, r, u})) return ULY_ERR_ALIGN;
  const size_t e = dtype == ULY_BF16 ? 2 : 4, tb = (size_t)batch * seq_len * hidden * e;
  const Span sg{gate, gate_elems(gate_mode, batch, seq_len, hidden) * e}, sp{w_post, hidden * e}, sq{w_pre, hidden * e};
  if (!outputs_apart({{r, tb}, {u, tb}}, {sg, sp, sq}) || meet({r, tb}, unless_same({x, tb}, r)) ||
      meet({r, tb}, unless_same({h, tb}, r)) || meet({u, tb}, {x, tb}) || meet({u, tb}, unless_same({h, tb}, u)))
    return ULY_ERR_ALIAS;
  return residual_norm_launch(batch, seq_len, world, hidden, dtype, x, h, gate, gate_mode, w_post, w_pre, res_scale,
                              eps, r, u, static_cast<cudaStream_t>(stream));
}

uly_status ulysses_residual_norm_bwd_workspace_size(int32_t batch, int32_t seq_len, int32_t hidden, int32_t dtype,
                                                    int32_t gate_mode, size_t *bytes) {
  if (!bytes) return ULY_ERR_NULL;
  const uly_status st = norm_shape(batch, seq_len, 1, hidden, dtype, gate_mode);
  if (st != ULY_OK) return st;
  *bytes = align256(residual_norm_bwd_workspace_bytes(batch, seq_len, hidden, dtype, gate_mode));
  return ULY_OK;
}

uly_status ulysses_residual_norm_bwd(int32_t batch, int32_t seq_len, int32_t world, int32_t hidden, int32_t dtype,
                                     const void *r, const void *h, const void *dr, const void *du, const void *gate,
                                     int32_t gate_mode, const void *w_post, const void *w_pre, float res_scale,
                                     float eps, void *dx, void *dh, float *dw_post, float *dw_pre, void *dgate,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  const uly_status st = norm_shape(batch, seq_len, world, hidden, dtype, gate_mode);
  if (st != ULY_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(res_scale)) return ULY_ERR_SHAPE;
  if ((!dr && !du) || (du && (!r || !w_pre)) || (gate_mode != ULY_GATE_NONE && !gate)) return ULY_ERR_NULL;
  if (!dx && !dh && !dw_post && !dw_pre && !dgate) return ULY_ERR_NULL;
  if (!h && (gate_mode != ULY_GATE_NONE || w_post || dh)) return ULY_ERR_NULL;
  if ((dw_post && !w_post) || (dw_pre && !du) || (dgate && gate_mode == ULY_GATE_NONE)) return ULY_ERR_NULL;
  if (!du) r = w_pre = nullptr;
  if (gate_mode == ULY_GATE_NONE) gate = nullptr;
  size_t need = 0;
  ulysses_residual_norm_bwd_workspace_size(batch, seq_len, hidden, dtype, gate_mode, &need);
  if (!workspace || workspace_bytes < need) return ULY_ERR_WORKSPACE;
  if (!all_aligned({r, h, dr, du, gate, w_post, w_pre, dx, dh, dw_post, dw_pre, dgate, workspace}))
    return ULY_ERR_ALIGN;
  const size_t e = dtype == ULY_BF16 ? 2 : 4, tb = (size_t)batch * seq_len * hidden * e, cb = (size_t)hidden * 4;
  const size_t ge = gate_elems(gate_mode, batch, seq_len, hidden);
  const Span sg{gate, ge * e}, sp{w_post, hidden * e}, sq{w_pre, hidden * e};
  const Span odx{dx, tb}, odh{dh, tb}, odg{dgate, gate_mode == ULY_GATE_TOKEN ? ge * e : ge * 4};
  if (!outputs_apart({odx, odh, {dw_post, cb}, {dw_pre, cb}, odg, {workspace, need}}, {{r, tb}, {h, tb}, sg, sp, sq}) ||
      !outputs_apart({{dw_post, cb}, {dw_pre, cb}, odg, {workspace, need}}, {{dr, tb}, {du, tb}}) ||
      meet(odx, unless_same({dr, tb}, dx)) || meet(odx, {du, tb}) || meet(odh, {dr, tb}) ||
      meet(odh, unless_same({du, tb}, dh)))
    return ULY_ERR_ALIAS;
  return residual_norm_bwd_launch(batch, seq_len, world, hidden, dtype, r, h, dr, du, gate, gate_mode, w_post, w_pre,
                                  res_scale, eps, dx, dh, dw_post, dw_pre, dgate, workspace,
                                  static_cast<cudaStream_t>(stream));
}

uly_status ulysses_linear_loss_workspace_size(int32_t world, int64_t tokens, int32_t hidden, int32_t vocab,
                                              size_t *bytes) {
  if (!bytes) return ULY_ERR_NULL;
  const uly_status st = loss_shape(world, tokens, hidden, vocab);
  if (st != ULY_OK) return st;
  *bytes = align256(linear_loss_workspace_bytes(world, tokens, hidden, vocab));
  return ULY_OK;
}

uly_status ulysses_linear_loss(int32_t world, int64_t tokens, int32_t hidden, int32_t vocab, const void *x,
                               const void *w, const int32_t *labels, int32_t ignore_index, float *shard_sum,
                               int64_t *shard_count, float *loss, void *workspace, size_t workspace_bytes,
                               void *stream) {
  const uly_status st = loss_shape(world, tokens, hidden, vocab);
  if (st != ULY_OK) return st;
  if (!w || !shard_sum || !shard_count || !loss || (tokens > 0 && (!x || !labels))) return ULY_ERR_NULL;
  size_t need = 0;
  ulysses_linear_loss_workspace_size(world, tokens, hidden, vocab, &need);
  if (!workspace || workspace_bytes < need) return ULY_ERR_WORKSPACE;
  if (!all_aligned({x, w, labels, workspace})) return ULY_ERR_ALIGN;
  if (!outputs_apart({{shard_sum, (size_t)world * 4}, {shard_count, (size_t)world * 8}, {loss, 4}, {workspace, need}},
                     {{x, (size_t)tokens * hidden * 2}, {w, (size_t)vocab * hidden * 2}, {labels, (size_t)tokens * 4}}))
    return ULY_ERR_ALIAS;
  return linear_loss_launch(world, tokens, hidden, vocab, x, w, labels, ignore_index, shard_sum, shard_count, loss,
                            workspace, static_cast<cudaStream_t>(stream));
}

uly_status ulysses_linear_loss_bwd_workspace_size(int32_t world, int64_t tokens, int32_t hidden, int32_t vocab,
                                                  int32_t dw_dtype, int64_t piece_tokens, size_t *bytes) {
  if (!bytes) return ULY_ERR_NULL;
  const uly_status st = loss_shape(world, tokens, hidden, vocab);
  if (st != ULY_OK) return st;
  if (dw_dtype != ULY_F32 && dw_dtype != ULY_BF16) return ULY_ERR_DTYPE;
  if (piece_tokens < 0) return ULY_ERR_SHAPE;
  *bytes = align256(linear_loss_bwd_workspace_bytes(world, tokens, hidden, vocab, dw_dtype, piece_tokens));
  return ULY_OK;
}

uly_status ulysses_linear_loss_bwd(int32_t world, int64_t tokens, int32_t hidden, int32_t vocab, const void *x,
                                   const void *w, const int32_t *labels, int32_t ignore_index, void *dx, void *dw,
                                   int32_t dw_dtype, int64_t piece_tokens, float *shard_sum, int64_t *shard_count,
                                   float *loss, void *workspace, size_t workspace_bytes, void *stream) {
  size_t need = 0;
  const uly_status st =
      ulysses_linear_loss_bwd_workspace_size(world, tokens, hidden, vocab, dw_dtype, piece_tokens, &need);
  if (st != ULY_OK) return st;
  if (!w || !dw || !shard_sum || !shard_count || !loss || (tokens > 0 && (!x || !labels || !dx))) return ULY_ERR_NULL;
  if (!workspace || workspace_bytes < need) return ULY_ERR_WORKSPACE;
  if (!all_aligned({x, w, labels, dx, dw, workspace})) return ULY_ERR_ALIGN;
  const size_t xb = (size_t)tokens * hidden * 2, wb = (size_t)vocab * hidden * 2;
  if (!outputs_apart({{dx, xb}, {dw, dw_dtype == ULY_F32 ? 2 * wb : wb}, {shard_sum, (size_t)world * 4},
                      {shard_count, (size_t)world * 8}, {loss, 4}, {workspace, need}},
                     {{x, xb}, {w, wb}, {labels, (size_t)tokens * 4}}))
    return ULY_ERR_ALIAS;
  return linear_loss_bwd_launch(world, tokens, hidden, vocab, x, w, labels, ignore_index, dx, dw, dw_dtype,
                                piece_tokens, shard_sum, shard_count, loss, workspace,
                                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
