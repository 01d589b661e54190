// C-ABI entry points of what a block holds between its linears: the gated
// residual with its norms, rotary positions and attention. Argument checks,
// workspace carving and launches on the caller's stream. No allocation, no
// synchronization, nothing printed.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "svdq.h"
#include "svdq_internal.h"
#include "svdq_layout.h"

namespace svdq {

namespace {

constexpr int64_t kMaxRows = 1 << 24;
// Attention's gradients recompute exp(s - lse) from an lse in fp32, whose
// rounding grows with the scores; the forward subtracts before it scales.
constexpr float kAttnGradScale = 0x1p10f;

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == SVDQ_DT_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype == SVDQ_DT_BF16 || dtype == SVDQ_DT_F16 || dtype == SVDQ_DT_F32; }

// ---------------------------------------------------------------------------
svdq_status check_residual(const svdq_residual_desc* d, int64_t M) {
  if (!d) return SVDQ_ERR_NULL;
  if (!known_dtype(d->dtype) || !known_dtype(d->param_dtype) || (d->norm != SVDQ_NORM_LAYER && d->norm != SVDQ_NORM_RMS))
    return SVDQ_ERR_FORMAT;
  if (d->channels < 1 || d->channels > kResidualChannels || d->groups < 1 || d->groups > kMaxRows || d->rows_per_group < 1 ||
      !(d->eps >= 0.f) || !std::isfinite(d->alpha))
    return SVDQ_ERR_SHAPE;
  if (M < 0 || M > kMaxRows) return SVDQ_ERR_SHAPE;
  if (M > 0 && (M - 1) / d->rows_per_group >= d->groups) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

svdq_status check_rows(const void* p, int64_t ld, int channels, int dtype) {
  if (!p) return SVDQ_ERR_NULL;
  if (ld < channels || ld > ((int64_t)1 << 32) || !aligned(p, elem_bytes(dtype))) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

svdq_status check_params(const svdq_residual_desc* d, const svdq_residual_params* p) {
  if (!p) return SVDQ_OK;
  const void* at[] = {p->gate, p->weight, p->bias, p->post_weight};
  const int64_t ld[] = {p->ld_gate, p->ld_weight, p->ld_bias, p->ld_post};
  for (int i = 0; i < 4; ++i) {
    if (!at[i]) continue;
    const svdq_status st = check_rows(at[i], d->groups > 1 ? ld[i] : d->channels, d->channels, d->param_dtype);
    if (st != SVDQ_OK) return st;
  }
  return p->post_weight && !d->post_norm ? SVDQ_ERR_SHAPE : SVDQ_OK;
}

ResidualArgs residual_args(const svdq_residual_desc* d, const void* x, int64_t ldx, const void* h, int64_t ldh,
                           const svdq_residual_params* p, int64_t M) {
  ResidualArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = d->dtype;
  a.pdtype = d->param_dtype;
  a.one_plus = d->one_plus ? 1 : 0;
  a.layer = d->norm == SVDQ_NORM_LAYER;
  a.C = d->channels;
  a.G = d->groups;
  a.post = d->post_norm ? 1 : 0;
  a.eps = d->eps;
  a.alpha = d->alpha;
  a.M = M;
  a.rpg = std::min<int64_t>(d->rows_per_group, std::max<int64_t>(M, 1));   // (past M the same groups)
  a.x = x;
  a.ldx = ldx;
  a.h = h;
  a.ldh = ldh;
  if (p) {
    a.gate = p->gate;
    a.w = p->weight;
    a.b = p->bias;
    a.pw = p->post_weight;
    const bool many = d->groups > 1;   // (a stride counts with several groups)
    a.ldgate = many ? p->ld_gate : 0;
    a.ldw = many ? p->ld_weight : 0;
    a.ldb = many ? p->ld_bias : 0;
    a.ldpw = many ? p->ld_post : 0;
  }
  return a;
}

// ---------------------------------------------------------------------------
// a tensor of heads: n samples, tokens and heads of it
svdq_status check_heads(const svdq_heads* t, int64_t samples, int64_t tokens, int64_t heads, int bytes) {
  if (!t || !t->p) return SVDQ_ERR_NULL;
  const int64_t vec = 16 / bytes, most = (int64_t)1 << 40;
  if (!aligned(t->p, 16)) return SVDQ_ERR_SHAPE;
  const int64_t stride[] = {t->batch, t->token, t->head}, n[] = {samples, tokens, heads};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (stride[i] < 0 || stride[i] > most || stride[i] % vec != 0)) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}
// (a dimension of one has stride 0)
Heads heads_of(const svdq_heads* t, int64_t samples, int64_t tokens, int64_t heads) {
  return Heads{t->p, samples > 1 ? t->batch : 0, tokens > 1 ? t->token : 0, heads > 1 ? t->head : 0};
}
// an output's elements lie apart: nested strides, in the order of their size
svdq_status check_apart(const svdq_heads* t, int64_t samples, int64_t tokens, int64_t heads, int64_t dim) {
  int64_t stride[] = {t->batch, t->token, t->head}, n[] = {samples, tokens, heads};
  for (int i = 0; i < 3; ++i)   // sorted by stride
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(n[i], n[j]);
      }
  int64_t span = dim;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (stride[i] < span) return SVDQ_ERR_SHAPE;
    span += (n[i] - 1) * stride[i];   // (n < 2^31, strides up to 2^40: their product may pass 2^63)
    if (span > ((int64_t)1 << 50) || span < 0) return SVDQ_ERR_SHAPE;
  }
  return SVDQ_OK;
}

svdq_status check_rope(const svdq_rope_desc* d, int* pairs) {
  if (!d) return SVDQ_ERR_NULL;
  if (!known_dtype(d->dtype) || (d->position_type != SVDQ_POS_I32 && d->position_type != SVDQ_POS_F32)) return SVDQ_ERR_FORMAT;
  if (d->axes < 1 || d->axes > 4 || d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8 != 0) return SVDQ_ERR_SHAPE;
  int n = 0;
  for (int i = 0; i < d->axes; ++i) {
    if (d->pairs[i] < 0 || d->pairs[i] > 128) return SVDQ_ERR_SHAPE;
    n += d->pairs[i];
  }
  if (n < 1 || 2 * n > d->head_dim || (d->half && n % 8 != 0)) return SVDQ_ERR_SHAPE;
  if (d->q_heads < 0 || d->q_heads > 65536 || d->k_heads < 0 || d->k_heads > 65536) return SVDQ_ERR_SHAPE;
  if (d->samples < 0 || d->tokens < 0 || d->samples > kMaxRows || d->tokens > kMaxRows || d->samples * d->tokens > kMaxRows / 2)
    return SVDQ_ERR_SHAPE;
  *pairs = n;
  return SVDQ_OK;
}

// ---------------------------------------------------------------------------
svdq_status check_attention(const svdq_attention_desc* d) {
  if (!d) return SVDQ_ERR_NULL;
  if (d->dtype != SVDQ_DT_BF16 && d->dtype != SVDQ_DT_F16) return SVDQ_ERR_FORMAT;
  if (d->head_dim < 8 || d->head_dim > 128 || d->head_dim % 8 != 0 || d->kv_heads < 1 || d->heads < d->kv_heads ||
      d->heads > 65535 || d->heads % d->kv_heads != 0 || !(d->scale >= 0x1p-64f && d->scale <= 0x1p64f))   // (lse / scale is fp32)
    return SVDQ_ERR_SHAPE;
  const int64_t most = (int64_t)1 << 30, group = d->heads / d->kv_heads;
  if (d->samples < 0 || d->queries < 0 || d->keys < 0 || d->samples > 65535 || d->queries >= most || d->keys >= most)
    return SVDQ_ERR_SHAPE;
  const int64_t heads = d->samples * d->kv_heads, rows = d->queries * group;
  const int64_t blocks = (std::max(rows, d->keys) + 4 * kAttnWave - 1) / (4 * kAttnWave);
  if (heads > 65535 || rows >= most || blocks * std::max<int64_t>(heads, 1) > ((int64_t)1 << 22)) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}
// a tensor's place, and the span of 64 of its tokens (with `group` heads)
svdq_status check_attn_heads(const svdq_heads* t, const svdq_attention_desc* d, bool of_q) {
  const int64_t tokens = of_q ? d->queries : d->keys, heads = of_q ? d->heads : d->kv_heads;
  const svdq_status st = check_heads(t, d->samples, tokens, heads, 2);
  if (st != SVDQ_OK) return st;
  const int64_t span = (tokens > 1 ? 63 * t->token : 0) + (of_q && heads > 1 ? (d->heads / d->kv_heads - 1) * t->head : 0) + 128;
  return span >= ((int64_t)1 << 30) ? SVDQ_ERR_SHAPE : SVDQ_OK;
}
svdq_status check_attn_out(const svdq_heads* t, const svdq_attention_desc* d, bool of_q) {
  const svdq_status st = check_attn_heads(t, d, of_q);
  return st != SVDQ_OK ? st
                       : check_apart(t, d->samples, of_q ? d->queries : d->keys, of_q ? d->heads : d->kv_heads, d->head_dim);
}
Heads attn_heads(const svdq_heads* t, const svdq_attention_desc* d, bool of_q) {
  return heads_of(t, d->samples, of_q ? d->queries : d->keys, of_q ? d->heads : d->kv_heads);
}
AttnSizes sizes_of(const svdq_attention_desc* d) {
  return AttnSizes{d->samples, d->queries, d->keys, d->heads, d->kv_heads, d->head_dim,
                   d->causal != 0, d->dtype == SVDQ_DT_F16, d->fine != 0};
}
AttnArgs attn_args(const svdq_attention_desc* d, const uint8_t* mask, int64_t mask_batch) {
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = d->dtype;
  a.B = (int)d->samples;
  a.Lq = (int)d->queries;
  a.Lk = (int)d->keys;
  a.H = d->heads;
  a.Hk = d->kv_heads;
  a.G = d->heads / d->kv_heads;
  a.group = attn_group(a.G);
  a.D = d->head_dim;
  a.causal = d->causal ? 1 : 0;
  a.scale = d->scale;
  a.scale_log2 = (float)((double)d->scale * 1.4426950408889634);
  a.mask = mask;
  a.mask_batch = d->samples > 1 ? mask_batch : 0;
  return a;
}
svdq_status check_mask(const svdq_attention_desc* d, const uint8_t* mask, int64_t mask_batch) {
  return mask && d->samples > 1 && (mask_batch < 0 || mask_batch > ((int64_t)1 << 40)) ? SVDQ_ERR_SHAPE : SVDQ_OK;
}
svdq_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return SVDQ_OK;
  if (!ws) return SVDQ_ERR_NULL;
  if (!aligned(ws, 16)) return SVDQ_ERR_SHAPE;
  return have < need ? SVDQ_ERR_WORKSPACE : SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

#define SVDQ_TRY(expr)                    \
  do {                                    \
    const svdq_status st_ = (expr);       \
    if (st_ != SVDQ_OK) return st_;       \
  } while (0)

extern "C" {

svdq_status svdq_residual_norm_forward(const svdq_residual_desc* d, const void* x, int64_t ldx, const void* h, int64_t ldh,
                                       const svdq_residual_params* params, int64_t M, void* s, int64_t lds, void* y,
                                       int64_t ldy, float* stats, void* stream) {
  SVDQ_TRY(check_residual(d, M));
  SVDQ_TRY(check_params(d, params));
  if (M == 0) return SVDQ_OK;
  SVDQ_TRY(check_rows(x, ldx, d->channels, d->dtype));
  SVDQ_TRY(check_rows(h, ldh, d->channels, d->dtype));
  SVDQ_TRY(check_rows(s, lds, d->channels, d->dtype));
  SVDQ_TRY(check_rows(y, ldy, d->channels, d->dtype));
  if (s == y || !aligned(stats, 4)) return SVDQ_ERR_SHAPE;
  int cus = 0;
  SVDQ_TRY(check_device(&cus));
  ResidualArgs a = residual_args(d, x, ldx, h, ldh, params, M);
  a.s = s;
  a.lds = lds;
  a.y = y;
  a.ldy = ldy;
  a.stats = stats;
  hipStream_t st = (hipStream_t)stream;
  return after_launch(launch_residual(a, cus, st), st);
}

svdq_status svdq_residual_norm_backward_workspace_bytes(const svdq_residual_desc* d, int64_t M, size_t* out) {
  SVDQ_TRY(check_residual(d, M));
  if (!out) return SVDQ_ERR_NULL;
  *out = residual_grad_ws(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype), d->post_norm);
  return SVDQ_OK;
}

svdq_status svdq_residual_norm_backward(const svdq_residual_desc* d, const void* dy, int64_t lddy, const void* ds, int64_t ldds,
                                        const void* s, int64_t lds, const void* h, int64_t ldh,
                                        const svdq_residual_params* params, const float* stats, int64_t M, void* dx,
                                        int64_t lddx, void* dh, int64_t lddh, const svdq_residual_grads* grads,
                                        int32_t grad_dtype, void* ws, size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_residual(d, M));
  SVDQ_TRY(check_params(d, params));
  if (!known_dtype(grad_dtype)) return SVDQ_ERR_FORMAT;
  ResidualGradArgs g;
  std::memset(&g, 0, sizeof(g));
  if (grads) {
    g.out[0] = grads->gate;
    g.out[1] = grads->weight;
    g.out[2] = grads->bias;
    g.out[3] = grads->post_weight;
  }
  bool any = false;
  for (void* p : g.out) {
    any = any || p;
    if (!aligned(p, elem_bytes(grad_dtype))) return SVDQ_ERR_SHAPE;
  }
  if (g.out[3] && !d->post_norm) return SVDQ_ERR_SHAPE;
  if (M == 0 && !any) return SVDQ_OK;
  if (M > 0) {
    SVDQ_TRY(check_rows(dy, lddy, d->channels, d->dtype));
    if (ds) SVDQ_TRY(check_rows(ds, ldds, d->channels, d->dtype));
    SVDQ_TRY(check_rows(s, lds, d->channels, d->dtype));
    SVDQ_TRY(check_rows(h, ldh, d->channels, d->dtype));
    SVDQ_TRY(check_rows(dx, lddx, d->channels, d->dtype));
    SVDQ_TRY(check_rows(dh, lddh, d->channels, d->dtype));
    if (!stats) return SVDQ_ERR_NULL;
    if (dx == dh || !aligned(stats, 4)) return SVDQ_ERR_SHAPE;
  }
  const size_t need = any ? residual_grad_ws(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype), d->post_norm) : 0;
  SVDQ_TRY(check_ws(ws, ws_bytes, need));
  SVDQ_TRY(check_device());
  g.f = residual_args(d, s, lds, h, ldh, params, M);
  g.f.stats = const_cast<float*>(stats);
  g.dy = dy;
  g.lddy = lddy;
  g.ds = ds;
  g.ldds = ds ? ldds : 0;
  g.dx = dx;
  g.lddx = lddx;
  g.dh = dh;
  g.lddh = lddh;
  for (const void* in : {dy, ds, s, h}) g.in_place |= M > 0 && in && (in == dx || in == dh);
  g.gdtype = grad_dtype;
  g.part = need > 0 ? (float*)ws : nullptr;
  hipStream_t st = (hipStream_t)stream;
  return after_launch(
      launch_residual_grad(g, residual_grad_plan(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype), d->post_norm), st), st);
}

svdq_status svdq_rope(const svdq_rope_desc* d, const svdq_heads* q, const svdq_heads* k, const void* positions,
                      int64_t position_batch, const double* freqs, const svdq_heads* q_out, const svdq_heads* k_out,
                      void* stream) {
  int pairs = 0;
  SVDQ_TRY(check_rope(d, &pairs));
  if (d->samples * d->tokens == 0 || d->q_heads + d->k_heads == 0) return SVDQ_OK;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const svdq_heads* in[] = {q, k};
  const svdq_heads* out[] = {q_out, k_out};
  const int heads[] = {d->q_heads, d->k_heads}, bytes = elem_bytes(d->dtype);
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    SVDQ_TRY(check_heads(in[i], d->samples, d->tokens, heads[i], bytes));
    SVDQ_TRY(check_heads(out[i], d->samples, d->tokens, heads[i], bytes));
    SVDQ_TRY(check_apart(out[i], d->samples, d->tokens, heads[i], d->head_dim));
    a.x[i] = heads_of(in[i], d->samples, d->tokens, heads[i]);
    a.y[i] = heads_of(out[i], d->samples, d->tokens, heads[i]);
    a.H[i] = heads[i];
  }
  if (!positions || !freqs) return SVDQ_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(freqs, 8) || position_batch < 0 || position_batch > ((int64_t)1 << 40))
    return SVDQ_ERR_SHAPE;
  SVDQ_TRY(check_device());
  a.dtype = d->dtype;
  a.pos_dtype = d->position_type;
  a.B = (int)d->samples;
  a.L = (int)d->tokens;
  a.D = d->head_dim;
  a.axes = d->axes;
  a.pairs = pairs;
  a.half = d->half ? 1 : 0;
  a.inverse = d->inverse ? 1 : 0;
  for (int i = 0; i < 4; ++i) a.first[i + 1] = a.first[i] + (i < d->axes ? d->pairs[i] : 0);
  a.pos = positions;
  a.pos_batch = d->samples > 1 ? position_batch : 0;
  a.freqs = freqs;
  hipStream_t st = (hipStream_t)stream;
  return after_launch(launch_rope(a, st), st);
}

svdq_status svdq_attention_workspace_bytes(const svdq_attention_desc* d, size_t* out) {
  SVDQ_TRY(check_attention(d));
  if (!out) return SVDQ_ERR_NULL;
  *out = d->samples * d->queries == 0 ? 0 : attn_ws(sizes_of(d)).total;
  return SVDQ_OK;
}

svdq_status svdq_attention_forward(const svdq_attention_desc* d, const svdq_heads* q, const svdq_heads* k, const svdq_heads* v,
                                   const uint8_t* key_mask, int64_t mask_batch, const svdq_heads* o, float* lse, void* ws,
                                   size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_attention(d));
  if (d->samples * d->queries == 0) return SVDQ_OK;
  AttnArgs a = attn_args(d, key_mask, mask_batch);
  SVDQ_TRY(check_attn_heads(q, d, true));
  SVDQ_TRY(check_attn_out(o, d, true));
  a.q = attn_heads(q, d, true);
  a.o = attn_heads(o, d, true);
  if (d->keys > 0) {
    SVDQ_TRY(check_attn_heads(k, d, false));
    SVDQ_TRY(check_attn_heads(v, d, false));
    SVDQ_TRY(check_mask(d, key_mask, mask_batch));
    a.k = attn_heads(k, d, false);
    a.v = attn_heads(v, d, false);
  }
  if (!lse) return SVDQ_ERR_NULL;
  if (!aligned(lse, 4)) return SVDQ_ERR_SHAPE;
  const AttnWs w = attn_ws(sizes_of(d));
  SVDQ_TRY(check_ws(ws, ws_bytes, w.total));
  SVDQ_TRY(check_device(nullptr, nullptr, kKernelsAttention));
  a.lse = lse;
  a.cost = w.cost;
  a.plan = w.plan;
  a.part_rows = (int)attn_part_rows(a.cost);
  a.part = (float*)((uint8_t*)ws + w.part);
  a.part_stat = (float*)((uint8_t*)ws + w.part_stat);
  hipStream_t st = (hipStream_t)stream;
  return after_launch(launch_attention(a, st), st);
}

svdq_status svdq_attention_backward_workspace_bytes(const svdq_attention_desc* d, size_t* out) {
  SVDQ_TRY(check_attention(d));
  if (!out) return SVDQ_ERR_NULL;
  *out = d->samples * (d->queries + d->keys) == 0 ? 0 : attn_grad_ws(sizes_of(d)).total;
  return SVDQ_OK;
}

svdq_status svdq_attention_backward(const svdq_attention_desc* d, const svdq_heads* dout, const svdq_heads* q,
                                    const svdq_heads* k, const svdq_heads* v, const svdq_heads* o, const float* lse,
                                    const uint8_t* key_mask, int64_t mask_batch, const svdq_heads* dq, const svdq_heads* dk,
                                    const svdq_heads* dv, void* ws, size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_attention(d));
  if (d->scale > kAttnGradScale) return SVDQ_ERR_SHAPE;
  if (d->samples * (d->queries + d->keys) == 0) return SVDQ_OK;
  AttnGradArgs g;
  std::memset(&g, 0, sizeof(g));
  g.f = attn_args(d, key_mask, mask_batch);
  if (d->queries > 0) {
    for (const svdq_heads* t : {dout, q, o}) SVDQ_TRY(check_attn_heads(t, d, true));
    SVDQ_TRY(check_attn_out(dq, d, true));
    g.f.q = attn_heads(q, d, true);
    g.f.o = attn_heads(o, d, true);
    g.dout = attn_heads(dout, d, true);
    g.dq = attn_heads(dq, d, true);
    if (!lse) return SVDQ_ERR_NULL;
    if (!aligned(lse, 4)) return SVDQ_ERR_SHAPE;
    g.f.lse = const_cast<float*>(lse);
  }
  if (d->keys > 0) {
    for (const svdq_heads* t : {k, v}) SVDQ_TRY(check_attn_heads(t, d, false));
    for (const svdq_heads* t : {dk, dv}) SVDQ_TRY(check_attn_out(t, d, false));
    SVDQ_TRY(check_mask(d, key_mask, mask_batch));
    g.f.k = attn_heads(k, d, false);
    g.f.v = attn_heads(v, d, false);
    g.dk = attn_heads(dk, d, false);
    g.dv = attn_heads(dv, d, false);
  }
  const AttnGradWs w = attn_grad_ws(sizes_of(d));
  SVDQ_TRY(check_ws(ws, ws_bytes, w.total));
  SVDQ_TRY(check_device(nullptr, nullptr, kKernelsAttention));
  uint8_t* at = (uint8_t*)ws;
  g.lse = (float*)(at + w.lse);
  g.delta = (float*)(at + w.delta);
  g.top_do = (float*)(at + w.top_do);
  g.top_v = (float*)(at + w.top_v);
  g.f.part = (float*)(at + w.part);
  g.row_blocks = w.dq.blocks;
  g.rows_padded = (int64_t)w.dq.blocks * w.rows.block;
  g.key_runs = w.key_runs;
  hipStream_t st = (hipStream_t)stream;
  return after_launch(launch_attention_grad(g, w, st), st);
}

}  // extern "C"
