// C-ABI entry points of the layer norm and the FP8 linear: argument checks,
// workspace carving and launches on the caller's stream. No allocation, no
// synchronization, nothing printed.
#include <algorithm>
#include <cstring>

#include "svdq.h"
#include "svdq_internal.h"
#include "svdq_layout.h"

namespace svdq {

namespace {

constexpr int64_t kMaxRows = 1 << 24;
constexpr int64_t kMaxGradRows = 1 << 20;   // keeps a tile of a transposed operand below 2^31 bytes

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == SVDQ_DT_F32 ? 4 : 2; }
bool known_dtype(int dtype) { return dtype == SVDQ_DT_BF16 || dtype == SVDQ_DT_F16 || dtype == SVDQ_DT_F32; }

svdq_status check_norm(const svdq_norm_desc* d, int64_t M) {
  if (!d) return SVDQ_ERR_NULL;
  if (!known_dtype(d->dtype) || !known_dtype(d->param_dtype)) return SVDQ_ERR_FORMAT;
  if (d->channels < 1 || d->channels > 16384 || d->groups < 1 || d->groups > kMaxRows || d->rows_per_group < 1 ||
      !(d->eps >= 0.f))
    return SVDQ_ERR_SHAPE;
  if (M < 0 || M > kMaxRows) return SVDQ_ERR_SHAPE;
  if (M > 0 && (M - 1) / d->rows_per_group >= d->groups) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}

// rows of a matrix: stride and the alignment of one element
svdq_status check_rows(const void* p, int64_t ld, int channels, int dtype) {
  if (!p) return SVDQ_ERR_NULL;
  if (ld < channels || ld > ((int64_t)1 << 32) || !aligned(p, elem_bytes(dtype))) return SVDQ_ERR_SHAPE;
  return SVDQ_OK;
}
svdq_status check_params(const svdq_norm_desc* d, const void* p, int64_t ld) {
  return p ? check_rows(p, d->groups > 1 ? ld : d->channels, d->channels, d->param_dtype) : SVDQ_OK;
}

NormArgs norm_args(const svdq_norm_desc* d, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* b,
                   int64_t ldb, int64_t M) {
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = d->dtype;
  a.pdtype = d->param_dtype;
  a.one_plus = d->one_plus ? 1 : 0;
  a.C = d->channels;
  a.G = d->groups;
  a.eps = d->eps;
  a.M = M;
  a.rpg = std::min<int64_t>(d->rows_per_group, std::max<int64_t>(M, 1));   // (past M the same groups)
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = d->groups > 1 ? ldw : d->channels;
  a.b = b;
  a.ldb = d->groups > 1 ? ldb : d->channels;
  return a;
}

svdq_status check_fp8_m(const svdq_fp8_desc* d, int64_t M, int64_t most) {
  const svdq_status st = check_fp8_desc(d);
  if (st != SVDQ_OK) return st;
  return M < 0 || M > most ? SVDQ_ERR_SHAPE : SVDQ_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

svdq_status check_fp8_dev(const svdq_fp8_packed* p) {
  if (!p || !p->q || !p->s) return SVDQ_ERR_NULL;
  return aligned(p->q, 16) && aligned(p->s, 16) && aligned(p->bias, 16) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

Fp8Gemm forward_gemm(const svdq_fp8_desc* d, const svdq_fp8_packed* dev, int64_t M, uint16_t* y) {
  Fp8Gemm g;
  std::memset(&g, 0, sizeof(g));
  g.a_rows = M;
  g.lda = round128(d->K);
  g.b = dev->q;
  g.bs = dev->s;
  g.b_rows = d->N;
  g.ldb = d->K;
  g.K = d->K;
  g.bias = dev->bias;
  g.out = y;
  return g;
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

svdq_status svdq_layer_norm_forward(const svdq_norm_desc* d, const void* x, int64_t ldx, const void* weight, int64_t ldw,
                                    const void* bias, int64_t ldb, int64_t M, void* y, int64_t ldy, float* mean,
                                    float* rstd, void* stream) {
  SVDQ_TRY(check_norm(d, M));
  if (M == 0) return SVDQ_OK;
  SVDQ_TRY(check_rows(x, ldx, d->channels, d->dtype));
  SVDQ_TRY(check_rows(y, ldy, d->channels, d->dtype));
  SVDQ_TRY(check_params(d, weight, ldw));
  SVDQ_TRY(check_params(d, bias, ldb));
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return SVDQ_ERR_SHAPE;
  int cus = 0;
  SVDQ_TRY(check_device(&cus, nullptr, kKernelsNorm));
  NormArgs a = norm_args(d, x, ldx, weight, ldw, bias, ldb, M);
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  hipStream_t s = (hipStream_t)stream;
  return after_launch(launch_norm(a, cus, s), s);
}

svdq_status svdq_layer_norm_backward_workspace_bytes(const svdq_norm_desc* d, int64_t M, size_t* out) {
  SVDQ_TRY(check_norm(d, M));
  if (!out) return SVDQ_ERR_NULL;
  *out = norm_grad_ws(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype));
  return SVDQ_OK;
}

svdq_status svdq_layer_norm_backward(const svdq_norm_desc* d, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                     const void* weight, int64_t ldw, const float* mean, const float* rstd, int64_t M,
                                     void* dx, int64_t lddx, void* dweight, void* dbias, int32_t grad_dtype, void* ws,
                                     size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_norm(d, M));
  if (!known_dtype(grad_dtype)) return SVDQ_ERR_FORMAT;
  const bool pg = dweight || dbias;
  if (!aligned(dweight, elem_bytes(grad_dtype)) || !aligned(dbias, elem_bytes(grad_dtype))) return SVDQ_ERR_SHAPE;
  if (M == 0 && !pg) return SVDQ_OK;
  if (M > 0) {
    SVDQ_TRY(check_rows(dy, lddy, d->channels, d->dtype));
    SVDQ_TRY(check_rows(x, ldx, d->channels, d->dtype));
    SVDQ_TRY(check_rows(dx, lddx, d->channels, d->dtype));
    SVDQ_TRY(check_params(d, weight, ldw));
    if (!mean || !rstd) return SVDQ_ERR_NULL;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return SVDQ_ERR_SHAPE;
  }
  const size_t need = pg ? norm_grad_ws(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype)) : 0;
  if (need > 0) {
    if (!ws) return SVDQ_ERR_NULL;
    if (!aligned(ws, 16)) return SVDQ_ERR_SHAPE;
    if (ws_bytes < need) return SVDQ_ERR_WORKSPACE;
  }
  SVDQ_TRY(check_device(nullptr, nullptr, kKernelsNorm));
  NormGradArgs g;
  std::memset(&g, 0, sizeof(g));
  g.f = norm_args(d, x, ldx, weight, ldw, nullptr, 0, M);
  g.f.mean = const_cast<float*>(mean);
  g.f.rstd = const_cast<float*>(rstd);
  g.dy = dy;
  g.lddy = lddy;
  g.dx = dx;
  g.lddx = lddx;
  g.dw = dweight;
  g.db = dbias;
  g.gdtype = grad_dtype;
  g.part = need > 0 ? (float*)ws : nullptr;
  hipStream_t s = (hipStream_t)stream;
  return after_launch(launch_norm_grad(g, norm_grad_plan(M, d->groups, d->rows_per_group, d->channels, elem_bytes(d->dtype)), s), s);
}

svdq_status svdq_fp8_packed_bytes(const svdq_fp8_desc* d, svdq_fp8_sizes* out) {
  SVDQ_TRY(check_fp8_desc(d));
  if (!out) return SVDQ_ERR_NULL;
  out->q = out->qt = (size_t)d->N * d->K;
  out->s = (size_t)((d->N + 127) / 128) * fp8_block_row(d->K);
  out->st = (size_t)((d->K + 127) / 128) * fp8_block_row(d->N);
  out->bias = (size_t)d->N * 2;
  return SVDQ_OK;
}

svdq_status svdq_fp8_pack(const svdq_fp8_desc* d, const void* w, int32_t dtype, const svdq_fp8_packed* o, void* stream) {
  SVDQ_TRY(check_fp8_desc(d));
  if (!known_dtype(dtype)) return SVDQ_ERR_FORMAT;
  if (!w || !o || !o->q || !o->s || !o->qt != !o->st) return SVDQ_ERR_NULL;
  if (!aligned(w, 16) || !aligned(o->q, 16) || !aligned(o->s, 16) || !aligned(o->qt, 16) || !aligned(o->st, 16))
    return SVDQ_ERR_SHAPE;
  SVDQ_TRY(check_device(nullptr, nullptr, kKernelsFp8));
  hipStream_t s = (hipStream_t)stream;
  return after_launch(launch_fp8_pack(w, dtype, d->K, d->N, o->q, o->s, o->qt, o->st, s), s);
}

svdq_status svdq_fp8_workspace_bytes(const svdq_fp8_desc* d, int64_t M, size_t* out) {
  SVDQ_TRY(check_fp8_m(d, M, kMaxRows));
  if (!out) return SVDQ_ERR_NULL;
  *out = fp8_inline(M, d->K) ? 0 : fp8_ws(d, M).total;
  return SVDQ_OK;
}

svdq_status svdq_fp8_forward(const svdq_fp8_desc* d, const svdq_fp8_packed* dev, const uint16_t* x, int64_t M,
                             uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_fp8_m(d, M, kMaxRows));
  SVDQ_TRY(check_fp8_dev(dev));
  if (M == 0) return SVDQ_OK;
  if (!x || !y) return SVDQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16)) return SVDQ_ERR_SHAPE;
  const bool in_line = fp8_inline(M, d->K);
  const Fp8Ws L = fp8_ws(d, M);
  // one kernel, whose workgroups read all of x while others write y
  if (in_line && overlap(x, (size_t)M * d->K * 2, y, (size_t)M * d->N * 2)) return SVDQ_ERR_SHAPE;
  if (!in_line) {
    if (!ws) return SVDQ_ERR_NULL;
    if (!aligned(ws, 16)) return SVDQ_ERR_SHAPE;
    if (ws_bytes < L.total) return SVDQ_ERR_WORKSPACE;
  }
  int cus = 0;
  SVDQ_TRY(check_device(&cus, nullptr, kKernelsFp8));
  hipStream_t s = (hipStream_t)stream;
  Fp8Gemm g = forward_gemm(d, dev, M, y);
  if (in_line) {
    g.x = x;
    return after_launch(launch_fp8_gemm_small(g, cus, s), s);
  }
  uint8_t* b = fp8_ws_start(ws);
  SVDQ_TRY(after_launch(launch_fp8_quant_rows(x, M, d->K, b + L.q, b + L.s, false, (uint32_t*)(b + L.tickets), s), s));
  g.a = b + L.q;
  g.as = b + L.s;
  g.part = (float*)(b + L.part);
  g.tickets = (uint32_t*)(b + L.tickets);
  return after_launch(launch_fp8_gemm(g, cus, s), s);
}

svdq_status svdq_fp8_norm_workspace_bytes(const svdq_fp8_desc* d, int64_t M, size_t* out) {
  SVDQ_TRY(check_fp8_m(d, M, kMaxRows));
  if (!out) return SVDQ_ERR_NULL;
  *out = M == 0 ? 0 : fp8_ws(d, M).total;
  return SVDQ_OK;
}

svdq_status svdq_fp8_norm_forward(const svdq_norm_desc* n, const void* weight, int64_t ldw, const void* bias, int64_t ldb,
                                  const svdq_fp8_desc* d, const svdq_fp8_packed* dev, const uint16_t* x, int64_t M,
                                  uint16_t* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
  SVDQ_TRY(check_norm(n, M));
  SVDQ_TRY(check_fp8_m(d, M, kMaxRows));
  if (n->dtype != SVDQ_DT_BF16) return SVDQ_ERR_FORMAT;
  if (n->channels != d->K) return SVDQ_ERR_SHAPE;
  SVDQ_TRY(check_fp8_dev(dev));
  if (M == 0) return SVDQ_OK;
  if (!x || !y || !ws) return SVDQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SVDQ_ERR_SHAPE;
  SVDQ_TRY(check_params(n, weight, ldw));
  SVDQ_TRY(check_params(n, bias, ldb));
  const Fp8Ws L = fp8_ws(d, M);
  if (ws_bytes < L.total) return SVDQ_ERR_WORKSPACE;
  int cus = 0;
  SVDQ_TRY(check_device(&cus, nullptr, kKernelsNorm | kKernelsFp8));
  hipStream_t s = (hipStream_t)stream;
  uint8_t* b = fp8_ws_start(ws);
  NormArgs a = norm_args(n, x, d->K, weight, ldw, bias, ldb, M);
  a.mean = mean;
  a.rstd = rstd;
  a.q = b + L.q;
  a.qs = b + L.s;
  a.Kp = (int)round128(d->K);
  a.qs_rows = M;
  a.tickets = (uint32_t*)(b + L.tickets);
  SVDQ_TRY(after_launch(launch_norm(a, cus, s), s));
  Fp8Gemm g = forward_gemm(d, dev, M, y);
  g.a = b + L.q;
  g.as = b + L.s;
  g.part = (float*)(b + L.part);
  g.tickets = (uint32_t*)(b + L.tickets);
  // (the same kernel as svdq_fp8_forward, so the same sums)
  return after_launch(fp8_inline(M, d->K) ? launch_fp8_gemm_small(g, cus, s) : launch_fp8_gemm(g, cus, s), s);
}

svdq_status svdq_fp8_backward_workspace_bytes(const svdq_fp8_desc* d, int64_t M, size_t* out) {
  SVDQ_TRY(check_fp8_m(d, M, kMaxGradRows));
  if (!out) return SVDQ_ERR_NULL;
  *out = M == 0 ? 0 : fp8_grad_ws(d, M).total;
  return SVDQ_OK;
}

svdq_status svdq_fp8_backward(const svdq_fp8_desc* d, const svdq_fp8_packed* dev, const uint16_t* x, const uint16_t* dy,
                              int64_t M, uint16_t* dx, uint16_t* dw, uint16_t* db, void* ws, size_t ws_bytes,
                              void* stream) {
  SVDQ_TRY(check_fp8_m(d, M, kMaxGradRows));
  if (dx && (!dev || !dev->qt || !dev->st)) return SVDQ_ERR_NULL;
  if (dx && (!aligned(dev->qt, 16) || !aligned(dev->st, 16))) return SVDQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 16) || !aligned(ws, 16))
    return SVDQ_ERR_SHAPE;
  if (!dx && !dw && !db) return SVDQ_OK;
  const Fp8GradWs L = fp8_grad_ws(d, M);
  if (M > 0) {
    if (!dy || (dw && !x) || !ws) return SVDQ_ERR_NULL;
    if (ws_bytes < L.total) return SVDQ_ERR_WORKSPACE;
  }
  int cus = 0;
  SVDQ_TRY(check_device(&cus, nullptr, kKernelsFp8));
  hipStream_t s = (hipStream_t)stream;
  if (M == 0) {
    if (dw) SVDQ_TRY(after_launch(launch_fp8_zero(dw, (size_t)d->N * d->K * 2, cus, s), s));
    if (db) SVDQ_TRY(after_launch(launch_fp8_zero(db, (size_t)d->N * 2, cus, s), s));
    return SVDQ_OK;
  }
  uint8_t* b = fp8_ws_start(ws);
  Fp8QuantT qy, qx;
  std::memset(&qy, 0, sizeof(qy));
  std::memset(&qx, 0, sizeof(qx));
  qy.x = dy;
  qy.C = d->N;
  if (dx) {
    qy.q = b + L.q;
    qy.s = b + L.s;
  }
  if (db) qy.sums = (float*)(b + L.db);
  if (dw) {
    qy.qt = b + L.yt;
    qy.st = b + L.yts;
    qx.x = x;
    qx.C = d->K;
    qx.qt = b + L.xt;
    qx.st = b + L.xts;
  }
  SVDQ_TRY(after_launch(launch_fp8_quant_t(qy, qx, M, (uint32_t*)(b + L.tickets), s), s));
  Fp8Gemm gx, gw;
  std::memset(&gx, 0, sizeof(gx));
  std::memset(&gw, 0, sizeof(gw));
  if (dx) {
    Fp8Gemm& g = gx;
    g.a = qy.q;
    g.as = qy.s;
    g.a_rows = M;
    g.lda = round128(d->N);
    g.b = dev->qt;
    g.bs = dev->st;
    g.b_rows = d->K;
    g.ldb = d->N;
    g.K = d->N;
    g.out = dx;
    g.part = (float*)(b + L.part);
    g.tickets = (uint32_t*)(b + L.tickets);
  }
  if (dw) {
    Fp8Gemm& g = gw;
    g.a = qy.qt;
    g.as = qy.st;
    g.a_rows = d->N;
    g.lda = round128(M);
    g.b = qx.qt;
    g.bs = qx.st;
    g.b_rows = d->K;
    g.ldb = round128(M);
    g.b_row_scales = 1;
    g.K = round128(M);
    g.out = dw;
    g.part = (float*)(b + L.part);
    g.tickets = (uint32_t*)(b + L.tickets) + kFp8Tickets;
  }
  // the bias gradient: in the first product's launch that takes it, else its own
  const Fp8BiasGrad bias = {qy.sums, (int)(round128(M) / 128), d->N, db};
  const bool in_dx = db && dx && fp8_gemm_takes_bias(gx), in_dw = db && dw && !in_dx && fp8_gemm_takes_bias(gw);
  if (db && !in_dx && !in_dw) SVDQ_TRY(after_launch(launch_fp8_bias_grad(bias, s), s));
  if (dx) SVDQ_TRY(after_launch(launch_fp8_gemm(gx, cus, s, in_dx ? &bias : nullptr), s));
  if (dw) SVDQ_TRY(after_launch(launch_fp8_gemm(gw, cus, s, in_dw ? &bias : nullptr), s));
  return SVDQ_OK;
}

svdq_status svdq_fp8_quantize(const uint16_t* x, int64_t M, int32_t K, uint8_t* codes, uint8_t* scales, void* stream) {
  const svdq_fp8_desc d = {K, 16};
  SVDQ_TRY(check_fp8_m(&d, M, kMaxRows));
  if (M == 0) return SVDQ_OK;
  if (!x || !codes || !scales) return SVDQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return SVDQ_ERR_SHAPE;
  SVDQ_TRY(check_device(nullptr, nullptr, kKernelsFp8));
  hipStream_t s = (hipStream_t)stream;
  return after_launch(launch_fp8_quant_rows(x, M, K, codes, scales, true, nullptr, s), s);
}

}  // extern "C"
