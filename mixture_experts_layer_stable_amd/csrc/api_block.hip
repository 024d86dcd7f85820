// C-ABI entry points of the operators around the layer step: argument checks, workspace
// layouts, launches.
#include <cmath>

#include "api.h"
#include "block.h"

using namespace mok;

namespace {

mok_status check_norm(const mok_norm_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->act != MOK_F32 && d->act != MOK_BF16) return MOK_ERR_DTYPE;
  const bool mx = d->quant == MOK_MXFP8 || d->quant == MOK_MXFP4;
  if (d->quant != d->act && !(mx && d->act == MOK_BF16)) return MOK_ERR_DTYPE;
  if (d->reserved != 0 || (d->flags & ~MOK_FLAG_WGRAD_F32) != 0) return MOK_ERR_SHAPE;
  if (d->T < 0 || d->T >= ((int64_t)1 << 31)) return MOK_ERR_SHAPE;
  if (d->H < 8 || d->H > 32768 || d->H % 8 != 0) return MOK_ERR_SHAPE;
  if (mx && d->H % (d->quant == MOK_MXFP4 ? 256 : 128) != 0) return MOK_ERR_SHAPE;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return MOK_ERR_SHAPE;
  return MOK_OK;
}

mok_status check_balance(const mok_balance_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->grad != MOK_F32 && d->grad != MOK_BF16) return MOK_ERR_DTYPE;
  if (d->score != MOK_SCORE_SOFTMAX && d->score != MOK_SCORE_SIGMOID) return MOK_ERR_DTYPE;
  if (d->reserved != 0) return MOK_ERR_SHAPE;
  if (d->T < 0 || d->T >= ((int64_t)1 << 31) || d->E < 1 || d->E > 1024) return MOK_ERR_SHAPE;
  if (d->k < 1 || d->k > 16 || d->k > d->E || d->S < 0 || d->S > 65535) return MOK_ERR_SHAPE;
  if (d->T * d->k >= ((int64_t)1 << 31)) return MOK_ERR_SHAPE;  // an expert's count fits int32
  if (!std::isfinite(d->coef) || !std::isfinite(d->zcoef)) return MOK_ERR_SHAPE;
  if (d->zcoef != 0.0f && d->score != MOK_SCORE_SOFTMAX) return MOK_ERR_SHAPE;
  return MOK_OK;
}

BalanceArgs balance_args(const mok_balance_desc* d, const float* logits, const int32_t* seg, const uint8_t* mask) {
  BalanceArgs a{};
  a.T = d->T;
  a.E = d->E;
  a.k = d->k;
  a.S = std::max(d->S, 1);
  a.sigmoid = d->score == MOK_SCORE_SIGMOID;
  a.bf16_grad = d->grad == MOK_BF16;
  a.coef = d->coef;
  a.zcoef = d->zcoef;
  a.logits = logits;
  a.seg = d->S > 0 ? seg : nullptr;
  a.mask = mask;
  return a;
}

mok_status check_linear(const mok_linear_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->act != MOK_F32 && d->act != MOK_BF16) return MOK_ERR_DTYPE;
  if (d->epi < MOK_EPI_NONE || d->epi > MOK_EPI_SWIGLU) return MOK_ERR_DTYPE;
  if (d->reserved != 0 || (d->flags & ~MOK_FLAG_WGRAD_F32) != 0) return MOK_ERR_SHAPE;
  if (d->M < 0 || d->M >= ((int64_t)1 << 30)) return MOK_ERR_SHAPE;
  if (d->N < 8 || d->N > (1 << 20) || d->N % 8 != 0) return MOK_ERR_SHAPE;
  if (d->K < 8 || d->K > (1 << 20) || d->K % 8 != 0) return MOK_ERR_SHAPE;
  // an array of 2^37 elements is as large as the GPU's memory; the output tiles' threads fit 32 bits
  const int64_t P = d->epi == MOK_EPI_SWIGLU ? 2LL * d->N : d->N;
  if (std::max<int64_t>(d->M, 1) * std::max<int64_t>(P, d->K) >= (1LL << 37) || P * d->K >= (1LL << 37))
    return MOK_ERR_SHAPE;
  return MOK_OK;
}

int linear_p(const mok_linear_desc* d) { return d->epi == MOK_EPI_SWIGLU ? 2 * d->N : d->N; }

// Backward workspace: dp rows, bias-gradient parts, then the partial products of dx and dw
// (used one after the other).
struct LinearBwd {
  size_t dp, db, part, bytes;
};
LinearBwd linear_bwd(const mok_linear_desc* d) {
  const int P = linear_p(d);
  LinearBwd w;
  size_t o = 0;
  w.dp = o; o = up(o + (d->epi == MOK_EPI_NONE ? 0 : (size_t)elem_size(d->act) * (size_t)d->M * P));
  w.db = o; o = up(o + 4 * (size_t)linear_db_parts(d->M, d->N) * P);
  w.part = o;
  o = up(o + std::max(linear_part_bytes(LIN_DX, d->act, MOK_EPI_NONE, d->M, d->K, P),
                      linear_part_bytes(LIN_DW, d->act, MOK_EPI_NONE, P, d->K, d->M)));
  w.bytes = o;
  return w;
}

}  // namespace

// A pointer that may be NULL, aligned when it is not.
#define MOK_OPTIONAL(p)                                            \
  do {                                                             \
    if ((p) != nullptr && !aligned16(p)) return MOK_ERR_ALIGN;     \
  } while (0)

extern "C" {

mok_status mok_norm_workspace_query(const mok_norm_desc* d, size_t* bwd_ws) {
  mok_status st = check_norm(d);
  if (st != MOK_OK) return st;
  if (bwd_ws == nullptr) return MOK_ERR_NULL;
  *bwd_ws = up(4 * (size_t)norm_parts(d->T, d->H, d->act) * d->H);
  return MOK_OK;
}

mok_status mok_rmsnorm_forward(const mok_norm_desc* d, const void* x, const void* res, const void* w, void* r, void* y,
                               void* q, void* s, float* rstd, void* stream) {
  mok_status st = check_norm(d);
  if (st != MOK_OK) return st;
  if (d->T == 0) return MOK_OK;  // empty arrays may be NULL
  const bool mx = d->quant != d->act;
  MOK_REQUIRE(x);
  MOK_OPTIONAL(res);
  MOK_REQUIRE(w);
  MOK_OPTIONAL(r);
  if (mx) {
    MOK_OPTIONAL(y);
    MOK_REQUIRE(q);
    MOK_REQUIRE(s);
  } else {
    MOK_REQUIRE(y);
  }
  MOK_OPTIONAL(rstd);
  NormArgs a{};
  a.T = d->T;
  a.H = d->H;
  a.eps = d->eps;
  a.x = x;
  a.res = res;
  a.w = w;
  a.r = r;
  a.y = y;
  a.q = (uint8_t*)q;
  a.s = (uint8_t*)s;
  a.rstd = rstd;
  MOK_LAUNCH("norm", (hipStream_t)stream, launch_norm_fwd(a, d->act, d->quant, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_rmsnorm_backward(const mok_norm_desc* d, const void* dy, const void* dr, const void* r, const void* w,
                                const float* rstd, void* dx, void* dw, void* ws, size_t ws_bytes, void* stream) {
  size_t want = 0;
  mok_status st = mok_norm_workspace_query(d, &want);
  if (st != MOK_OK) return st;
  if (dw != nullptr && (st = need(ws_bytes, want)) != MOK_OK) return st;
  MOK_OPTIONAL(dw);
  if (d->T > 0) {
    MOK_REQUIRE(dy);
    MOK_OPTIONAL(dr);
    MOK_REQUIRE(r);
    MOK_REQUIRE(w);
    MOK_REQUIRE(rstd);
    MOK_REQUIRE(dx);
    if (dw != nullptr) MOK_REQUIRE(ws);
    NormArgs a{};
    a.T = d->T;
    a.H = d->H;
    a.w = w;
    a.r = const_cast<void*>(r);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dr = dr;
    a.dx = dx;
    a.part = dw != nullptr ? (float*)ws : nullptr;
    MOK_LAUNCH("norm", (hipStream_t)stream, launch_norm_bwd(a, d->act, (hipStream_t)stream));
  }
  if (dw != nullptr)
    MOK_LAUNCH("norm", (hipStream_t)stream,
               launch_col_sum((const float*)ws, norm_parts(d->T, d->H, d->act), d->H, dw,
                              d->act == MOK_F32 || (d->flags & MOK_FLAG_WGRAD_F32) != 0, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_balance_workspace_query(const mok_balance_desc* d, size_t* fwd_ws) {
  mok_status st = check_balance(d);
  if (st != MOK_OK) return st;
  if (fwd_ws == nullptr) return MOK_ERR_NULL;
  *fwd_ws = balance_ws(d->T, d->E, std::max(d->S, 1)).bytes;
  return MOK_OK;
}

mok_status mok_balance_forward(const mok_balance_desc* d, const float* logits, const int32_t* idx, const int32_t* seg,
                               const uint8_t* mask, float* loss, int32_t* counts, int32_t* tokens, float* prob,
                               float* stat, void* ws, size_t ws_bytes, void* stream) {
  size_t want = 0;
  mok_status st = mok_balance_workspace_query(d, &want);
  if (st != MOK_OK) return st;
  if ((st = need(ws_bytes, want)) != MOK_OK) return st;
  if (d->T > 0) {
    MOK_REQUIRE(logits);
    MOK_REQUIRE(idx);
    MOK_REQUIRE(stat);
  }
  if (d->S > 0) MOK_REQUIRE(seg);
  MOK_OPTIONAL(mask);
  MOK_REQUIRE(loss);
  MOK_REQUIRE(counts);
  MOK_REQUIRE(tokens);
  MOK_REQUIRE(prob);
  MOK_REQUIRE(ws);
  BalanceArgs a = balance_args(d, logits, seg, mask);
  const BalanceWs w = balance_ws(a.T, a.E, a.S);
  char* wb = (char*)ws;
  a.rows = w.rows;
  a.chunks = w.chunks;
  a.idx = idx;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.prob = prob;
  a.stat = stat;
  a.wq = (float*)(wb + w.q);
  a.wc = (int32_t*)(wb + w.c);
  a.wn = (int32_t*)(wb + w.n);
  a.wz = (float*)(wb + w.z);
  a.done = (int32_t*)(wb + w.done);
  a.wl = (double*)(wb + w.loss);
  MOK_LAUNCH("balance", (hipStream_t)stream, launch_balance_fwd(a, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_balance_backward(const mok_balance_desc* d, const float* logits, const int32_t* seg, const uint8_t* mask,
                                const int32_t* counts, const int32_t* tokens, const float* stat, const float* dloss,
                                void* dlogits, void* stream) {
  mok_status st = check_balance(d);
  if (st != MOK_OK) return st;
  if (d->T == 0) return MOK_OK;  // empty arrays may be NULL
  MOK_REQUIRE(logits);
  if (d->S > 0) MOK_REQUIRE(seg);
  MOK_OPTIONAL(mask);
  MOK_REQUIRE(counts);
  MOK_REQUIRE(tokens);
  MOK_REQUIRE(stat);
  MOK_REQUIRE(dloss);
  MOK_REQUIRE(dlogits);
  BalanceArgs a = balance_args(d, logits, seg, mask);
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.stat = const_cast<float*>(stat);
  a.dloss = dloss;
  a.dlogits = dlogits;
  MOK_LAUNCH("balance", (hipStream_t)stream, launch_balance_bwd(a, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_linear_workspace_query(const mok_linear_desc* d, mok_linear_sizes* sizes) {
  mok_status st = check_linear(d);
  if (st != MOK_OK) return st;
  if (sizes == nullptr) return MOK_ERR_NULL;
  sizes->fwd_ws = up(linear_part_bytes(LIN_FWD, d->act, d->epi, d->M, d->N, d->K));
  sizes->bwd_ws = linear_bwd(d).bytes;
  return MOK_OK;
}

mok_status mok_linear_forward(const mok_linear_desc* d, const void* x, const void* w, const float* bias,
                              const void* res, void* y, void* pre, void* ws, size_t ws_bytes, void* stream) {
  mok_linear_sizes sz;
  mok_status st = mok_linear_workspace_query(d, &sz);
  if (st != MOK_OK) return st;
  if ((st = need(ws_bytes, sz.fwd_ws)) != MOK_OK) return st;
  if (d->M == 0) return MOK_OK;  // empty arrays may be NULL
  MOK_REQUIRE(x);
  MOK_REQUIRE(w);
  MOK_OPTIONAL(bias);
  MOK_OPTIONAL(res);
  MOK_REQUIRE(y);
  MOK_OPTIONAL(pre);
  if (sz.fwd_ws > 0) MOK_REQUIRE(ws);
  LinearArgs a{};
  a.a = x;
  a.b = w;
  a.M = d->M;
  a.N = d->N;
  a.K = d->K;
  a.bias = bias;
  a.add = res;
  a.out = y;
  a.pre = pre;
  a.part = (float*)ws;
  MOK_LAUNCH("linear", (hipStream_t)stream,
             launch_linear(a, LIN_FWD, d->act, d->epi, d->act == MOK_F32, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_linear_backward(const mok_linear_desc* d, const void* dy, const void* pre, const void* x, const void* w,
                               const void* dx_add, const void* dw_add, void* dx, void* dw, float* db, void* ws,
                               size_t ws_bytes, void* stream) {
  mok_status st = check_linear(d);
  if (st != MOK_OK) return st;
  const LinearBwd L = linear_bwd(d);
  if ((st = need(ws_bytes, L.bytes)) != MOK_OK) return st;
  const bool f = d->epi != MOK_EPI_NONE;
  MOK_OPTIONAL(dx_add);
  MOK_OPTIONAL(dw_add);
  MOK_OPTIONAL(dx);
  MOK_OPTIONAL(dw);
  MOK_OPTIONAL(db);
  if (d->M > 0) {
    MOK_REQUIRE(dy);
    if (f) MOK_REQUIRE(pre);
    if (dx != nullptr) MOK_REQUIRE(w);
    if (dw != nullptr) MOK_REQUIRE(x);
  }
  if (L.bytes > 0) MOK_REQUIRE(ws);
  const int P = linear_p(d);
  const hipStream_t s = (hipStream_t)stream;
  char* wb = (char*)ws;
  const void* dp = f ? wb + L.dp : dy;
  float* dbp = db != nullptr ? (float*)(wb + L.db) : nullptr;
  if (d->M > 0 && ((f && (dx != nullptr || dw != nullptr)) || db != nullptr))
    MOK_LAUNCH("linear", s, launch_linear_dpre(dy, pre, d->M, d->N, d->act, d->epi, f ? wb + L.dp : nullptr, dbp, s));
  if (db != nullptr) MOK_LAUNCH("linear", s, launch_col_sum(dbp, linear_db_parts(d->M, d->N), P, db, true, s));
  LinearArgs a{};
  a.a = dp;
  a.N = d->K;
  a.part = (float*)(wb + L.part);
  if (dx != nullptr && d->M > 0) {
    a.b = w;
    a.M = d->M;
    a.K = P;
    a.add = dx_add;
    a.out = dx;
    MOK_LAUNCH("linear", s, launch_linear(a, LIN_DX, d->act, MOK_EPI_NONE, d->act == MOK_F32, s));
  }
  if (dw != nullptr) {
    a.b = x;
    a.M = P;
    a.K = d->M;
    a.add = dw_add;
    a.out = dw;
    MOK_LAUNCH("linear", s, launch_linear(a, LIN_DW, d->act, MOK_EPI_NONE,
                                          d->act == MOK_F32 || (d->flags & MOK_FLAG_WGRAD_F32) != 0, s));
  }
  return MOK_OK;
}

}  // extern "C"
