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

}  // extern "C"
