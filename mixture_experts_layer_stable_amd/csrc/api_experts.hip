// C-ABI entry points of the parts that an expert layer is built from: grouped products, products
// with 4-bit weights, dispatch and combine. Argument checks, workspace layouts, launches.
#include "api.h"
#include "permute.h"
#include "q4.h"

using namespace mok;

namespace {

// Sizes that the grouped and the 4-bit products share: every array below 2^37 elements (as large as the
// GPU's memory), and fewer output tiles than a launch has workgroups of 256 threads.
mok_status check_sizes(int64_t M, int32_t N, int32_t K, int32_t E, int32_t epi) {
  if (E < 1 || E > 1024) return MOK_ERR_SHAPE;
  if (M < 0 || M >= ((int64_t)1 << 30)) return MOK_ERR_SHAPE;
  if (N < 8 || N > (1 << 20) || N % 8 != 0) return MOK_ERR_SHAPE;
  if (K < 8 || K > (1 << 20) || K % 8 != 0) return MOK_ERR_SHAPE;
  const int64_t P = epi == MOK_EPI_SWIGLU ? 2LL * N : N, most = std::max<int64_t>(P, K);
  if (std::max<int64_t>(M, 1) * most >= (1LL << 37) || P * K >= (1LL << 37) / E) return MOK_ERR_SHAPE;
  if ((M / 128 + E) * ((most + 127) / 128) >= (1LL << 24)) return MOK_ERR_SHAPE;
  if (E * ((P + 127) / 128) * ((K + 127) / 128) >= (1LL << 24)) return MOK_ERR_SHAPE;
  return MOK_OK;
}

mok_status check_grouped(const mok_grouped_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->act != MOK_F32 && d->act != MOK_BF16) return MOK_ERR_DTYPE;
  if (d->epi < MOK_EPI_NONE || d->epi > MOK_EPI_SWIGLU) return MOK_ERR_DTYPE;
  if (d->reserved != 0 || (d->flags & ~MOK_FLAG_WGRAD_F32) != 0) return MOK_ERR_SHAPE;
  return check_sizes(d->M, d->N, d->K, d->E, d->epi);
}

int grouped_p(const mok_grouped_desc* d) { return d->epi == MOK_EPI_SWIGLU ? 2 * d->N : d->N; }

// Backward workspace: dp rows, bias-gradient parts, partial products of dw.
struct GroupedBwd {
  size_t dp, db, part, bytes;
};
GroupedBwd grouped_bwd(const mok_grouped_desc* d) {
  const int P = grouped_p(d);
  GroupedBwd w;
  size_t o = 0;
  w.dp = o; o = up(o + (d->epi == MOK_EPI_NONE ? 0 : (size_t)elem_size(d->act) * (size_t)d->M * P));
  w.db = o; o = up(o + 4 * (size_t)grouped_db_parts(d->M, d->N, d->E) * P);
  w.part = o; o = up(o + grouped_part_bytes(LIN_DW, d->act, MOK_EPI_NONE, P, d->K, d->M, d->E));
  w.bytes = o;
  return w;
}

mok_status check_q4(const mok_q4_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->act != MOK_F32 && d->act != MOK_BF16) return MOK_ERR_DTYPE;
  if (d->epi < MOK_EPI_NONE || d->epi > MOK_EPI_SWIGLU) return MOK_ERR_DTYPE;
  if (d->reserved != 0 || d->flags != 0) return MOK_ERR_SHAPE;
  if (d->group != 32 && d->group != 64 && d->group != 128) return MOK_ERR_SHAPE;
  if (d->K % d->group != 0) return MOK_ERR_SHAPE;
  return check_sizes(d->M, d->N, d->K, d->E, d->epi);
}

mok_status check_permute(const mok_permute_desc* d) {
  if (d == nullptr) return MOK_ERR_NULL;
  if (d->act != MOK_F32 && d->act != MOK_BF16) return MOK_ERR_DTYPE;
  if (d->reserved != 0) return MOK_ERR_SHAPE;
  if (d->k < 1 || d->k > 16) return MOK_ERR_SHAPE;
  if (d->H < 8 || d->H > (1 << 20) || d->H % 8 != 0) return MOK_ERR_SHAPE;
  if (d->T < 0 || d->T >= ((int64_t)1 << 31) || d->T * d->k >= ((int64_t)1 << 31)) return MOK_ERR_SHAPE;
  if (d->R < 0 || d->R >= ((int64_t)1 << 31)) return MOK_ERR_SHAPE;
  if (std::max(d->T, d->R) * d->H >= (1LL << 37)) return MOK_ERR_SHAPE;
  return MOK_OK;
}

PermuteArgs permute_args(const mok_permute_desc* d) {
  PermuteArgs a{};
  a.T = d->T;
  a.R = d->R;
  a.H = d->H;
  a.k = d->k;
  return a;
}

}  // namespace

// A pointer that may be NULL, aligned when it is not.
#define MOK_OPTIONAL(p)                                            \
  do {                                                             \
    if ((p) != nullptr && !aligned16(p)) return MOK_ERR_ALIGN;     \
  } while (0)

extern "C" {

mok_status mok_grouped_workspace_query(const mok_grouped_desc* d, mok_linear_sizes* sizes) {
  mok_status st = check_grouped(d);
  if (st != MOK_OK) return st;
  if (sizes == nullptr) return MOK_ERR_NULL;
  sizes->fwd_ws = 0;
  sizes->bwd_ws = grouped_bwd(d).bytes;
  return MOK_OK;
}

mok_status mok_grouped_forward(const mok_grouped_desc* d, const void* x, const void* w, const float* bias,
                               const int32_t* off, const void* res, void* y, void* pre, void* ws, size_t ws_bytes,
                               void* stream) {
  mok_linear_sizes sz;
  mok_status st = mok_grouped_workspace_query(d, &sz);
  if (st != MOK_OK) return st;
  if ((st = need(ws_bytes, sz.fwd_ws)) != MOK_OK) return st;
  if (d->M == 0) return MOK_OK;  // empty arrays may be NULL
  MOK_REQUIRE(x);
  MOK_REQUIRE(w);
  MOK_OPTIONAL(bias);
  MOK_REQUIRE(off);
  MOK_OPTIONAL(res);
  MOK_REQUIRE(y);
  MOK_OPTIONAL(pre);
  if (sz.fwd_ws > 0) MOK_REQUIRE(ws);
  GroupedArgs a{};
  a.l.a = x;
  a.l.b = w;
  a.l.M = d->M;
  a.l.N = d->N;
  a.l.K = d->K;
  a.l.bias = bias;
  a.l.add = res;
  a.l.out = y;
  a.l.pre = pre;
  a.off = off;
  a.E = d->E;
  MOK_LAUNCH("grouped", (hipStream_t)stream,
             launch_grouped(a, LIN_FWD, d->act, d->epi, d->act == MOK_F32, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_grouped_backward(const mok_grouped_desc* d, const void* dy, const void* pre, const void* x,
                                const void* w, const int32_t* off, const void* dx_add, const void* dw_add, void* dx,
                                void* dw, float* db, void* ws, size_t ws_bytes, void* stream) {
  mok_status st = check_grouped(d);
  if (st != MOK_OK) return st;
  const GroupedBwd L = grouped_bwd(d);
  if ((st = need(ws_bytes, L.bytes)) != MOK_OK) return st;
  const bool f = d->epi != MOK_EPI_NONE;
  MOK_REQUIRE(off);
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
  const int P = grouped_p(d);
  const hipStream_t s = (hipStream_t)stream;
  char* wb = (char*)ws;
  const void* dp = f ? wb + L.dp : dy;
  float* dbp = db != nullptr ? (float*)(wb + L.db) : nullptr;
  if (d->M > 0 && ((f && (dx != nullptr || dw != nullptr)) || db != nullptr))
    MOK_LAUNCH("grouped", s,
               launch_grouped_dpre(dy, pre, off, d->M, d->N, d->E, d->act, d->epi, f ? wb + L.dp : nullptr, dbp, s));
  if (db != nullptr) MOK_LAUNCH("grouped", s, launch_grouped_db(dbp, off, d->M, d->N, P, d->E, db, s));
  GroupedArgs a{};
  a.l.a = dp;
  a.l.N = d->K;
  a.l.part = (float*)(wb + L.part);
  a.off = off;
  a.E = d->E;
  if (dx != nullptr && d->M > 0) {
    a.l.b = w;
    a.l.M = d->M;
    a.l.K = P;
    a.l.add = dx_add;
    a.l.out = dx;
    MOK_LAUNCH("grouped", s, launch_grouped(a, LIN_DX, d->act, MOK_EPI_NONE, d->act == MOK_F32, s));
  }
  if (dw != nullptr) {
    a.l.b = x;
    a.l.M = P;
    a.l.K = d->M;
    a.l.add = dw_add;
    a.l.out = dw;
    MOK_LAUNCH("grouped", s, launch_grouped(a, LIN_DW, d->act, MOK_EPI_NONE,
                                            d->act == MOK_F32 || (d->flags & MOK_FLAG_WGRAD_F32) != 0, s));
  }
  return MOK_OK;
}

mok_status mok_q4_workspace_query(const mok_q4_desc* d, size_t* fwd_ws) {
  mok_status st = check_q4(d);
  if (st != MOK_OK) return st;
  if (fwd_ws == nullptr) return MOK_ERR_NULL;
  const int split = d->E == 1 ? q4_split(d->act, d->epi, d->M, d->N, d->K, 1) : 0;
  *fwd_ws = split > 1 ? up(4 * (size_t)split * (size_t)d->M * (d->epi == MOK_EPI_SWIGLU ? 2 * d->N : d->N)) : 0;
  return MOK_OK;
}

mok_status mok_q4_quantize(const mok_q4_desc* d, const void* w, void* q, void* s, uint8_t* z, void* stream) {
  mok_status st = check_q4(d);
  if (st != MOK_OK) return st;
  MOK_REQUIRE(w);
  MOK_REQUIRE(q);
  MOK_REQUIRE(s);
  MOK_OPTIONAL(z);
  const int64_t rows = (int64_t)d->E * (d->epi == MOK_EPI_SWIGLU ? 2 * d->N : d->N);
  MOK_LAUNCH("q4", (hipStream_t)stream,
             launch_q4_quantize(w, rows, d->K, d->group, d->act, q, s, z, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_q4_forward(const mok_q4_desc* d, const void* x, const void* q, const void* s, const uint8_t* z,
                          const float* bias, const int32_t* off, const void* res, void* y, void* ws, size_t ws_bytes,
                          void* stream) {
  size_t want = 0;
  mok_status st = mok_q4_workspace_query(d, &want);
  if (st != MOK_OK) return st;
  if ((st = need(ws_bytes, want)) != MOK_OK) return st;
  if (d->M == 0) return MOK_OK;  // empty arrays may be NULL
  MOK_REQUIRE(x);
  MOK_REQUIRE(q);
  MOK_REQUIRE(s);
  MOK_OPTIONAL(z);
  MOK_OPTIONAL(bias);
  if (d->E > 1) MOK_REQUIRE(off);
  MOK_OPTIONAL(off);
  MOK_OPTIONAL(res);
  MOK_REQUIRE(y);
  if (want > 0) MOK_REQUIRE(ws);
  Q4Args a{};
  a.l.a = x;
  a.l.b = q;
  a.l.M = d->M;
  a.l.N = d->N;
  a.l.K = d->K;
  a.l.bias = bias;
  a.l.add = res;
  a.l.out = y;
  a.l.part = (float*)ws;
  a.s = s;
  a.z = z != nullptr ? z : (const uint8_t*)s;
  a.zeros = z != nullptr;
  a.off = off;
  a.E = d->E;
  a.group = d->group;
  a.epi = d->epi;
  MOK_LAUNCH("q4", (hipStream_t)stream, launch_q4(a, d->act, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_dispatch_forward(const mok_permute_desc* d, const void* x, const int32_t* perm, void* xs, void* stream) {
  mok_status st = check_permute(d);
  if (st != MOK_OK) return st;
  if (d->R == 0) return MOK_OK;  // empty arrays may be NULL
  if (d->T > 0) MOK_REQUIRE(x);
  MOK_REQUIRE(perm);
  MOK_REQUIRE(xs);
  PermuteArgs a = permute_args(d);
  a.in = x;
  a.perm = perm;
  a.out = xs;
  MOK_LAUNCH("permute", (hipStream_t)stream, launch_dispatch(a, d->act, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_combine_forward(const mok_permute_desc* d, const void* o, const float* gate, const int32_t* inv,
                               const void* res, void* y, void* stream) {
  mok_status st = check_permute(d);
  if (st != MOK_OK) return st;
  if (d->T == 0) return MOK_OK;  // empty arrays may be NULL
  if (d->R > 0) MOK_REQUIRE(o);
  MOK_OPTIONAL(gate);
  MOK_REQUIRE(inv);
  MOK_OPTIONAL(res);
  MOK_REQUIRE(y);
  PermuteArgs a = permute_args(d);
  a.in = o;
  a.gate = gate;
  a.inv = inv;
  a.add = res;
  a.out = y;
  MOK_LAUNCH("permute", (hipStream_t)stream, launch_combine(a, d->act, (hipStream_t)stream));
  return MOK_OK;
}

mok_status mok_dispatch_backward(const mok_permute_desc* d, const void* dxs, const int32_t* inv, const void* dx_add,
                                 void* dx, void* stream) {
  return mok_combine_forward(d, dxs, nullptr, inv, dx_add, dx, stream);
}

mok_status mok_combine_backward(const mok_permute_desc* d, const void* dy, const void* o, const float* gate,
                                const int32_t* inv, const int32_t* perm, void* d_o, float* dgate, void* stream) {
  mok_status st = check_permute(d);
  if (st != MOK_OK) return st;
  if (d->T == 0 && (d->R == 0 || perm == nullptr)) return MOK_OK;  // empty arrays may be NULL
  if (d->T > 0) {
    MOK_REQUIRE(dy);
    MOK_REQUIRE(inv);
  }
  MOK_OPTIONAL(gate);
  MOK_OPTIONAL(perm);
  MOK_OPTIONAL(dgate);
  if (d->R > 0) {
    if (dgate != nullptr) MOK_REQUIRE(o);
    MOK_REQUIRE(d_o);
  }
  PermuteArgs a = permute_args(d);
  a.in = dy;
  a.o = o;
  a.gate = gate;
  a.inv = inv;
  a.perm = perm;
  a.out = d_o;
  a.dgate = dgate;
  MOK_LAUNCH("permute", (hipStream_t)stream, launch_combine_bwd(a, d->act, (hipStream_t)stream));
  return MOK_OK;
}

}  // extern "C"
