// Launch interface between the C-ABI layer (api_block.hip) and the operators around the
// layer step (norm.hip, balance.hip).
#pragma once
#include "common.h"

namespace mok {

// ---- RMS norm ----
struct NormArgs {
  int64_t T;
  int H;
  float eps;
  const void* x;    // forward
  const void* res;  // forward, or nullptr
  const void* w;
  void* r;          // forward output or nullptr; backward input
  void* y;          // forward, or nullptr
  uint8_t* q;       // forward, MX only
  uint8_t* s;
  float* rstd;      // forward output or nullptr; backward input
  const void* dy;   // backward
  const void* dr;   // backward, or nullptr
  void* dx;
  float* part;      // backward: [norm_parts][H] fp32 partial sums of dw, or nullptr
};
// Workgroups of the backward pass and rows of its dw partials: a function of T and H only.
int norm_parts(int64_t T, int H, int act);
hipError_t launch_norm_fwd(const NormArgs& a, int act, int quant, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int act, hipStream_t s);

// out[h] = sum_p part[p][h] in fixed order, p < P (zero for P = 0); out as fp32 or bf16
hipError_t launch_col_sum(const float* part, int P, int H, void* out, bool f32, hipStream_t s);

// ---- balance loss ----
// Workspace of the forward: chunk c (rows c*rows ..) and segment s meet in at most one run of
// rows, and the pairs that meet form a staircase, so c + s names the pair.
struct BalanceWs {
  int chunks, rows;  // chunks of `rows` tokens
  size_t q, c, n, z, loss, bytes;
};
BalanceWs balance_ws(int64_t T, int E, int S);

struct BalanceArgs {
  int64_t T;
  int E, k, S;  // S >= 1
  int rows, chunks;
  bool sigmoid, bf16_grad;
  float coef, zcoef;
  const float* logits;
  const int32_t* idx;
  const int32_t* seg;  // nullptr: one segment of all tokens
  const uint8_t* mask; // or nullptr
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  float* prob;
  float* stat;
  float* wq;           // [chunks + S][E] sums of p
  int32_t* wc;         // [chunks + S][E] counts
  int32_t* wn;         // [chunks + S] tokens
  float* wz;           // [chunks] sums of lse^2
  double* wl;          // [S][ceil(E / 64)] parts of the loss
  const float* dloss;
  void* dlogits;
};
hipError_t launch_balance_fwd(const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s);

}  // namespace mok
