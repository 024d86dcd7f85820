// Launch interface between the C-ABI layer (api_block.hip) and the operators around the
// layer step (norm.hip, balance.hip, linear.hip).
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
  size_t q, c, n, z, done, loss, bytes;
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
  int32_t* done;       // workgroups of the second launch that are through
  double* wl;          // [S][workgroups of a segment in the second launch] parts of the loss
  const float* dloss;
  void* dlogits;
};
hipError_t launch_balance_fwd(const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s);

// ---- matrix product with epilogue ----
enum LinearKind { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

// out[m][n] = sum_k A(m, k) B(n, k), m < M, n < N, k < K; ld in elements.
//   LIN_FWD  A = x rows, B = w rows (both K-contiguous); N counts the outputs y has; with
//            SWIGLU, B has 2N rows
//   LIN_DX   A = dp rows (K-contiguous), B(n, k) = w[k][n]
//   LIN_DW   A(m, k) = dp[k][m], B(n, k) = x[k][n]
struct LinearArgs {
  const void* a;
  const void* b;
  int64_t M, K;
  int N;
  const float* bias;  // LIN_FWD
  const void* add;    // [M][N] added to the result, or nullptr
  void* out;          // [M][N]
  void* pre;          // LIN_FWD: [M][P], or nullptr
  float* part;        // partial products of a split K: [split][M][P] fp32
  int split;          // set by launch_linear
};
// Tile and slices of K of a product: a function of the shape and type only, so that the sums are.
struct LinearPlan {
  int tile;   // 0..3: 256x256, 128x128, 64x128, 32x128 (bf16); 0, 1: 128x128, 64x64 (SWIGLU 64x128) (fp32); kFewTile
  int split;
};
constexpr int kFewTile = 4;  // linear_few.hip
LinearPlan linear_plan(int kind, int act, int epi, int64_t M, int N, int64_t K);
size_t linear_part_bytes(int kind, int act, int epi, int64_t M, int N, int64_t K);
hipError_t launch_linear(const LinearArgs& a, int kind, int act, int epi, bool out_f32, hipStream_t s);
hipError_t launch_linear_bf16(const LinearArgs& a, int tile, int kind, int epi, bool out_f32, hipStream_t s);
hipError_t launch_linear_few(const LinearArgs& a, int act, int epi, hipStream_t s);
hipError_t launch_linear_f32(const LinearArgs& a, int tile, int kind, int epi, hipStream_t s);

// dp = dy f'(pre) (epi != NONE; dp may be nullptr with NONE) and the column sums' parts
// [linear_db_parts][P] fp32 (nullptr: not formed)
int linear_db_parts(int64_t M, int N);
hipError_t launch_linear_dpre(const void* dy, const void* pre, int64_t M, int N, int act, int epi, void* dp, float* part,
                              hipStream_t s);

}  // namespace mok
