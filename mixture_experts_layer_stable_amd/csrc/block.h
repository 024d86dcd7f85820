// Launch interface between the C-ABI layer (api_block.hip) and the operators around the
// layer step (norm.hip).
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

}  // namespace mok
