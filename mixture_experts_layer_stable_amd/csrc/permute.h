// Launch interface of the rows' way to the experts' order and back (permute.hip).
#pragma once
#include "common.h"

namespace mok {

struct PermuteArgs {
  int64_t T, R;
  int H, k;
  const void* in;       // dispatch: x [T][H]; combine: o [R][H]; combine backward: dy [T][H]
  const int32_t* perm;  // [R] or nullptr
  const int32_t* inv;   // [T][k]
  const float* gate;    // [T][k] or nullptr
  const void* add;      // [T][H] or nullptr
  void* out;            // dispatch, combine backward: [R][H]; combine: [T][H]
  const void* o;        // combine backward, with dgate
  float* dgate;         // combine backward, or nullptr
};
hipError_t launch_dispatch(const PermuteArgs& a, int act, hipStream_t s);
hipError_t launch_combine(const PermuteArgs& a, int act, hipStream_t s);
hipError_t launch_combine_bwd(const PermuteArgs& a, int act, hipStream_t s);

}  // namespace mok
