// Products with 4-bit weights and group scales (q4*.hip): launch interface and what the kernels share.
#pragma once
#include "grouped.h"
#include "linear.h"

namespace mok {

struct Q4Args {
  LinearArgs l;         // a = x, M, N, K, bias, add, out; b = codes [E][P][K / 2]
  const void* s;        // [E][P][K / group] in the operands' type
  const uint8_t* z;     // [E][P][K / group]; without zero points any readable bytes of that number
  bool zeros;           // false: 8 for every group
  const int32_t* off;   // [E + 1] or nullptr: one group of all rows
  int E, group, epi;
};
hipError_t launch_q4(const Q4Args& a, int act, hipStream_t s);
hipError_t launch_q4_few(const Q4Args& a, int act, hipStream_t s);
hipError_t launch_q4_tile(const Q4Args& a, int act, hipStream_t s);
// Slices of K in tiles of 128 x 128, or 0: q4_few.hip. A function of the shape and type only.
int q4_split(int act, int epi, int64_t M, int N, int K, int E);
hipError_t launch_q4_quantize(const void* w, int64_t rows, int K, int group, int act, void* q, void* s, uint8_t* z,
                              hipStream_t st);

inline int64_t q4_tiles_bound(const Q4Args& a, int bm) {
  return a.off == nullptr ? (a.l.M + bm - 1) / bm : group_tiles_bound(a.l.M, a.E, bm);
}

// y of eight columns from their products p (u: of the up columns).
template <typename T, bool SW>
__device__ __forceinline__ void q4_finish(LinearArgs a, const float* bias, int epi, int64_t m, int c, float (&p)[8],
                                          float (&u)[8], const Raw8<T>& add) {
  a.bias = bias;  // of the group
  if constexpr (SW) {
    linear_bias8<MOK_EPI_SWIGLU>(a, c, p, u);
    linear_store8<LIN_FWD, MOK_EPI_SWIGLU, T, T>(a, m, c, p, u, add);
  } else {
    linear_bias8<MOK_EPI_NONE>(a, c, p, u);
    if (epi == MOK_EPI_SILU) linear_store8<LIN_FWD, MOK_EPI_SILU, T, T>(a, m, c, p, u, add);
    else if (epi == MOK_EPI_GELU) linear_store8<LIN_FWD, MOK_EPI_GELU, T, T>(a, m, c, p, u, add);
    else linear_store8<LIN_FWD, MOK_EPI_NONE, T, T>(a, m, c, p, u, add);
  }
}

}  // namespace mok
