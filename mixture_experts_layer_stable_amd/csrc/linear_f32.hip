// fp32 matrix products of linear.hip on the direct-to-LDS loop of linear_dense.h.
#include "linear_dense.h"

namespace mok {

namespace {

template <class Tl>
void run_f32(const LinearArgs& a, int kind, int epi, hipStream_t s) {
  if (kind == LIN_FWD) run_dense_fwd<float, Tl>(a, epi, s);
  else if (kind == LIN_DX) run_dense<float, Tl, LIN_DX, MOK_EPI_NONE, float>(a, s);
  else run_dense<float, Tl, LIN_DW, MOK_EPI_NONE, float>(a, s);
}

}  // namespace

hipError_t launch_linear_f32(const LinearArgs& a, int tile, int kind, int epi, hipStream_t s) {
  if (tile == 0) run_f32<Tiling<128, 128, 2, 2>>(a, kind, epi, s);
  else if (epi == MOK_EPI_SWIGLU) run_dense<float, Tiling<64, 128, 2, 2>, LIN_FWD, MOK_EPI_SWIGLU, float>(a, s);
  else run_f32<Tiling<64, 64, 2, 2>>(a, kind, epi, s);
  return hipGetLastError();
}

}  // namespace mok
