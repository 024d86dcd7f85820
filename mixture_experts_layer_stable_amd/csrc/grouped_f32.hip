// fp32 grouped products on the tiles of linear_dense.h.
#include "grouped_dense.h"

namespace mok {

namespace {

template <class Tl>
void run_f32(const GroupedArgs& a, int kind, int epi, hipStream_t s) {
  if (kind == LIN_FWD) run_grouped_fwd<float, Tl>(a, epi, s);
  else if (kind == LIN_DX) run_grouped<float, Tl, LIN_DX, MOK_EPI_NONE, float>(a, s);
  else run_grouped<float, Tl, LIN_DW, MOK_EPI_NONE, float>(a, s);
}

}  // namespace

hipError_t launch_grouped_f32(const GroupedArgs& a, int tile, int kind, int epi, hipStream_t s) {
  if (tile == 0) run_f32<Tiling<128, 128, 2, 2>>(a, kind, epi, s);
  else if (epi == MOK_EPI_SWIGLU) run_grouped<float, Tiling<64, 128, 2, 2>, LIN_FWD, MOK_EPI_SWIGLU, float>(a, s);
  else run_f32<Tiling<64, 64, 2, 2>>(a, kind, epi, s);
  return hipGetLastError();
}

}  // namespace mok
