// bf16 grouped products on the tiles of linear_dense.h.
#include "grouped_dense.h"

namespace mok {

namespace {

template <class Tl>
void run_bf16(const GroupedArgs& a, int kind, int epi, bool out_f32, hipStream_t s) {
  if (kind == LIN_FWD) run_grouped_fwd<bf16, Tl>(a, epi, s);
  else if (kind == LIN_DX) run_grouped<bf16, Tl, LIN_DX, MOK_EPI_NONE, bf16>(a, s);
  else if (out_f32) run_grouped<bf16, Tl, LIN_DW, MOK_EPI_NONE, float>(a, s);
  else run_grouped<bf16, Tl, LIN_DW, MOK_EPI_NONE, bf16>(a, s);
}

}  // namespace

hipError_t launch_grouped_bf16(const GroupedArgs& a, int tile, int kind, int epi, bool out_f32, hipStream_t s) {
  if (tile == kShortTile) {
    if (out_f32) run_grouped_short_dw<float>(a, s);
    else run_grouped_short_dw<bf16>(a, s);
  } else if (tile == 0) run_bf16<Tiling<256, 256, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 1) run_bf16<Tiling<128, 128, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 2) run_bf16<Tiling<64, 128, 1, 2>>(a, kind, epi, out_f32, s);
  else run_bf16<Tiling<32, 128, 1, 2>>(a, kind, epi, out_f32, s);
  return hipGetLastError();
}

}  // namespace mok
