// bf16 matrix products of linear.hip on the direct-to-LDS loop of linear_dense.h.
#include "linear_dense.h"

namespace mok {

namespace {

template <class Tl>
void run_bf16(const LinearArgs& a, int kind, int epi, bool out_f32, hipStream_t s) {
  if (kind == LIN_FWD) run_dense_fwd<bf16, Tl>(a, epi, s);
  else if (kind == LIN_DX) run_dense<bf16, Tl, LIN_DX, MOK_EPI_NONE, bf16>(a, s);
  else if (out_f32) run_dense<bf16, Tl, LIN_DW, MOK_EPI_NONE, float>(a, s);
  else run_dense<bf16, Tl, LIN_DW, MOK_EPI_NONE, bf16>(a, s);
}

}  // namespace

hipError_t launch_linear_bf16(const LinearArgs& a, int tile, int kind, int epi, bool out_f32, hipStream_t s) {
  if (tile == 0) run_bf16<Tiling<256, 256, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 1) run_bf16<Tiling<128, 128, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 2) run_bf16<Tiling<64, 128, 1, 2>>(a, kind, epi, out_f32, s);
  else run_bf16<Tiling<32, 128, 1, 2>>(a, kind, epi, out_f32, s);
  return hipGetLastError();
}

}  // namespace mok
