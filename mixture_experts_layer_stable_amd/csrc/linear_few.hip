// Matrix products of linear.hip for a few rows (a decoding step's tokens).
#include "linear_few.h"

namespace mok {

namespace {

template <typename T, int EPI, int RT>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(LinearArgs a) {
  __shared__ __align__(16) float s_sum[kFewWaves][RT * 16][kFewLd];
  few_work<T, EPI, RT>(a, blockIdx.x, s_sum);
}

template <typename T, int EPI>
void run_few(const LinearArgs& a, hipStream_t s) {
  const int cols = EPI == MOK_EPI_SWIGLU ? 8 : 16;
  const dim3 grid((a.N + cols - 1) / cols), block(64 * kFewWaves);
  if (a.M <= 16) hipLaunchKernelGGL((linear_few_kernel<T, EPI, 1>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((linear_few_kernel<T, EPI, 2>), grid, block, 0, s, a);
}

template <typename T>
void run_few(const LinearArgs& a, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_few<T, MOK_EPI_NONE>(a, s);
  else if (epi == MOK_EPI_SILU) run_few<T, MOK_EPI_SILU>(a, s);
  else if (epi == MOK_EPI_GELU) run_few<T, MOK_EPI_GELU>(a, s);
  else run_few<T, MOK_EPI_SWIGLU>(a, s);
}

}  // namespace

hipError_t launch_linear_few(const LinearArgs& a, int act, int epi, hipStream_t s) {
  if (act == MOK_F32) run_few<float>(a, epi, s);
  else run_few<bf16>(a, epi, s);
  return hipGetLastError();
}

}  // namespace mok
