// Products with 4-bit weights and group scales: the quantiser, and the choice of a kernel.
#include "q4.h"

namespace mok {

namespace {

// A thread takes eight consecutive weights of a row, G / 8 threads a group. The scale is rounded to
// the operands' type before codes are formed with it, so that no code is off by that rounding; the
// divisions are fp32's own, rounded to nearest, and so are the codes (ties to even).
template <typename T, int G, bool ZERO>
__global__ __launch_bounds__(256) void q4_quantize_kernel(const T* __restrict__ w, int64_t groups, uint32_t* __restrict__ q,
                                                          T* __restrict__ s, uint8_t* __restrict__ z) {
  constexpr int LG = G / 8;
  const int64_t n = groups * LG, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {  // whole groups leave together
    float v[8];
    if constexpr (std::is_same<T, bf16>::value) {
      unpack(ldg16(w + 8 * i), v, (bf16*)nullptr);
    } else {
      float a[4], b[4];
      unpack(ldg16(w + 8 * i), a, (float*)nullptr);
      unpack(ldg16(w + 8 * i + 4), b, (float*)nullptr);
#pragma unroll
      for (int k = 0; k < 4; ++k) { v[k] = a[k]; v[4 + k] = b[k]; }
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) { lo = fminf(lo, v[k]); hi = fmaxf(hi, v[k]); }
#pragma unroll
    for (int o = 1; o < LG; o <<= 1) { lo = fminf(lo, __shfl_xor(lo, o)); hi = fmaxf(hi, __shfl_xor(hi, o)); }
    float sc = ZERO ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
    if constexpr (std::is_same<T, bf16>::value) sc = bf16_to_f32(f32_to_bf16(sc));
    float zp = 8.0f;
    if (ZERO && sc > 0.0f) zp = fminf(fmaxf(rintf(-lo / sc), 0.0f), 15.0f);
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = sc > 0.0f ? fminf(fmaxf(rintf(v[k] / sc) + zp, 0.0f), 15.0f) : zp;
      c |= (uint32_t)f << (4 * k);
    }
    q[i] = c;
    if (i % LG == 0) {
      Elem<T>::put(s, i / LG, sc);
      if (ZERO) z[i / LG] = (uint8_t)zp;
    }
  }
}

template <typename T, int G>
void run_quantize(const void* w, int64_t groups, void* q, void* s, uint8_t* z, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>((groups * (G / 8) + 255) / 256, 1 << 22)), block(256);
  if (z != nullptr)
    hipLaunchKernelGGL((q4_quantize_kernel<T, G, true>), grid, block, 0, st, (const T*)w, groups, (uint32_t*)q, (T*)s, z);
  else
    hipLaunchKernelGGL((q4_quantize_kernel<T, G, false>), grid, block, 0, st, (const T*)w, groups, (uint32_t*)q, (T*)s, z);
}

template <typename T>
void run_quantize(const void* w, int64_t rows, int K, int group, void* q, void* s, uint8_t* z, hipStream_t st) {
  const int64_t groups = rows * (K / group);
  if (group == 32) run_quantize<T, 32>(w, groups, q, s, z, st);
  else if (group == 64) run_quantize<T, 64>(w, groups, q, s, z, st);
  else run_quantize<T, 128>(w, groups, q, s, z, st);
}

}  // namespace

hipError_t launch_q4_quantize(const void* w, int64_t rows, int K, int group, int act, void* q, void* s, uint8_t* z,
                              hipStream_t st) {
  if (act == MOK_F32) run_quantize<float>(w, rows, K, group, q, s, z, st);
  else run_quantize<bf16>(w, rows, K, group, q, s, z, st);
  return hipGetLastError();
}

hipError_t launch_q4(const Q4Args& a, int act, hipStream_t s) {
  const int64_t rows = a.l.M / std::min<int64_t>(a.E, a.l.M);
  if (rows < 64) return launch_q4_few(a, act, s);
  return launch_q4_tile(a, act, rows < 256 ? 128 : 256, s);
}

}  // namespace mok
