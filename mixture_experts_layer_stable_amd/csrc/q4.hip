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

// The faster of the two kernels by estimates (us) fitted to shapes from 1 to 4096 rows. q4_few.hip: what 16 rows
// of a group take for a million codes (up to 2^27 rows, whose tiles GroupScan counts). Tiles: K-tiles (of 64,
// fp32 32) one after the other, half as long on an empty chip as on a full one, in rounds of 512 (fp32 256);
// slices of K, of a dense product only (a second launch that adds them would have to know the rows' groups),
// cost their partial products' way to memory and back. 2 x 2048 x 7168, measured on two cards: 64 rows 28 to 35 us,
// 128 31 to 36, 256 39 to 41, 512 62, 1024 98 to 103; the few-row kernel takes 19 for 16 rows, and 31 for 32 where tiles in
// slices, which those take now, need 25. The quantiser: 8 x 4096 x 7168 in 160 to 165 us bf16 (3.6 to 3.7 TB/s), 183 to 193 fp32 (5.6 to 5.8).
int q4_split(int act, int epi, int64_t M, int N, int K, int E) {
  if (M == 0) return 0;
  const bool f32 = act == MOK_F32;
  const double P = epi == MOK_EPI_SWIGLU ? 2.0 * N : N, groups = (double)std::min<int64_t>(E, M);
  const double row_tiles = std::max(groups, (double)M / 16 + 0.5 * groups), rows = (double)M / groups;
  double least = M > (1 << 27) ? 1e30 : 6.0 + row_tiles * P * K * 1e-6 * (f32 ? 0.75 : (rows > 4 ? 0.38 : 0.2));
  int best = 0;
  const double tiles = std::max(groups, (double)M / 128 + 0.5 * groups) * std::max(1.0, P / 128), slots = f32 ? 256 : 512;
  const int pieces = (K + 127) / 128;
  for (int split = 1; split <= (E == 1 ? 64 : 1); split *= 2) {
    if (split > 1 && (pieces / split < 2 || tiles * split >= 4096)) break;
    const double fill = std::min(1.0, tiles * split / slots), kts = (double)((pieces + split - 1) / split) * (f32 ? 4 : 2);
    double us = std::max(1.0, tiles * split / slots) * (kts * (f32 ? 2.0 : 1.45) * (0.6 + 0.4 * fill) + 6.0);
    if (split > 1) us += 5.0 + 8.0 * split * (double)M * P / 4e6;
    if (us < least) {
      least = us;
      best = split;
    }
  }
  return best;
}

hipError_t launch_q4(const Q4Args& args, int act, hipStream_t s) {
  Q4Args a = args;
  // E = 1 with offsets: rows outside the group are not to be written, so no slices
  const int split = q4_split(act, a.epi, a.l.M, a.l.N, (int)a.l.K, a.off == nullptr ? 1 : std::max(a.E, 2));
  if (split == 0) return launch_q4_few(a, act, s);
  a.l.split = split;
  if (split == 1) a.l.part = nullptr;
  return launch_q4_tile(a, act, s);
}

}  // namespace mok
