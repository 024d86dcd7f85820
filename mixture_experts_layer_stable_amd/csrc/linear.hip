// Matrix product with bias, activation and residual in its epilogue, forward and backward.
#include "linear.h"

namespace mok {

namespace {

// ---- dp = dy f'(pre), and the parts of the bias gradient ----
// A thread keeps eight columns of dp and walks down the rows of its part; each input is read
// once and dp written once (HBM-bound). dp is rounded to the operands' type, in which the matrix units
// take both operands of dx's and dw's products (bf16: errors of 2.35e-3 of the norm, 1.7e-3 with the
// results' own rounding alone; dp as a sum of two bf16 would double the products). The bias gradient is
// summed ahead of that rounding, in fp32 over a part's rows and then over the parts.

template <typename T, int EPI>
__global__ __launch_bounds__(256) void linear_dpre_kernel(const T* __restrict__ dy, const T* __restrict__ pre,
                                                          int64_t M, int N, int64_t rows, T* __restrict__ dp,
                                                          float* __restrict__ part) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8, P = SW ? 2 * N : N;
  if (c >= N) return;
  const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = min(M, m0 + rows);
  float sg[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.0f;
#pragma unroll 4
  for (int64_t m = m0; m < m1; ++m) {
    float d[8], p[8], u[8];
    load8(dy + m * N + c, d);
    if constexpr (EPI != MOK_EPI_NONE) load8(pre + m * P + c, p);
    if constexpr (SW) load8(pre + m * P + N + c, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (EPI == MOK_EPI_SILU || SW) {
        const float s = sigmoid_t<T>(p[i]), f = s * (1.0f + p[i] * (1.0f - s));
        if constexpr (SW) {
          const float up = d[i] * p[i] * s;
          d[i] *= u[i] * f;
          u[i] = up;
        } else {
          d[i] *= f;
        }
      } else if constexpr (EPI == MOK_EPI_GELU) {
        d[i] *= phi_f(p[i]) + p[i] * 0.39894228040143268f * expf(-0.5f * p[i] * p[i]);
      }
      sg[i] += d[i];
      if constexpr (SW) su[i] += u[i];
    }
    if constexpr (EPI != MOK_EPI_NONE) store8(dp + m * P + c, d);
    if constexpr (SW) store8(dp + m * P + N + c, u);
  }
  if (part == nullptr) return;
  float* o = part + (int64_t)blockIdx.y * P + c;
  store8(o, sg);
  if constexpr (SW) store8(o + N, su);
}

// Rows of a part: the M rows go to about 2048 workgroups' worth of (256 x 8 columns, part). With sums
// to write, a part has 16 rows, so that its fp32 sums stay an eighth of what is read, or as few as 4
// where CUs would be left with fewer than two workgroups (2048 x (2 x 2048) with 16: 128 workgroups, 7 us
// more than with 8; without sums, 8192 rows: 512 workgroups 41.7 us, 2048 28.4, 5.9 TB/s).
int64_t dpre_rows(int64_t M, int N, bool sums) {
  const int64_t cols = (N + 2047) / 2048, parts = std::max<int64_t>(1, 2048 / cols);
  const int64_t least = sums ? std::min<int64_t>(16, std::max<int64_t>(4, M * cols / 512)) : 1;
  return std::max<int64_t>(least, (M + parts - 1) / parts);
}

template <typename T>
void run_dpre(const void* dy, const void* pre, int64_t M, int N, int epi, void* dp, float* part, hipStream_t s) {
  const int64_t rows = dpre_rows(M, N, part != nullptr);
  const dim3 grid((N + 2047) / 2048, (unsigned)((M + rows - 1) / rows)), block(256);
  const T *d = (const T*)dy, *p = (const T*)pre;
  if (epi == MOK_EPI_NONE)
    hipLaunchKernelGGL((linear_dpre_kernel<T, MOK_EPI_NONE>), grid, block, 0, s, d, p, M, N, rows, (T*)dp, part);
  else if (epi == MOK_EPI_SILU)
    hipLaunchKernelGGL((linear_dpre_kernel<T, MOK_EPI_SILU>), grid, block, 0, s, d, p, M, N, rows, (T*)dp, part);
  else if (epi == MOK_EPI_GELU)
    hipLaunchKernelGGL((linear_dpre_kernel<T, MOK_EPI_GELU>), grid, block, 0, s, d, p, M, N, rows, (T*)dp, part);
  else
    hipLaunchKernelGGL((linear_dpre_kernel<T, MOK_EPI_SWIGLU>), grid, block, 0, s, d, p, M, N, rows, (T*)dp, part);
}

}  // namespace

// The plan of least estimated time, with constants (us) fitted to 28 (bf16) and 17 (fp32) shapes
// from 1 to 16384 rows at every tile and split: the plan taken is the fastest or within a tenth of it.
// bf16: a tile's time is its K-tiles times what one takes (half as long on an empty chip as on a full
// one), plus a fixed part (first loads, epilogue); the tiles go out in rounds of as many as fit the
// 256 CUs. fp32, bound by its MFMAs: the K-tiles of the CU with the most tiles one after the other.
// Slices of K cost their fp32 partial products' way to memory and back, and a second launch. The 256 CUs
// are the whole chip's whatever the current device has: sizes of workspaces and orders of sums depend on
// the plan, and both are to be those of the shape alone.
LinearPlan linear_plan(int kind, int act, int epi, int64_t M, int N, int64_t K) {
  LinearPlan best{0, 1};
  if (M == 0) return best;
  struct Tile {
    int bm, bn, per_cu;
    double ktile, fixed;
  };
  static const Tile kTiles[4] = {
      {256, 256, 1, 1.55, 11.0}, {128, 128, 2, 0.97, 5.0}, {64, 128, 3, 1.1, 4.0}, {32, 128, 4, 1.2, 3.5}};
  static const Tile kTilesF32[2] = {{128, 128, 2, 1.75, 11.0}, {64, 64, 4, 0.45, 6.0}};  // K-tiles of 32
  static const Tile kTilesF32Sw[2] = {{128, 128, 2, 1.75, 11.0}, {64, 128, 3, 1.05, 6.0}};
  const bool f32 = act == MOK_F32;
  const int64_t P = epi == MOK_EPI_SWIGLU ? 2 * (int64_t)N : N, kt = f32 ? (K + 31) / 32 : (K + 63) / 64;
  double least = 1e30;
  for (int t = 0; t < (f32 ? 2 : 4); ++t) {
    const Tile& c = f32 ? (epi == MOK_EPI_SWIGLU ? kTilesF32Sw[t] : kTilesF32[t]) : kTiles[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((P + c.bn - 1) / c.bn), slots = 256 * c.per_cu;
    if (t > 0 && tiles >= (1 << 23)) continue;  // 2^32 threads a launch; the largest tile always fits
    for (int split = 1; split <= 256; split *= 2) {
      if (split > 1 && (kt / split < 2 || tiles * split >= (1 << 16))) break;
      const double rounds = (double)((tiles * split + slots - 1) / slots), kts = (double)((kt + split - 1) / split);
      const double bytes = 8.0 * split * (double)M * (double)P;  // of the partial products, written and read
      double us;
      if (f32) {
        us = (double)((tiles * split + 255) / 256) * kts * c.ktile + c.fixed + 2.5 * rounds;
        if (split > 1) us += 3.0 + bytes / 8e6;
      } else {
        const double fill = std::min(1.0, (double)(tiles * split) / (double)slots);
        us = rounds * (kts * c.ktile * (0.5 + 0.5 * fill) + c.fixed);
        if (split > 1) us += 5.0 + bytes / 4e6;
      }
      if (us < least) {
        least = us;
        best = {t, split};
      }
    }
  }
  // Up to 32 rows, forward: linear_few.hip's kernel takes a round of eight 256-byte pieces of K at a
  // time, `lat` us of latency each, or `full` when every CU has one of its workgroups; the tiles at
  // least the time of their operands' way from HBM.
  if (kind == LIN_FWD && M <= 32) {
    const double lat = M <= 16 ? (f32 ? 1.1 : 0.7) : (f32 ? 1.6 : 1.15);
    const double full = M <= 16 ? (f32 ? 1.6 : 1.35) : (f32 ? 2.5 : 2.0);
    const int64_t es = f32 ? 4 : 2, piece = 8 * (256 / es), rounds = (K + piece - 1) / piece;
    const double few = 4.0 + (double)rounds * std::max(lat, full * (double)((P + 15) / 16) / 256.0);
    if (few < std::max(least, (double)(es * P * K) / 5.4e6)) best = {kFewTile, 1};
  }
  return best;
}

size_t linear_part_bytes(int kind, int act, int epi, int64_t M, int N, int64_t K) {
  const int split = linear_plan(kind, act, epi, M, N, K).split;
  return split > 1 ? 4 * (size_t)split * (size_t)M * (epi == MOK_EPI_SWIGLU ? 2 * N : N) : 0;
}

hipError_t launch_linear(const LinearArgs& args, int kind, int act, int epi, bool out_f32, hipStream_t s) {
  LinearArgs a = args;
  const LinearPlan p = linear_plan(kind, act, epi, a.M, a.N, a.K);
  a.split = p.split;
  if (p.tile == kFewTile) return launch_linear_few(a, act, epi, s);
  if (act == MOK_BF16) return launch_linear_bf16(a, p.tile, kind, epi, out_f32, s);
  return launch_linear_f32(a, p.tile, kind, epi, s);
}

int linear_db_parts(int64_t M, int N) {
  if (M == 0) return 0;
  const int64_t rows = dpre_rows(M, N, true);
  return (int)((M + rows - 1) / rows);
}

hipError_t launch_linear_dpre(const void* dy, const void* pre, int64_t M, int N, int act, int epi, void* dp, float* part,
                              hipStream_t s) {
  if (act == MOK_F32) run_dpre<float>(dy, pre, M, N, epi, dp, part, s);
  else run_dpre<bf16>(dy, pre, M, N, epi, dp, part, s);
  return hipGetLastError();
}

}  // namespace mok
