// Matrix product with bias, activation and residual in its epilogue, forward and backward.
#include "linear.h"

namespace mok {

namespace {

// K-contiguous operand rows with a ragged K: 16-byte chunks at or past K read as zeros.
template <typename T, int ROWS>
struct KTailStager {
  static constexpr int VE = Elem<T>::VE;
  static constexpr int BKE = kRowBytes / (int)sizeof(T);
  static constexpr int NV = ROWS * 8 / kThreads;
  const T* ptr[NV];
  uint4 r[NV];
  int64_t K;
  int tid;
  // rowptr(row): start of the row, or nullptr for a row of zeros
  template <class F> __device__ __forceinline__ void init(int tid_, int64_t K_, F rowptr) {
    tid = tid_;
    K = K_;
#pragma unroll
    for (int v = 0; v < NV; ++v) ptr[v] = rowptr((tid + v * kThreads) >> 3);
  }
  __device__ __forceinline__ void load(int kt) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t k = (int64_t)kt * BKE + ((tid + v * kThreads) & 7) * VE;
      r[v] = ptr[v] != nullptr && k < K ? ldg16(ptr[v] + k) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = tid + v * kThreads;
      *reinterpret_cast<uint4*>(lds + lds_off(i >> 3, i & 7)) = r[v];
    }
  }
};

// MN-contiguous operand: element (k, mn) at base[k * ld + mn], zeros outside.
template <typename T>
struct MnSource {
  const T* base;
  int64_t ld, K, MN, mn0;
  __device__ __forceinline__ uint4 operator()(int64_t k, int mn) const {
    return k < K && mn0 + mn < MN ? ldg16(base + k * ld + mn0 + mn) : make_uint4(0, 0, 0, 0);
  }
};

// One tile per workgroup: operands staged through registers into a double-buffered LDS tile
// (gemm.h). PART: the tile's sums over a slice of K, for linear_join_kernel.
template <class Tile, typename T, int KIND, int EPI, typename TO, bool PART>
__global__ __launch_bounds__(256) void linear_simple_kernel(LinearArgs a) {
  constexpr int PATCH = Tile::NW * 32 * kPatchLd * 4;  // the epilogue's
  __shared__ __align__(1024) char smem[Tile::LDS_BYTES > PATCH ? Tile::LDS_BYTES : PATCH];
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  constexpr int BKE = kRowBytes / (int)sizeof(T);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  constexpr int BN = SW ? Tile::BN / 2 : Tile::BN;  // outputs of a tile's columns
  const int NT = (a.N + BN - 1) / BN, MT = (int)((a.M + Tile::BM - 1) / Tile::BM);
  const int slice = blockIdx.x / (MT * NT), L = blockIdx.x - slice * (MT * NT);
  const int64_t m0 = (int64_t)(L / NT) * Tile::BM;
  const int n0 = (L % NT) * BN;
  const int64_t tiles = (a.K + BKE - 1) / BKE, kt0 = tiles * slice / a.split, kt1 = tiles * (slice + 1) / a.split;
  const int64_t k0 = kt0 * BKE, k1 = min(a.K, kt1 * BKE);  // this slice
  const int KT = (int)(kt1 - kt0);
  f32x16_t acc[Tile::FM][Tile::FN];
  const T* A = (const T*)a.a + (KIND == LIN_DW ? k0 * a.M : k0);
  const T* B = (const T*)a.b + (KIND == LIN_FWD ? k0 : k0 * a.N);
  // first output column of tile column j (SWIGLU: 32-column blocks of gate and up in turn)
  const auto col = [&](int j) { return SW ? n0 + (j / Tile::WTN) * (Tile::WTN / 2) + (j & 31) : n0 + j; };
  if constexpr (KIND == LIN_FWD) {
    KTailStager<T, Tile::BM> sa;
    sa.init(tid, k1 - k0, [&](int r) { return m0 + r < a.M ? A + (m0 + r) * a.K : nullptr; });
    KTailStager<T, Tile::BN> sb;
    sb.init(tid, k1 - k0, [&](int j) -> const T* {
      const int c = col(j);
      if (c >= a.N) return nullptr;
      return B + (int64_t)(SW && (j & 32) ? a.N + c : c) * a.K;
    });
    main_loop<T, Tile>(sa, sb, KT, smem, wm, wn, lane, acc);
  } else if constexpr (KIND == LIN_DX) {
    KTailStager<T, Tile::BM> sa;
    sa.init(tid, k1 - k0, [&](int r) { return m0 + r < a.M ? A + (m0 + r) * a.K : nullptr; });
    MNStager<T, Tile::BN, MnSource<T>> sb;
    sb.tid = tid;
    sb.src = MnSource<T>{B, a.N, k1 - k0, a.N, n0};
    main_loop<T, Tile>(sa, sb, KT, smem, wm, wn, lane, acc);
  } else {
    MNStager<T, Tile::BM, MnSource<T>> sa;
    sa.tid = tid;
    sa.src = MnSource<T>{A, a.M, k1 - k0, a.M, m0};
    MNStager<T, Tile::BN, MnSource<T>> sb;
    sb.tid = tid;
    sb.src = MnSource<T>{B, a.N, k1 - k0, a.N, n0};
    main_loop<T, Tile>(sa, sb, KT, smem, wm, wn, lane, acc);
  }
  __syncthreads();
  epilogue16<Tile, SW>(acc, smem, wave, wm, wn, lane,
                       [&](int row, int j, const float (&g)[16], const float (&u)[16]) {
    const int64_t m = m0 + row;
    if (m >= a.M) return;
    const int c = col(j), P = SW ? 2 * a.N : a.N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (c + 8 * h >= a.N) continue;
      float g8[8], u8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g8[i] = g[8 * h + i];
        u8[i] = SW ? u[8 * h + i] : 0.0f;
      }
      if constexpr (PART) {
        float* p = a.part + ((int64_t)slice * a.M + m) * P + c + 8 * h;
        store8(p, g8);
        if constexpr (SW) store8(p + a.N, u8);
        continue;
      }
      if constexpr (KIND == LIN_FWD) linear_bias8<EPI>(a, c + 8 * h, g8, u8);
      linear_store8<KIND, EPI, TO, T>(a, m, c + 8 * h, g8, u8, linear_add8<TO>(a, m, c + 8 * h));
    }
  });
}

template <class Tile, int KIND, int EPI>
void run_simple(const LinearArgs& a, hipStream_t s) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  const int bn = SW ? Tile::BN / 2 : Tile::BN;
  const dim3 grid((unsigned)((int64_t)((a.N + bn - 1) / bn) * ((a.M + Tile::BM - 1) / Tile::BM) * a.split));
  if (a.split == 1) {
    hipLaunchKernelGGL((linear_simple_kernel<Tile, float, KIND, EPI, float, false>), grid, dim3(256), 0, s, a);
    return;
  }
  hipLaunchKernelGGL((linear_simple_kernel<Tile, float, KIND, SW ? MOK_EPI_SWIGLU : MOK_EPI_NONE, float, true>), grid,
                     dim3(256), 0, s, a);
  linear_join<KIND, EPI, float, float>(a, s);
}

template <class Tile>
void run_f32(const LinearArgs& a, int kind, int epi, hipStream_t s) {
  if (kind == LIN_DX) run_simple<Tile, LIN_DX, MOK_EPI_NONE>(a, s);
  else if (kind == LIN_DW) run_simple<Tile, LIN_DW, MOK_EPI_NONE>(a, s);
  else if (epi == MOK_EPI_NONE) run_simple<Tile, LIN_FWD, MOK_EPI_NONE>(a, s);
  else if (epi == MOK_EPI_SILU) run_simple<Tile, LIN_FWD, MOK_EPI_SILU>(a, s);
  else if (epi == MOK_EPI_GELU) run_simple<Tile, LIN_FWD, MOK_EPI_GELU>(a, s);
  else if constexpr (Tile::FN % 2 == 0) run_simple<Tile, LIN_FWD, MOK_EPI_SWIGLU>(a, s);  // gate and up side by side
}

// ---- dp = dy f'(pre), and the parts of the bias gradient ----
// A thread keeps eight columns of dp and walks down the rows of its part; each input is read
// once and dp written once (HBM-bound).
constexpr int kDpreRows = 16;  // rows of a part, at least: its fp32 sums then stay an eighth of what is read

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
        const float s = sigmoid_f(p[i]), f = s * (1.0f + p[i] * (1.0f - s));
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

// Rows of a part: the M rows go to about 2048 workgroups' worth of (256 x 8 columns, part).
int64_t dpre_rows(int64_t M, int N) {
  const int64_t cols = (N + 2047) / 2048, parts = std::max<int64_t>(1, 2048 / cols);
  return std::max<int64_t>(kDpreRows, (M + parts - 1) / parts);
}

template <typename T>
void run_dpre(const void* dy, const void* pre, int64_t M, int N, int epi, void* dp, float* part, hipStream_t s) {
  const int64_t rows = dpre_rows(M, N);
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

// The plan of least estimated time. A tile's time is its K-tiles times what one takes (half as long
// on an empty chip as on a full one), plus a fixed part (first loads, epilogue); the tiles go out in
// rounds of as many as fit the 256 CUs. Slices of K cost their fp32 partial products' way to memory
// and back, and a second launch. The constants (us) are fitted
// to 28 shapes from 1 to 16384 rows at every tile and split: the plan taken is the fastest or within
// a tenth of it.
LinearPlan linear_plan(int kind, int act, int epi, int64_t M, int N, int64_t K) {
  LinearPlan best{0, 1};
  if (M == 0) return best;
  struct Tile {
    int bm, bn, per_cu;
    double ktile, fixed;
  };
  static const Tile kTiles[4] = {
      {256, 256, 1, 1.55, 11.0}, {128, 128, 2, 1.1, 5.0}, {64, 128, 3, 1.1, 4.0}, {32, 128, 4, 1.2, 3.5}};
  static const Tile kTilesF32[2] = {{128, 128, 2, 4.6, 6.0}, {64, 64, 4, 2.9, 5.0}};  // K-tiles of 32
  static const Tile kTilesF32Sw[2] = {{128, 128, 2, 4.6, 6.0}, {64, 128, 3, 3.6, 5.0}};
  const bool f32 = act == MOK_F32;
  const int64_t P = epi == MOK_EPI_SWIGLU ? 2 * (int64_t)N : N, kt = f32 ? (K + 31) / 32 : (K + 63) / 64;
  double least = 1e30;
  for (int t = 0; t < (f32 ? 2 : 4); ++t) {
    const Tile& c = f32 ? (epi == MOK_EPI_SWIGLU ? kTilesF32Sw[t] : kTilesF32[t]) : kTiles[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((P + c.bn - 1) / c.bn), slots = 256 * c.per_cu;
    if (t > 0 && tiles >= (1 << 23)) continue;  // 2^32 threads a launch; the largest tile always fits
    for (int split = 1; split <= 256; split *= 2) {
      if (split > 1 && (kt / split < 2 || tiles * split >= (1 << 16))) break;
      const double rounds = (double)((tiles * split + slots - 1) / slots);
      const double fill = std::min(1.0, (double)(tiles * split) / (double)slots);
      double us = rounds * ((double)((kt + split - 1) / split) * c.ktile * (0.5 + 0.5 * fill) + c.fixed);
      if (split > 1) us += 5.0 + 8.0 * split * (double)M * (double)P / 4e6;
      if (us < least) {
        least = us;
        best = {t, split};
      }
    }
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
  if (act == MOK_BF16) return launch_linear_bf16(a, p.tile, kind, epi, out_f32, s);
  if (p.tile == 0) run_f32<Tiling<128, 128, 2, 2>>(a, kind, epi, s);
  else if (epi == MOK_EPI_SWIGLU) run_simple<Tiling<64, 128, 2, 2>, LIN_FWD, MOK_EPI_SWIGLU>(a, s);
  else run_f32<Tiling<64, 64, 2, 2>>(a, kind, epi, s);
  return hipGetLastError();
}

int linear_db_parts(int64_t M, int N) {
  if (M == 0) return 0;
  const int64_t rows = dpre_rows(M, N);
  return (int)((M + rows - 1) / rows);
}

hipError_t launch_linear_dpre(const void* dy, const void* pre, int64_t M, int N, int act, int epi, void* dp, float* part,
                              hipStream_t s) {
  if (act == MOK_F32) run_dpre<float>(dy, pre, M, N, epi, dp, part, s);
  else run_dpre<bf16>(dy, pre, M, N, epi, dp, part, s);
  return hipGetLastError();
}

}  // namespace mok
