// bf16 matrix products of linear.hip on the direct-to-LDS loop of linear_dense.h.
#include "linear_dense.h"

namespace mok {

namespace {

constexpr int kBand = 8;  // tile rows of a band of the tile walk

// PART: the tile's sums over this slice of K go to a.part; linear_join_kernel adds the slices.
template <class Tl, int KIND, int EPI, typename TO, bool PART>
__global__ __launch_bounds__(Tl::NT) void linear_dense_kernel(LinearArgs a) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  // 256 x 256 tiles belong to outputs that no cache keeps: stored past L2, they leave it to the
  // operands' bands (16384 x (2 x 2048) x 7168: 818 -> 745 us)
  constexpr bool NTS = Tl::BM * Tl::BN >= 256 * 256;
  using OA = std::conditional_t<KIND == LIN_DW, DenseMN<Tl::BM, Tl::FM, Tl::NW>, DenseK<Tl::BM, Tl::FM, Tl::NW>>;
  using OB = std::conditional_t<KIND == LIN_FWD, DenseK<Tl::BN, Tl::FN, Tl::NW, SW>, DenseMN<Tl::BN, Tl::FN, Tl::NW>>;
  constexpr int PATCH = Tl::NW * 32 * kDensePatch * 4;
  constexpr int BST = Tl::BM * Tl::BN >= 256 * 256 ? 3 : 2;  // B's LDS stages
  constexpr int RING = DenseRing<OA, OB, BST>::BYTES;
  __shared__ __align__(1024) char smem[RING > PATCH ? RING : PATCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Tl::WN, wn = wave % Tl::WN;
  constexpr int BN = SW ? Tl::BN / 2 : Tl::BN;  // outputs of a tile's columns
  const int NT = (a.N + BN - 1) / BN, MT = (int)((a.M + Tl::BM - 1) / Tl::BM);
  // tile walk: consecutive workgroups of an XCD take a band of kBand tile rows column by column
  int L = xcd_logical(blockIdx.x, gridDim.x);
  const int slice = L / (MT * NT);
  L -= slice * MT * NT;
  const int band = L / (kBand * NT), gm = min(kBand, MT - band * kBand), r = L - band * kBand * NT;
  const int64_t m0 = (int64_t)(band * kBand + r % gm) * Tl::BM;
  const int n0 = (r / gm) * BN;
  const int64_t KT = (a.K + 63) / 64, kt0 = KT * slice / a.split, kt1 = KT * (slice + 1) / a.split;

  const auto frow_a = [&](int f) { return wm * Tl::WTM + f * 32; };
  const auto frow_b = [&](int f) { return wn * Tl::WTN + f * 32; };
  // first output column of tile column j (SWIGLU: 32-column blocks of gate and up in turn)
  const auto col = [&](int j) { return SW ? n0 + (j / 64) * 32 + (j & 31) : n0 + j; };
  const bf16* A = (const bf16*)a.a;
  const bf16* B = (const bf16*)a.b;
  OA oa;
  OB ob;
  if constexpr (KIND == LIN_DW) {
    oa.init(A + m0, 2 * a.M, a.K, a.M - m0, frow_a, wave, lane);
  } else {
    const int last = (int)min<int64_t>(a.M - 1 - m0, Tl::BM - 1);  // rows past M re-read the last one
    oa.init(A + m0 * a.K, 0, a.K, [&](int row) { return (uint32_t)min(row, last) * (uint32_t)(2 * a.K); }, frow_a, wave,
            lane);
  }
  if constexpr (KIND == LIN_FWD) {
    ob.init(B + (int64_t)n0 * a.K, 2 * (int64_t)a.N * a.K, a.K,
            [&](int j) { return (uint32_t)(min(col(j), a.N - 1) - n0) * (uint32_t)(2 * a.K); }, frow_b, wave, lane);
  } else {
    ob.init(B + n0, 2 * (int64_t)a.N, a.K, a.N - n0, frow_b, wave, lane);
  }
  f32x16_t acc[Tl::FM][Tl::FN];
  zero_acc<Tl>(acc);
  if (kt1 > kt0) dense_loop<Tl, BST>(oa, ob, kt0, kt1, smem, wave, acc);

  const auto in = [&](int row, int j) { return m0 + row < a.M && col(j) < a.N; };
  if constexpr (PART) {
    float* part = a.part + (int64_t)slice * a.M * (SW ? 2 * a.N : a.N);
    dense_epilogue<Tl, SW>(
        acc, smem, wave, wm, wn, lane, [](int, int) { return 0; },
        [&](auto, int row, int j, float (&g)[8], float (&u)[8], int) {
          if (!in(row, j)) return;
          float* p = part + (m0 + row) * (SW ? 2 * a.N : a.N) + col(j);
          store8(p, g);
          if constexpr (SW) store8(p + a.N, u);
        });
    return;
  }
  // bias of the eight columns that this lane stores of each block pair
  constexpr int LPR = SW ? 4 : 8;
  float bg[Tl::FN / 2][8], bu[Tl::FN / 2][8];
#pragma unroll
  for (int p = 0; p < Tl::FN / 2; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bg[p][i] = bu[p][i] = 0.0f;
    const int c = col(wn * Tl::WTN + 64 * p + (lane % LPR) * 8);
    if (KIND == LIN_FWD && c < a.N) linear_bias8<EPI>(a, c, bg[p], bu[p]);
  }
  dense_epilogue<Tl, SW>(
      acc, smem, wave, wm, wn, lane,
      [&](int row, int j) { return in(row, j) ? linear_add8<TO>(a, m0 + row, col(j)) : Raw8<TO>{}; },
      [&](auto pc, int row, int j, float (&g)[8], float (&u)[8], const Raw8<TO>& add) {
        if constexpr (KIND == LIN_FWD) {
          constexpr int p = decltype(pc)::value;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g[i] += bg[p][i];
            u[i] += bu[p][i];
          }
        }
        if (in(row, j)) linear_store8<KIND, EPI, TO, bf16, NTS>(a, m0 + row, col(j), g, u, add);
      });
}

template <class Tl, int KIND, int EPI, typename TO>
void run(const LinearArgs& a, hipStream_t s) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  const int bn = SW ? Tl::BN / 2 : Tl::BN;
  const int64_t tiles = (int64_t)((a.N + bn - 1) / bn) * ((a.M + Tl::BM - 1) / Tl::BM);
  const dim3 grid((unsigned)(tiles * a.split)), block(Tl::NT);
  if (a.split == 1) {
    hipLaunchKernelGGL((linear_dense_kernel<Tl, KIND, EPI, TO, false>), grid, block, 0, s, a);
    return;
  }
  hipLaunchKernelGGL((linear_dense_kernel<Tl, KIND, SW ? MOK_EPI_SWIGLU : MOK_EPI_NONE, bf16, true>), grid, block, 0, s,
                     a);
  linear_join<KIND, EPI, TO, bf16>(a, s);
}

template <class Tl>
void run_tile(const LinearArgs& a, int kind, int epi, bool out_f32, hipStream_t s) {
  if (kind == LIN_FWD) {
    if (epi == MOK_EPI_NONE) run<Tl, LIN_FWD, MOK_EPI_NONE, bf16>(a, s);
    else if (epi == MOK_EPI_SILU) run<Tl, LIN_FWD, MOK_EPI_SILU, bf16>(a, s);
    else if (epi == MOK_EPI_GELU) run<Tl, LIN_FWD, MOK_EPI_GELU, bf16>(a, s);
    else run<Tl, LIN_FWD, MOK_EPI_SWIGLU, bf16>(a, s);
  } else if (kind == LIN_DX) {
    run<Tl, LIN_DX, MOK_EPI_NONE, bf16>(a, s);
  } else if (out_f32) {
    run<Tl, LIN_DW, MOK_EPI_NONE, float>(a, s);
  } else {
    run<Tl, LIN_DW, MOK_EPI_NONE, bf16>(a, s);
  }
}

}  // namespace

hipError_t launch_linear_bf16(const LinearArgs& a, int tile, int kind, int epi, bool out_f32, hipStream_t s) {
  if (tile == 0) run_tile<Tiling<256, 256, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 1) run_tile<Tiling<128, 128, 2, 2>>(a, kind, epi, out_f32, s);
  else if (tile == 2) run_tile<Tiling<64, 128, 1, 2>>(a, kind, epi, out_f32, s);
  else run_tile<Tiling<32, 128, 1, 2>>(a, kind, epi, out_f32, s);
  return hipGetLastError();
}

}  // namespace mok
