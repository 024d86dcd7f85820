// Grouped products on the tiles of linear_dense.h: a workgroup finds its group and tile in the
// offsets, then does what a dense product's workgroup does on that group's operands.
#pragma once
#include "grouped.h"
#include "linear_dense.h"

namespace mok {

// Tiles of a launch: LIN_FWD, LIN_DX at most group_tiles_bound(M, E, BM) * NT, of which the offsets'
// own come first; LIN_DW E * MT * NT for each slice.
template <typename T, class Tl, int KIND, int EPI, typename TO, bool PART>
__global__ __launch_bounds__(Tl::NT) void grouped_dense_kernel(GroupedArgs ga) {
  using Cfg = DenseCfg<T, Tl, KIND, EPI>;
  __shared__ __align__(1024) char smem[Cfg::LDS];
  LinearArgs a = ga.l;
  const int NT = (a.N + Cfg::BN - 1) / Cfg::BN;
  const int64_t P = Cfg::SW ? 2 * (int64_t)a.N : a.N;
  int mt, nt;
  if constexpr (KIND == LIN_DW) {
    // a.M = rows of w, a.N its columns, a.K unused. An XCD takes kPiece consecutive tiles of one group, which
    // share its rows, and the pieces go around the XCDs: groups differ in rows, so an XCD with groups
    // of its own would finish before or behind the others.
    constexpr int kPiece = 64;
    const int MT = (int)((a.M + Tl::BM - 1) / Tl::BM), per = MT * NT;
    const int64_t tiles = (int64_t)per * ga.E * a.split;
    const int b = blockIdx.x, full = (int)(tiles / (8 * kPiece)) * (8 * kPiece);
    const int L = b < full ? (b / (8 * kPiece) * 8 + b % 8) * kPiece + b / 8 % kPiece : b;
    const int unit = L / per, g = unit % ga.E, slice = unit / ga.E;
    band_walk(L - unit * per, MT, NT, mt, nt);
    const int lo = group_clamp(ga.off[g], 0, (int)a.K), n = group_clamp(ga.off[g + 1], lo, (int)a.K) - lo;
    a.a = (const T*)a.a + (int64_t)lo * a.M;
    a.b = (const T*)a.b + (int64_t)lo * a.N;
    a.K = n;
    const int64_t o = (int64_t)g * a.M * a.N;
    a.out = (TO*)a.out + o;
    if (a.add != nullptr) a.add = (const TO*)a.add + o;
    const int64_t KT = (n + Cfg::BKE - 1) / Cfg::BKE, kt0 = KT * slice / a.split, kt1 = KT * (slice + 1) / a.split;
    dense_work<T, Tl, KIND, EPI, TO, PART>(a, (int64_t)mt * Tl::BM, nt * Cfg::BN, kt0, kt1,
                                           a.part + ((int64_t)slice * ga.E + g) * a.M * a.N, smem);
  } else {
    GroupScan scan;
    scan.init(ga.off, ga.E, a.M, Tl::BM);
    const int tiles = scan.total * NT;
    if ((int)blockIdx.x >= tiles) return;
    const int L = xcd_logical(blockIdx.x, tiles);
    const GroupTile t = scan.find(L / NT, Tl::BM);
    band_walk(L - t.first * NT, t.tiles, NT, mt, nt);
    a.M = t.hi;  // rows of other groups are neither read nor written
    a.b = (const T*)a.b + (int64_t)t.g * (KIND == LIN_FWD ? P * a.K : a.K * a.N);
    if (KIND == LIN_FWD && a.bias != nullptr) a.bias += t.g * P;
    const int64_t KT = (a.K + Cfg::BKE - 1) / Cfg::BKE;
    dense_work<T, Tl, KIND, EPI, TO, false>(a, t.lo + (int64_t)mt * Tl::BM, nt * Cfg::BN, 0, KT, nullptr, smem);
  }
}

template <typename T, class Tl, int KIND, int EPI, typename TO>
void run_grouped(const GroupedArgs& ga, hipStream_t s) {
  const LinearArgs& a = ga.l;
  const int bn = EPI == MOK_EPI_SWIGLU ? Tl::BN / 2 : Tl::BN;
  const int64_t nt = (a.N + bn - 1) / bn;
  if constexpr (KIND == LIN_DW) {
    const dim3 grid((unsigned)((a.M + Tl::BM - 1) / Tl::BM * nt * ga.E * a.split));
    if (a.split == 1) {
      hipLaunchKernelGGL((grouped_dense_kernel<T, Tl, KIND, EPI, TO, false>), grid, dim3(Tl::NT), 0, s, ga);
      return;
    }
    hipLaunchKernelGGL((grouped_dense_kernel<T, Tl, KIND, EPI, T, true>), grid, dim3(Tl::NT), 0, s, ga);
    LinearArgs j = a;  // all groups' rows of dw one after the other
    j.M = a.M * ga.E;
    linear_join<LIN_DW, MOK_EPI_NONE, TO, T>(j, s);
  } else {
    const dim3 grid((unsigned)(group_tiles_bound(a.M, ga.E, Tl::BM) * nt));
    hipLaunchKernelGGL((grouped_dense_kernel<T, Tl, KIND, EPI, TO, false>), grid, dim3(Tl::NT), 0, s, ga);
  }
}

template <typename T, class Tl>
void run_grouped_fwd(const GroupedArgs& a, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_grouped<T, Tl, LIN_FWD, MOK_EPI_NONE, T>(a, s);
  else if (epi == MOK_EPI_SILU) run_grouped<T, Tl, LIN_FWD, MOK_EPI_SILU, T>(a, s);
  else if (epi == MOK_EPI_GELU) run_grouped<T, Tl, LIN_FWD, MOK_EPI_GELU, T>(a, s);
  else if constexpr (Tl::FN % 2 == 0) run_grouped<T, Tl, LIN_FWD, MOK_EPI_SWIGLU, T>(a, s);  // gate and up side by side
}

}  // namespace mok
