// Grouped products on the tiles of linear_dense.h: a workgroup finds its group and tile in the
// offsets, then does what a dense product's workgroup does on that group's operands.
#pragma once
#include "grouped.h"
#include "linear_dense.h"

namespace mok {

// The weight gradient's tile of this workgroup (MT x NT a group, all groups, slice after slice). An XCD takes kPiece
// consecutive tiles, which share their group's rows, and the pieces go around the XCDs: groups differ in
// rows, so an XCD with groups of its own would finish before or behind the others.
__device__ __forceinline__ void dw_tile(const GroupedArgs& ga, int MT, int NT, int& g, int& slice, int& mt, int& nt) {
  constexpr int kPiece = 64;
  const int per = MT * NT, tiles = per * ga.E * ga.l.split;
  const int b = blockIdx.x, full = tiles / (8 * kPiece) * (8 * kPiece);
  const int L = b < full ? (b / (8 * kPiece) * 8 + b % 8) * kPiece + b / 8 % kPiece : b;
  const int unit = L / per;
  g = unit % ga.E;
  slice = unit / ga.E;
  band_walk(L - unit * per, MT, NT, mt, nt);
}

// ---- weight gradients of bf16 groups of some hundred rows ----
// A group's K is its rows: a handful of K-tiles, and then a tile's worth of output. With one workgroup a CU nothing
// runs during that epilogue and the next tile's first loads. So two share a CU: 256 x 128 tiles, K-tiles of
// 32 rows in three stages (72 KB), one's matrix instructions under the other's stores. 16384 rows of 48
// groups, 4096 x 7168 each: 1540 us with 256 x 256 tiles, 1360 so (1150 without its stores; the first loads'
// latency, a dependent chain from the offsets on, is what is left: 5.7 us a tile). One stream of K-tiles
// over a workgroup's tiles, stored from the accumulators without a patch, would hide it, but loads
// that have to tell the last K-tile of a group from others cost more: 1600.
template <class Tl>
struct ShortDw {
  static constexpr int KR = 32, KS = 2, ST = 3;  // rows of a K-tile, its steps, stages
  using OA = DenseMN<bf16, Tl::BM, Tl::FM, Tl::NW, KR>;
  using OB = DenseMN<bf16, Tl::BN, Tl::FN, Tl::NW, KR>;
  static constexpr int STAGE = OA::BYTES + OB::BYTES, NI = OA::NI + OB::NI;
  static constexpr int PATCH = Tl::NW * 32 * kDensePatch * 4;
  static constexpr int LDS = ST * STAGE > PATCH ? ST * STAGE : PATCH;
  static_assert(LDS <= 80 << 10, "two workgroups a CU");
};

// acc = the products of K-tiles 0 .. kt1-1 (kt1 > 0), scheduled as dense_tile: at a K-tile's last step the wave
// holds its fragments of it, waits for its loads of the next and for the workgroup, reads the next one's first
// fragments and loads the one three ahead into the stage that has become free.
template <class Tl>
__device__ __forceinline__ void short_dw_loop(const typename ShortDw<Tl>::OA& oa, const typename ShortDw<Tl>::OB& ob,
                                              int64_t kt1, char* smem, int wave, f32x16_t (&acc)[Tl::FM][Tl::FN]) {
  using C = ShortDw<Tl>;
  constexpr int NM = Tl::FM * Tl::FN, NR = Tl::FM + Tl::FN;
  static_assert(NR <= NM, "a fragment read behind each product");
  const uint32_t lds = lds_offset(smem);
  // past the end: the last K-tile again, which no one reads, so that the loads on their way can be counted
  const auto load = [&](auto fullc, int64_t kt, uint32_t to, int j0, int j1) {
    constexpr bool FULL = decltype(fullc)::value;
    const int64_t k = FULL ? kt : min(kt, kt1 - 1);
    if (j0 < C::OA::NI) oa.template issue<FULL>(k, to, wave, j0, min(j1, C::OA::NI));
    if (j1 > C::OA::NI) ob.template issue<FULL>(k, to + C::OA::BYTES, wave, max(j0 - C::OA::NI, 0), j1 - C::OA::NI);
  };
  const std::false_type no;
  for (int k = 0; k < C::ST; ++k) load(no, k, lds + k * C::STAGE, 0, C::NI);
  wait_vmcnt<2 * C::NI>();
  ring_barrier();
  uint4 a[2][Tl::FM], b[2][Tl::FN];
#pragma unroll
  for (int m = 0; m < Tl::FM; ++m) a[0][m] = oa.frag(smem, m, 0);
#pragma unroll
  for (int n = 0; n < Tl::FN; ++n) b[0][n] = ob.frag(smem + C::OA::BYTES, n, 0);
  uint32_t st = 0;  // stage of K-tile kt
  const auto tile = [&](auto fullc, int64_t kt) {
    const uint32_t nst = st + 1 == C::ST ? 0 : st + 1;
    static_for<0, C::KS>([&](auto kc) {
      constexpr int ks = decltype(kc)::value, c = ks & 1;
      constexpr bool last = ks == C::KS - 1;
      if constexpr (last) {
        wait_vmcnt<C::NI>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
      const char* f = smem + (last ? nst : st) * C::STAGE;
      static_for<0, NM>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        Mma<bf16>::run(acc[i / Tl::FN][i % Tl::FN], b[c][i % Tl::FN], a[c][i / Tl::FN]);
        if constexpr (i < NR) {
          if constexpr (i < Tl::FN) b[c ^ 1][i] = ob.frag(f + C::OA::BYTES, i, (ks + 1) % C::KS);
          else a[c ^ 1][i - Tl::FN] = oa.frag(f, i - Tl::FN, (ks + 1) % C::KS);
        }
        if constexpr (last) load(fullc, kt + C::ST, lds + st * C::STAGE, i * C::NI / NM, (i + 1) * C::NI / NM);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    st = nst;
  };
  int64_t kt = 0;
  for (const int64_t full = oa.full(); kt + C::ST < full; ++kt) tile(std::true_type(), kt);
#pragma unroll 1
  for (; kt < kt1; ++kt) tile(no, kt);
  wait_vmcnt<0>();  // no load into LDS outlives its user
  __syncthreads();
}

template <class Tl, typename TO>
__global__ __launch_bounds__(Tl::NT, 2) void grouped_short_dw_kernel(GroupedArgs ga) {
  using C = ShortDw<Tl>;
  __shared__ __align__(1024) char smem[C::LDS];
  LinearArgs a = ga.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Tl::WN, wn = wave % Tl::WN;
  int g, mt, nt, slice;
  dw_tile(ga, (int)((a.M + Tl::BM - 1) / Tl::BM), (a.N + Tl::BN - 1) / Tl::BN, g, slice, mt, nt);
  const int lo = group_clamp(ga.off[g], 0, (int)a.K), n = group_clamp(ga.off[g + 1], lo, (int)a.K) - lo;
  const int64_t m0 = (int64_t)mt * Tl::BM, o = (int64_t)g * a.M * a.N;
  const int n0 = nt * Tl::BN;
  f32x16_t acc[Tl::FM][Tl::FN];
  zero_acc<Tl>(acc);
  if (n > 0) {
    typename C::OA oa;
    typename C::OB ob;
    oa.init((const bf16*)a.a + (int64_t)lo * a.M + m0, 2 * a.M, n, a.M - m0, [&](int f) { return wm * Tl::WTM + f * 32; },
            wave, lane);
    ob.init((const bf16*)a.b + (int64_t)lo * a.N + n0, 2 * (int64_t)a.N, n, a.N - n0,
            [&](int f) { return wn * Tl::WTN + f * 32; }, wave, lane);
    short_dw_loop<Tl>(oa, ob, (n + C::KR - 1) / C::KR, smem, wave, acc);
  }
  a.out = (TO*)a.out + o;
  if (a.add != nullptr) a.add = (const TO*)a.add + o;
  const auto in = [&](int row, int j) { return m0 + row < a.M && n0 + j < a.N; };
  dense_epilogue<Tl, false>(
      acc, smem, wave, wm, wn, lane,
      [&](int row, int j) { return in(row, j) ? linear_add8<TO>(a, m0 + row, n0 + j) : Raw8<TO>{}; },
      [&](auto, int row, int j, float (&v)[8], float (&u)[8], const Raw8<TO>& add) {
        if (in(row, j)) linear_store8<LIN_DW, MOK_EPI_NONE, TO, bf16, true>(a, m0 + row, n0 + j, v, u, add);
      });
}

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
    int g, slice;
    dw_tile(ga, (int)((a.M + Tl::BM - 1) / Tl::BM), NT, g, slice, mt, nt);
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
    a.b = (const T*)a.b + (int64_t)t.g * (KIND == LIN_FWD ? P * a.K : a.K * a.N);
    if (KIND == LIN_FWD && a.bias != nullptr) a.bias += t.g * P;
    // 256 x 256 tiles: a group's rows are shared out evenly, and its tiles are as high as that needs (64, 128, 192 or
    // 256): they run side by side at one pace and share w (16384 rows of 42 groups, 4096 x 7168: 2.86 GB are read from
    // memory, where w and x are 2.70). Where a group's last tile alone was lower: 1133 us for 1045 there, 1063 for 1008
    // with 320 rows in each of 48 groups.
    constexpr bool CUT = Tl::BM == 256;
    const int64_t KT = (a.K + Cfg::BKE - 1) / Cfg::BKE;
    const int high = CUT ? (t.hi - t.lo + t.tiles - 1) / t.tiles : Tl::BM;
    const int64_t m0 = t.lo + (int64_t)mt * high, left = min((int64_t)t.hi, m0 + high) - m0;
    a.M = m0 + left;  // rows of other groups are neither read nor written
    using H1 = Tiling<CUT ? 64 : Tl::BM, Tl::BN, Tl::WM, Tl::WN>;
    using H2 = Tiling<CUT ? 128 : Tl::BM, Tl::BN, Tl::WM, Tl::WN>;
    using H3 = Tiling<CUT ? 192 : Tl::BM, Tl::BN, Tl::WM, Tl::WN>;
    if (!CUT || high > 192) dense_work<T, Tl, KIND, EPI, TO, false>(a, m0, nt * Cfg::BN, 0, KT, nullptr, smem);
    else if (high > 128) dense_work<T, H3, KIND, EPI, TO, false, true>(a, m0, nt * Cfg::BN, 0, KT, nullptr, smem);
    else if (high > 64) dense_work<T, H2, KIND, EPI, TO, false, true>(a, m0, nt * Cfg::BN, 0, KT, nullptr, smem);
    else dense_work<T, H1, KIND, EPI, TO, false, true>(a, m0, nt * Cfg::BN, 0, KT, nullptr, smem);
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

template <typename TO>
void run_grouped_short_dw(const GroupedArgs& ga, hipStream_t s) {
  using Tl = Tiling<256, 128, 2, 2>;
  const dim3 grid((unsigned)((ga.l.M + Tl::BM - 1) / Tl::BM * ((ga.l.N + Tl::BN - 1) / Tl::BN) * ga.E));
  hipLaunchKernelGGL((grouped_short_dw_kernel<Tl, TO>), grid, dim3(Tl::NT), 0, s, ga);
}

template <typename T, class Tl>
void run_grouped_fwd(const GroupedArgs& a, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_grouped<T, Tl, LIN_FWD, MOK_EPI_NONE, T>(a, s);
  else if (epi == MOK_EPI_SILU) run_grouped<T, Tl, LIN_FWD, MOK_EPI_SILU, T>(a, s);
  else if (epi == MOK_EPI_GELU) run_grouped<T, Tl, LIN_FWD, MOK_EPI_GELU, T>(a, s);
  else if constexpr (Tl::FN % 2 == 0) run_grouped<T, Tl, LIN_FWD, MOK_EPI_SWIGLU, T>(a, s);  // gate and up side by side
}

}  // namespace mok
