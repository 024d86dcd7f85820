// Grouped products with a few rows a group (a decoding batch): a workgroup takes up to 16 or 32 rows of
// one group and 16 rows of its w over all of K, as linear_few.hip does for one matrix.
#include "grouped.h"
#include "linear_few.h"

namespace mok {

namespace {

template <typename T, int EPI, int RT>
__global__ __launch_bounds__(64 * kFewWaves) void grouped_few_kernel(GroupedArgs ga) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  constexpr int BM = 16 * RT;
  __shared__ __align__(16) float s_sum[kFewWaves][BM][kFewLd];
  LinearArgs a = ga.l;
  const int NT = SW ? a.N / 8 : (a.N + 15) / 16;
  GroupScan scan;
  scan.init(ga.off, ga.E, a.M, BM);
  const int tiles = scan.total * NT;
  if ((int)blockIdx.x >= tiles) return;
  const int L = xcd_logical(blockIdx.x, tiles);
  const GroupTile t = scan.find(L / NT, BM);
  // the tiles of a group that share rows of w one after the other
  const int i = L - t.first * NT, mt = i % t.tiles, nt = i / t.tiles;
  const int64_t r0 = t.lo + (int64_t)mt * BM, P = SW ? 2 * (int64_t)a.N : a.N;
  a.M = min<int64_t>(BM, t.hi - r0);
  a.a = (const T*)a.a + r0 * a.K;
  a.b = (const T*)a.b + t.g * P * a.K;
  if (a.bias != nullptr) a.bias += t.g * P;
  if (a.add != nullptr) a.add = (const T*)a.add + r0 * a.N;
  a.out = (T*)a.out + r0 * a.N;
  if (a.pre != nullptr) a.pre = (T*)a.pre + r0 * P;
  few_work<T, EPI, RT>(a, nt, s_sum);
}

template <typename T, int EPI>
void run_few(const GroupedArgs& ga, int rt, hipStream_t s) {
  const int cols = EPI == MOK_EPI_SWIGLU ? 8 : 16;
  const dim3 grid((unsigned)(group_tiles_bound(ga.l.M, ga.E, 16 * rt) * ((ga.l.N + cols - 1) / cols)));
  if (rt == 1) hipLaunchKernelGGL((grouped_few_kernel<T, EPI, 1>), grid, dim3(64 * kFewWaves), 0, s, ga);
  else hipLaunchKernelGGL((grouped_few_kernel<T, EPI, 2>), grid, dim3(64 * kFewWaves), 0, s, ga);
}

template <typename T>
void run_few(const GroupedArgs& a, int rt, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_few<T, MOK_EPI_NONE>(a, rt, s);
  else if (epi == MOK_EPI_SILU) run_few<T, MOK_EPI_SILU>(a, rt, s);
  else if (epi == MOK_EPI_GELU) run_few<T, MOK_EPI_GELU>(a, rt, s);
  else run_few<T, MOK_EPI_SWIGLU>(a, rt, s);
}

}  // namespace

hipError_t launch_grouped_few(const GroupedArgs& a, int rt, int act, int epi, hipStream_t s) {
  if (act == MOK_F32) run_few<float>(a, rt, epi, s);
  else run_few<bf16>(a, rt, epi, s);
  return hipGetLastError();
}

}  // namespace mok
