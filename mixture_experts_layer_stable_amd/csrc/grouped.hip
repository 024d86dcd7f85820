// Matrix products grouped by expert with ragged sizes, forward and backward: the choice of a tile, dp and
// the bias gradient.
#include <cmath>

#include "grouped.h"
#include "linear.h"

namespace mok {

namespace {

// ---- dp = dy f'(pre) of the rows in groups, and the bias gradient ----
// As linear_dpre_kernel (a thread keeps eight columns and walks down the rows of a chunk, HBM-bound),
// and at a group's last row the sums go out and start again. A wave finds the group of a row in one round of
// loads (a search by halves is a chain of them). dp is rounded to the operands' type, as there: independent errors of
// half a step, 1.66e-3 of the norm for bf16, in the terms of dx and dw, and as much again from the results' own
// rounding: 2.3e-3 in all, 2.5e-3 from what is rounded at the end only. The sums of db are of dp before it is rounded.
template <typename T, int EPI>
__global__ __launch_bounds__(256) void grouped_dpre_kernel(const T* __restrict__ dy, const T* __restrict__ pre,
                                                           const int32_t* __restrict__ off, int M, int N, int E, int rows,
                                                           T* __restrict__ dp, float* __restrict__ part) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  const int64_t P = SW ? 2 * (int64_t)N : N;
  const int c0 = (blockIdx.x * 256 + threadIdx.x) * 8, c = min(c0, N - 8);  // whole waves search
  const bool live = c0 < N;
  int m = group_clamp(off[0], 0, M);
  m = max(m, (int)blockIdx.y * rows);
  const int end = (int)min<int64_t>(((int64_t)blockIdx.y + 1) * rows, group_clamp(off[E], 0, M));
  while (m < end) {
    int g = 0, m1 = end;
    if (part != nullptr) {  // the sums end with the group: the last one that begins at or before row m
      int n = 0;
#pragma unroll 4
      for (int i = threadIdx.x & 63; i < ((E + 63) & ~63); i += 64) n += __popcll(__ballot(i < E && off[min(i, E)] <= m));
      g = max(n - 1, 0);
      m1 = min(end, off[g + 1]);
      if (m1 <= m) return;  // offsets that descend
    }
    float sg[8], su[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.0f;
#pragma unroll 4
    for (; m < m1; ++m) {
      float d[8], p[8], u[8];
      load8(dy + (int64_t)m * N + c, d);
      if constexpr (EPI != MOK_EPI_NONE) load8(pre + m * P + c, p);
      if constexpr (SW) load8(pre + m * P + N + c, u);
      linear_dpre8<T, EPI>(d, p, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sg[i] += d[i];
        if constexpr (SW) su[i] += u[i];
      }
      if constexpr (EPI != MOK_EPI_NONE) {
        if (!live) continue;
        store8(dp + m * P + c, d);
        if constexpr (SW) store8(dp + m * P + N + c, u);
      }
    }
    if (part == nullptr || !live) continue;
    float* o = part + ((int64_t)blockIdx.y + g) * P + c;
    store8(o, sg);
    if constexpr (SW) store8(o + N, su);
  }
}

// db[g][p]: the parts of group g in 16 interleaved sums, added in order; 64 columns a workgroup.
__global__ __launch_bounds__(1024) void grouped_db_kernel(const float* __restrict__ part, const int32_t* __restrict__ off,
                                                          int M, int P, int rows, float* __restrict__ db) {
  __shared__ float s_sum[16][64];
  const int col = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * 64 + col, g = blockIdx.y;
  const int lo = group_clamp(off[g], 0, M), hi = group_clamp(off[g + 1], lo, M);
  float v = 0.0f;
  if (lo < hi && c < P)
    for (int i = lo / rows + w; i <= (hi - 1) / rows; i += 16) v += part[((int64_t)i + g) * P + c];
  s_sum[w][col] = v;
  __syncthreads();
  if (w != 0 || c >= P) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s_sum[i][col];
  db[(int64_t)g * P + c] = v;
}

template <typename T>
void run_dpre(const void* dy, const void* pre, const int32_t* off, int64_t M, int N, int E, int epi, void* dp, float* part,
              hipStream_t s) {
  const int rows = linear_db_rows(M, N);
  const dim3 grid((N + 2047) / 2048, (unsigned)((M + rows - 1) / rows)), block(256);
  const T *d = (const T*)dy, *p = (const T*)pre;
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, d, p, off, (int)M, N, E, rows, (T*)dp, part); };
  if (epi == MOK_EPI_NONE) go(grouped_dpre_kernel<T, MOK_EPI_NONE>);
  else if (epi == MOK_EPI_SILU) go(grouped_dpre_kernel<T, MOK_EPI_SILU>);
  else if (epi == MOK_EPI_GELU) go(grouped_dpre_kernel<T, MOK_EPI_GELU>);
  else go(grouped_dpre_kernel<T, MOK_EPI_SWIGLU>);
}

}  // namespace

// The tile of least estimated time, as linear_plan's, for rows spread evenly over the groups: the
// offsets stay on the device, and a launch's sizes and order of sums depend on the shape alone. Over 15 shapes
// from 16 to 32768 rows of 2 to 151 groups, forward and dx, at every tile: the one taken is the fastest or
// within a fifth of it.
GroupedPlan grouped_plan(int kind, int act, int epi, int64_t M, int N, int64_t K, int E) {
  GroupedPlan best{0, 1};
  const int64_t all = kind == LIN_DW ? K : M;  // rows of all groups
  if (all == 0) return best;
  struct Tile {
    int bm, bn, per_cu;
    double ktile, fixed;
  };
  static const Tile kTiles[4] = {
      {256, 256, 1, 1.55, 11.0}, {128, 128, 2, 0.97, 5.0}, {64, 128, 3, 1.1, 4.0}, {32, 128, 4, 1.2, 3.5}};
  static const Tile kTilesF32[2] = {{128, 128, 2, 1.75, 11.0}, {64, 64, 4, 0.45, 6.0}};  // K-tiles of 32
  static const Tile kTilesF32Sw[2] = {{128, 128, 2, 1.75, 11.0}, {64, 128, 3, 1.05, 6.0}};
  const bool f32 = act == MOK_F32;
  const int64_t P = epi == MOK_EPI_SWIGLU ? 2 * (int64_t)N : N, bk = f32 ? 32 : 64;
  const double groups = (double)std::min<int64_t>(E, all);
  double least = 1e30;
  for (int t = 0; t < (f32 ? 2 : 4); ++t) {
    const Tile& c = f32 ? (epi == MOK_EPI_SWIGLU ? kTilesF32Sw[t] : kTilesF32[t]) : kTiles[t];
    const double slots = 256.0 * c.per_cu;
    const int64_t nt = (P + c.bn - 1) / c.bn;
    double tiles, bound, kt;
    if (kind == LIN_DW) {
      tiles = bound = (double)((M + c.bm - 1) / c.bm) * (double)nt * E;
      kt = (double)all / E / (double)bk + 0.5;
    } else {
      // a group's last tile is half full on average (256 rows: an eighth of a tile is lost, see grouped_dense.h)
      const bool cut = c.bm == 256;
      tiles = std::max(groups * (cut ? 0.4 : 1.0), (double)M / c.bm + (cut ? 0.125 : 0.5) * groups) * (double)nt;
      bound = (double)group_tiles_bound(M, E, c.bm) * (double)nt;
      kt = (double)((K + bk - 1) / bk);
    }
    if (t > 0 && bound >= (1 << 23)) continue;  // 2^32 threads a launch; the largest tile always fits
    for (int split = 1; split <= (kind == LIN_DW ? 64 : 1); split *= 2) {
      if (split > 1 && (kt / split < 2 || tiles * split >= (1 << 16))) break;
      // a few rounds are whole ones: the tiles of a shape take about the same time
      double rounds = std::max(1.0, tiles * split / slots);
      if (rounds > 1) rounds = rounds < 4 ? std::ceil(rounds + 0.03) : rounds + 0.3;
      const double kts = kt / split;
      const double bytes = 8.0 * split * (double)E * (double)M * (double)P;
      double us;
      if (f32) {
        us = std::max(1.0, tiles * split / 256.0) * kts * c.ktile + c.fixed + 2.5 * rounds;
      } else {
        const double fill = std::min(1.0, tiles * split / slots);
        us = rounds * (kts * c.ktile * (0.5 + 0.5 * fill) + c.fixed);
      }
      if (split > 1) us += 5.0 + bytes / 4e6;
      if (us < least) {
        least = us;
        best = {t, split};
      }
    }
  }
  if (kind == LIN_DW && !f32) {
    // K-tiles of 32 rows, two workgroups a CU, and what a tile takes besides them
    const double tiles = (double)((M + 255) / 256) * (double)((N + 127) / 128) * E, kt = (double)all / E / 32 + 0.5;
    const double us = std::max(1.0, tiles / 512) * (kt * 0.86 * (0.6 + 0.4 * std::min(1.0, tiles / 512)) + 5.7);
    if (tiles < (1 << 24) && us < least) best = {kShortTile, 1};
  }
  if (kind == LIN_FWD) {
    for (int rt = 1; rt <= 2; ++rt) {
      const double nt = (double)((P + 15) / 16), tiles = std::max(groups, (double)M / (16 * rt) + 0.5 * groups) * nt;
      if ((double)group_tiles_bound(M, E, 16 * rt) * nt >= (1 << 22)) continue;  // 2^32 threads
      const double lat = rt == 1 ? (f32 ? 1.1 : 0.7) : (f32 ? 1.6 : 1.15);
      const double full = rt == 1 ? (f32 ? 2.0 : 1.7) : (f32 ? 3.1 : 2.5);
      const int64_t piece = 8 * (256 / (f32 ? 4 : 2));
      const double us = 4.0 + (double)((K + piece - 1) / piece) * std::max(lat, full * tiles / 256.0);
      const double hbm = (f32 ? 4.0 : 2.0) * groups * (double)P * (double)K / 5.4e6;
      if (us < std::max(least, hbm)) {
        least = us;
        best = {kFewTile + rt - 1, 1};
      }
    }
  }
  return best;
}

size_t grouped_part_bytes(int kind, int act, int epi, int64_t M, int N, int64_t K, int E) {
  const int split = grouped_plan(kind, act, epi, M, N, K, E).split;
  return split > 1 ? 4 * (size_t)split * (size_t)E * (size_t)M * N : 0;
}

hipError_t launch_grouped(const GroupedArgs& args, int kind, int act, int epi, bool out_f32, hipStream_t s) {
  GroupedArgs a = args;
  const GroupedPlan p = grouped_plan(kind, act, epi, a.l.M, a.l.N, a.l.K, a.E);
  a.l.split = p.split;
  if (p.tile == kFewTile || p.tile == kFewTile + 1) return launch_grouped_few(a, p.tile - kFewTile + 1, act, epi, s);
  if (act == MOK_BF16) return launch_grouped_bf16(a, p.tile, kind, epi, out_f32, s);
  return launch_grouped_f32(a, p.tile, kind, epi, s);
}

int64_t grouped_db_parts(int64_t M, int N, int E) { return M == 0 ? 0 : linear_db_parts(M, N) + (int64_t)E; }

hipError_t launch_grouped_dpre(const void* dy, const void* pre, const int32_t* off, int64_t M, int N, int E, int act,
                               int epi, void* dp, float* part, hipStream_t s) {
  if (act == MOK_F32) run_dpre<float>(dy, pre, off, M, N, E, epi, dp, part, s);
  else run_dpre<bf16>(dy, pre, off, M, N, E, epi, dp, part, s);
  return hipGetLastError();
}

hipError_t launch_grouped_db(const float* part, const int32_t* off, int64_t M, int N, int P, int E, float* db,
                             hipStream_t s) {
  hipLaunchKernelGGL(grouped_db_kernel, dim3((P + 63) / 64, E), dim3(1024), 0, s, part, off, (int)M, P,
                     M == 0 ? 1 : linear_db_rows(M, N), db);
  return hipGetLastError();
}

}  // namespace mok
