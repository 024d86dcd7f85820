// Rows grouped by expert: what the grouped products (grouped*.hip) and the products with 4-bit
// weights (q4*.hip) share.
#pragma once
#include "block.h"

namespace mok {

// off[0..E] are offsets of the groups' rows. Whatever they hold, no row outside [0, M) is touched.
__device__ __forceinline__ int group_clamp(int v, int lo, int M) { return min(max(v, lo), M); }

// One group's rows lo .. hi-1, and a tile of it.
struct GroupTile {
  int g, lo, hi;
  int first;  // tiles of the groups before it
  int tiles;  // of the group
};

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 to rows 2 and 3
  return v;
}

// The groups cut into tiles of bm rows: a lane holds 1/64 of the groups, the wave a prefix sum of
// their tiles, so a tile is found in one round of loads wherever it lies (a table of tiles would be a
// launch of its own, 3 us). Every wave of the workgroup does so for itself.
struct GroupScan {
  const int32_t* off;
  int C, M, E, g0;
  int excl;   // tiles before this lane's groups
  int total;  // tiles of all groups

  // at most: group_tiles_bound, which offsets that descend could pass
  __device__ __forceinline__ void init(const int32_t* __restrict__ off_, int E_, int64_t M_, int bm) {
    off = off_;
    E = E_;
    M = (int)M_;
    C = (E + 63) >> 6;
    g0 = (threadIdx.x & 63) * C;
    int lo = group_clamp(off[min(g0, E)], 0, M), n = 0;
#pragma unroll 4
    for (int c = 1; c <= C; ++c) {
      const int hi = group_clamp(off[min(g0 + c, E)], lo, M);
      n += (int)((uint32_t)(hi - lo + bm - 1) / (uint32_t)bm);
      lo = hi;
    }
    n = min(n, 1 << 24);
    const int incl = wave_scan(n);
    excl = incl - n;
    total = min(__builtin_amdgcn_readlane(incl, 63), M / bm + min(E, M));
  }

  // The group of tile q, 0 <= q < total.
  __device__ __forceinline__ GroupTile find(int q, int bm) const {
    GroupTile f{0, 0, 0, 0, 0};
    int lo = group_clamp(off[min(g0, E)], 0, M), at = excl;
    bool here = false;
#pragma unroll 4
    for (int c = 1; c <= C; ++c) {
      const int hi = group_clamp(off[min(g0 + c, E)], lo, M);
      const int t = (int)((uint32_t)(hi - lo + bm - 1) / (uint32_t)bm);
      if (q >= at && q < at + t) {
        here = true;
        f = {g0 + c - 1, lo, hi, at, t};
      }
      at += t;
      lo = hi;
    }
    const int src = __builtin_ctzll(__ballot(here));
    return {__builtin_amdgcn_readlane(f.g, src), __builtin_amdgcn_readlane(f.lo, src), __builtin_amdgcn_readlane(f.hi, src),
            __builtin_amdgcn_readlane(f.first, src), __builtin_amdgcn_readlane(f.tiles, src)};
  }
};

// Upper bound of the tiles of bm rows that M rows in E groups make: every full one, and one more for
// each group that can have rows.
inline int64_t group_tiles_bound(int64_t M, int E, int bm) { return M / bm + std::min<int64_t>(E, M); }

// ---- grouped products (launches) ----
struct GroupedArgs {
  LinearArgs l;        // M counts the rows of all groups; b, bias, dw: group after group
  const int32_t* off;  // [E + 1]
  int E;
};
constexpr int kShortTile = 6;
struct GroupedPlan {
  int tile;   // as LinearPlan's, or kFewTile, kFewTile + 1 (32 rows), or LIN_DW's kShortTile
  int split;  // LIN_DW: slices of every group's rows
};
GroupedPlan grouped_plan(int kind, int act, int epi, int64_t M, int N, int64_t K, int E);
size_t grouped_part_bytes(int kind, int act, int epi, int64_t M, int N, int64_t K, int E);
hipError_t launch_grouped(const GroupedArgs& a, int kind, int act, int epi, bool out_f32, hipStream_t s);
hipError_t launch_grouped_bf16(const GroupedArgs& a, int tile, int kind, int epi, bool out_f32, hipStream_t s);
hipError_t launch_grouped_f32(const GroupedArgs& a, int tile, int kind, int epi, hipStream_t s);
hipError_t launch_grouped_few(const GroupedArgs& a, int rt, int act, int epi, hipStream_t s);

// dp = dy f'(pre) of the rows in groups (epi != NONE) and, with part, the sums of dp over the rows of
// chunk c that are in group g, part[c + g][P] (chunks and groups meet in a staircase, so c + g names
// the pair); then db[g][P] of them.
int64_t grouped_db_parts(int64_t M, int N, int E);
hipError_t launch_grouped_dpre(const void* dy, const void* pre, const int32_t* off, int64_t M, int N, int E, int act,
                               int epi, void* dp, float* part, hipStream_t s);
hipError_t launch_grouped_db(const float* part, const int32_t* off, int64_t M, int N, int P, int E, float* db,
                             hipStream_t s);

}  // namespace mok
