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

// The groups cut into tiles of bm rows: a lane holds 1/64 of the groups, the wave a prefix sum of
// their tiles, so a tile is found in one round of loads wherever it lies (a table of tiles would be a
// launch of its own, 3 us). Every wave of the workgroup does so for itself.
struct GroupScan {
  int v[17];   // offsets of this lane's groups
  int excl;    // tiles before them
  int total;   // tiles of all groups
  int C, M, E, g0;

  __device__ __forceinline__ void init(const int32_t* __restrict__ off, int E_, int64_t M_, int bm) {
    const int lane = threadIdx.x & 63;
    E = E_;
    M = (int)M_;
    C = (E + 63) >> 6;
    g0 = lane * C;
#pragma unroll
    for (int c = 0; c < 17; ++c)
      if (c <= C) v[c] = off[min(g0 + c, E)];
    // offsets that descend count as the largest before them, so that the groups' rows are at most M
    int top = 0;
#pragma unroll
    for (int c = 0; c < 17; ++c)
      if (c <= C) top = group_clamp(v[c], top, M);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(top, o);
      if (lane >= o) top = max(top, t);
    }
    const int before = __shfl_up(top, 1);
    v[0] = group_clamp(v[0], lane == 0 ? 0 : before, M);
    int n = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (c < C) {
        v[c + 1] = group_clamp(v[c + 1], v[c], M);
        n += (v[c + 1] - v[c] + bm - 1) / bm;
      }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(incl, o);
      if (lane >= o) incl += t;
    }
    excl = incl - n;
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  // The group of tile q, 0 <= q < total.
  __device__ __forceinline__ GroupTile find(int q, int bm) const {
    int g = 0, lo = 0, hi = 0, first = 0, tiles = 0, at = excl;
    bool here = false;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (c < C) {
        const int t = (v[c + 1] - v[c] + bm - 1) / bm;
        if (q >= at && q < at + t) {
          here = true;
          g = g0 + c;
          lo = v[c];
          hi = v[c + 1];
          first = at;
          tiles = t;
        }
        at += t;
      }
    const int src = __builtin_ctzll(__ballot(here));
    return {__builtin_amdgcn_readlane(g, src), __builtin_amdgcn_readlane(lo, src), __builtin_amdgcn_readlane(hi, src),
            __builtin_amdgcn_readlane(first, src), __builtin_amdgcn_readlane(tiles, src)};
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
struct GroupedPlan {
  int tile;   // as LinearPlan's, or kFewTile, or kFewTile + 1 (32 rows)
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
