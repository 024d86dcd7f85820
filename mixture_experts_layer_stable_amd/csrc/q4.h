// Products with 4-bit weights and group scales (q4*.hip): launch interface and what the kernels share.
#pragma once
#include "grouped.h"

namespace mok {

struct Q4Args {
  LinearArgs l;         // a = x, M, N, K, bias, add, out; b = codes [E][P][K / 2]
  const void* s;        // [E][P][K / group] in the operands' type
  const uint8_t* z;     // [E][P][K / group] or nullptr: 8
  const int32_t* off;   // [E + 1] or nullptr: one group of all rows
  int E, group;
};
hipError_t launch_q4(const Q4Args& a, int act, int epi, hipStream_t s);
hipError_t launch_q4_few(const Q4Args& a, int rt, int act, int epi, hipStream_t s);
hipError_t launch_q4_quantize(const void* w, int64_t rows, int K, int group, int act, void* q, void* s, uint8_t* z,
                              hipStream_t st);

// The group and rows of tile q of bm rows; dense: one group of M rows.
__device__ __forceinline__ bool q4_tile(const Q4Args& qa, int bm, int NT, int& L, GroupTile& t) {
  if (qa.off == nullptr) {
    const int M = (int)qa.l.M, mt = (M + bm - 1) / bm;
    if ((int)blockIdx.x >= mt * NT) return false;
    L = xcd_logical(blockIdx.x, mt * NT);
    t = {0, 0, M, 0, mt};
    return true;
  }
  GroupScan scan;
  scan.init(qa.off, qa.E, qa.l.M, bm);
  const int tiles = scan.total * NT;
  if ((int)blockIdx.x >= tiles) return false;
  L = xcd_logical(blockIdx.x, tiles);
  t = scan.find(L / NT, bm);
  return true;
}
inline int64_t q4_tiles_bound(const Q4Args& a, int bm) {
  return a.off == nullptr ? (a.l.M + bm - 1) / bm : group_tiles_bound(a.l.M, a.E, bm);
}

}  // namespace mok
