// Products with 4-bit weights for a few rows of x a group (decoded tokens).
//
//   p[m][n] = sum over groups j of K of s[n][j] (sum_k x[m][k] (16 + q[n][k]) - (16 + z[n][j]) sum_k x[m][k])
//
// What bounds them is, from some hundred MB of codes on, the instructions that a code takes (128 rows of 48
// groups, 7168 x 2048: 84 to 91 us, 3.5 TB/s; 2 x 2048 x 7168 each: 143 to 168 us, 3.6 to 4.1 TB/s), and in small calls the
// latency of each step, of which the loop is less than half (one row, 2 x 2048 x 7168: 8.8 to 10.0 us; fp32 19.5). Dense
// products of more rows load and convert each code again for every 16 of them: from 8 rows of 2 x 2048 x 7168, and from the
// first of 7168 x 2048, the bf16 product of linear.hip is the faster one (16 rows: 19 and 15 us, 12 and 9). A
// wave takes 16 rows of w (8 gate and 8 up rows for SWIGLU) and 128 codes of each at a time; four such
// pieces are on their way while the four before them are worked on. Of a workgroup's eight waves WS share
// a row tile, each a part of K, and 8 / WS tiles lie side by side. The workgroups, one a CU, share the tiles
// of all groups evenly; a workgroup's rows of x stay in LDS for all of its tiles (or pass through it in two
// stages), in the order in which the matrix units want them, so a wave streams codes from tile to tile.
// (One workgroup for each set of tiles: 547 us for the 85. Codes through LDS by direct loads, or four pieces
// in a ring of registers: not faster. Sixteen waves: slower, they spill.)
// A code becomes a matrix operand without arithmetic: 16 + q in bf16 is 0x4180 | q << 3, two of a dword at
// a time. A second multiplication, by -(16 + z), takes off what the offset brought in; both are exact in
// fp32 up to its sums, and a group's result takes its scale in fp32. So w is never rounded to bf16.
// fp32 x: codes as fp32 numbers q - z.
#include "linear_few.h"
#include "q4.h"

namespace mok {

namespace {

constexpr int kPiece = 128;  // codes of a row that a wave takes at a time
constexpr int kBatch = 4;    // pieces that it loads at a time
constexpr int kWaves = 8;
constexpr int kRows = 16;    // rows of x of a workgroup

// A barrier for what the waves left in LDS. __syncthreads would wait for the codes that are on their way, too.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Lanes l, l + 16, l + 32, l + 48 hold four dwords each: dword d of lane group g <-> dword g of lane group d.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void group_transpose(uint32_t (&u)[4]) {
  swap32(u[0], u[2]);
  swap32(u[1], u[3]);
  swap16(u[0], u[1]);
  swap16(u[2], u[3]);
}

// Eight codes of a dword as bf16 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 codes_bf16(uint32_t v) {
  constexpr uint32_t m = 0x00780078u, o = 0x41804180u;
  return make_uint4((v << 3 & m) | o, (v >> 1 & m) | o, (v >> 5 & m) | o, (v >> 9 & m) | o);
}
// Eight bf16 values in that order.
__device__ __forceinline__ uint4 order_bf16(const uint4& x) {
  return make_uint4(__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                    __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u));
}

// G: codes that share a scale; WS: waves that share a tile of w
template <typename T, bool SW, int G, int WS>
__global__ __launch_bounds__(64 * kWaves) void q4_few_kernel(Q4Args qa) {
  constexpr bool BF = std::is_same<T, bf16>::value;
  constexpr int WN = kWaves / WS, NTH = 64 * kWaves;
  constexpr int XV = BF ? 1 : 2;                   // 16-byte vectors of eight values of x
  constexpr int GP = kPiece / G;                   // scales of a piece
  constexpr uint32_t XB = 128 << 10;               // of x in LDS, or twice a stage of it
  constexpr int NX = XB / 2 / 16 / NTH;            // vectors of a stage that a thread loads
  __shared__ __align__(16) struct {
    char x[XB];
    float sum[kWaves][kRows][kFewLd];
  } lds;
  LinearArgs a = qa.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, ks = wave % WS;
  const uint32_t K = (uint32_t)a.K, KG = K / G, pieces = (K + kPiece - 1) / kPiece, rounds = (pieces + WS - 1) / WS;
  const int64_t P = SW ? 2 * (int64_t)a.N : a.N;
  const int cols = SW ? 8 : 16, NS = ((a.N + cols - 1) / cols + WN - 1) / WN;  // sets of WN tiles of w

  // this workgroup's sets: an even share of those of all row tiles
  int cur = 0, end = 1;
  for (bool begin = true; cur < end; begin = false) {
    GroupTile t;
    int q;
    {
      GroupScan scan;
      int total = ((int)a.M + kRows - 1) / kRows;
      if (qa.off != nullptr) {
        scan.init(qa.off, qa.E, a.M, kRows);
        total = scan.total;
      }
      if (begin) {
        const int all = total * NS, wgs = min(all, (int)gridDim.x);
        if ((int)blockIdx.x >= wgs) return;
        const int l = xcd_logical(blockIdx.x, wgs), share = all == wgs ? 1 : all / wgs, more = all - share * wgs;
        cur = l * share + min(l, more);
        end = cur + share + (l < more);
      }
      q = total == 1 ? 0 : cur / NS;  // (a division takes 0.1 us of a small call)
      t = {0, 0, (int)a.M, 0, total};
      if (qa.off != nullptr) t = scan.find(q, kRows);
    }
    // row tile and sets of it: set0 ..
    const int set0 = cur - q * NS, nset = min(end - cur, NS - set0);
    cur += nset;
    const int64_t r0 = t.lo + (int64_t)(q - t.first) * kRows;
    const uint32_t M = (uint32_t)min<int64_t>(kRows, t.hi - r0);
    const T* x = (const T*)a.a + r0 * K;

    // x in LDS: 2^mb rows of SP pieces; eight values (unit u of a piece) are a lane's for one step: step
    // u % 4 of lane group u / 4 if the piece has one scale, else, as group_transpose leaves the codes, step
    // u / 4 of lane group u % 4. Rows past M hold what was there: it ends in results that are not stored.
    int mb = 0;
    while ((1u << mb) < M) ++mb;
    const uint32_t pb = (16 * 16 * XV) << mb;  // bytes of a piece
    const bool staged = pieces * pb > XB;
    uint32_t XR = rounds, SP = pieces, stages = 1;  // rounds and pieces of a stage, stages
    if (staged) {
      XR = XB / 2 / pb / WS;
      SP = XR * WS;
      stages = (pieces + SP - 1) / SP;
    }
    const auto slot = [&](uint32_t p, uint32_t step, uint32_t h, uint32_t lg, uint32_t m) {  // of 16 bytes
      return ((((p * 4 + step) * XV + h) * 4 + lg) << mb) + ((m ^ (4 * lg + step)) & ((1u << mb) - 1));
    };
    // 64 vectors of a row of the pieces from p0 on: block i of M * nb, nb blocks a row
    const auto get_x = [&](uint32_t p0, uint32_t i, uint32_t nb) {
      const uint32_t m = M == 1 ? 0 : i / nb, c = (i - m * nb) * 64 + lane, k = p0 * kPiece + c * (8 / XV);
      const uint4 d = ldg16(x + (uint64_t)min(m, M - 1) * K + min(k, K - 8 / XV));
      return k < K ? d : make_uint4(0, 0, 0, 0);
    };
    const auto put_x = [&](char* to, uint32_t i, uint32_t nb, uint32_t n, uint4 d) {
      const uint32_t m = M == 1 ? 0 : i / nb, c = (i - m * nb) * 64 + lane, u = c / XV % 16, h = c % XV;
      if constexpr (BF) d = order_bf16(d);
      if (m < M && c < n)
        *reinterpret_cast<uint4*>(to + 16 * slot(c / (16 * XV), GP > 1 ? u / 4 : u % 4, h, GP > 1 ? u % 4 : u / 4, m)) = d;
    };
    const uint32_t sv = SP * (16 * XV), sb = (sv + 63) / 64;  // vectors and blocks of a row of a stage
    uint4 xr[NX];
    const auto load_x = [&](uint32_t st) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NX; ++i) xr[i] = get_x(st * SP, i * kWaves + wave, sb);
    };
    const auto store_x = [&](uint32_t buf) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NX; ++i) put_x(lds.x + (buf & 1) * (XB / 2), i * kWaves + wave, sb, sv, xr[i]);
    };
    uint32_t xoff[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) xoff[e] = 16 * slot(0, e, 0, g, r);
    const uint32_t xhalf = 16 * 4 << mb;  // to the second vector

    // Codes and scales of a batch: of piece n, and of piece (lane group). Every load is made, whatever the piece:
    // behind a condition the compiler would not know how many are on their way, and wait for all of them;
    // for the same reason scales stay as loaded. Past the end the last codes come again, with a scale of 0.
    struct Batch {
      uint4 w[kBatch];
      T s[GP];
      uint8_t z[GP];
      bool in[GP];
    };
    int set_l = set0;
    uint32_t round_l = 0;  // the loads' place in the stream
    const uint8_t *wq, *wz;
    const T* ws;
    const auto rows_l = [&]() {
      const int n0 = (set_l * WN + wave / WS) * cols;  // rows past N re-read the last one
      const int64_t wr = t.g * P + (SW ? (int64_t)min(n0 + (r & 7), a.N - 1) + (r < 8 ? 0 : a.N) : min(n0 + r, a.N - 1));
      wq = (const uint8_t*)a.b + wr * (K / 2);
      ws = (const T*)qa.s + wr * KG;
      wz = qa.z + wr * KG;
    };
    const int last = set0 + nset - 1;
    const auto load = [&](Batch& d) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        const uint32_t p = min((round_l + n) * WS + ks, pieces - 1);
        d.w[n] = ldg16(wq + min(p * (kPiece / 2) + 16 * g, K / 2 - 16));
      }
      const uint32_t p = (round_l + g) * WS + ks;
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        const uint32_t i = p * GP + j;
        d.in[j] = p < pieces && i < KG;
        d.s[j] = ws[d.in[j] ? i : 0];
        d.z[j] = wz[d.in[j] ? i : 0];
      }
      round_l += kBatch;
      if (round_l >= rounds) {
        round_l = 0;
        set_l = min(set_l + 1, last);
        rows_l();
      }
    };
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    int set = set0;
    uint32_t round = 0, sc = 0, buf_round = 0;  // of the work; stages gone by; round within the stage
    // stagedc: whether x comes in stages, known to the compiler so that the rounds of a batch stay in one block
    // and overlap
    const auto work = [&](auto stagedc, const Batch& d) __attribute__((always_inline)) {
      constexpr bool staged = decltype(stagedc)::value;
      float ds[GP];
      uint32_t dz[GP];
#pragma unroll
      for (int j = 0; j < GP; ++j) {
        ds[j] = d.in[j] ? Elem<T>::get(&d.s[j], 0) : 0.0f;
        // bf16: -(16 + z) twice; fp32: z
        if constexpr (BF) dz[j] = 0xC180C180u | (qa.zeros ? d.z[j] & 15u : 8u) * 0x00080008u;
        else dz[j] = __float_as_uint(qa.zeros ? (float)d.z[j] : 8.0f);
      }
      static_for<0, kBatch>([&](auto nc) __attribute__((always_inline)) {
        constexpr int n = decltype(nc)::value;
        if constexpr (staged) {
          if (buf_round == XR && round + n < rounds) {  // the next stage of x
            ++sc;
            store_x(sc);
            lds_barrier();
            load_x((sc + 1) % stages);
            buf_round = 0;
          }
          ++buf_round;
        }
        const uint32_t p = min((round + n) * WS + ks, pieces - 1);
        const char* xs = lds.x + (staged ? (sc & 1) * (XB / 2) + min(p - sc % stages * SP, SP - 1) * pb : p * pb);
        uint32_t w[4] = {d.w[n].x, d.w[n].y, d.w[n].z, d.w[n].w};
        if constexpr (GP > 1) group_transpose(w);
#pragma unroll
        for (int j = 0; j < GP; ++j) {
          const float s = __shfl(ds[j], r + 16 * n);
          const uint32_t z = __shfl(dz[j], r + 16 * n);
          f32x4_t dd = {0.0f, 0.0f, 0.0f, 0.0f}, oo = dd;
#pragma unroll
          for (int e = j * (4 / GP); e < (j + 1) * (4 / GP); ++e) {
            const uint4 xv = *reinterpret_cast<const uint4*>(xs + xoff[e]);
            if constexpr (BF) {
              oo = mma16<bf16>(xv, make_uint4(z, z, z, z), oo);
              dd = mma16<bf16>(xv, codes_bf16(w[e]), dd);
            } else {
              const uint4 xw = *reinterpret_cast<const uint4*>(xs + xhalf + xoff[e]);
              const uint32_t lo = w[e] & 0x0F0F0F0Fu, hi = w[e] >> 4 & 0x0F0F0F0Fu;
              const uint32_t xa[8] = {xv.x, xv.y, xv.z, xv.w, xw.x, xw.y, xw.z, xw.w};
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float f = (float)((c & 1 ? hi : lo) >> (8 * (c / 2)) & 0xFFu) - __uint_as_float(z);
                dd = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xa[c]), f, dd, 0, 0, 0);
              }
            }
          }
          // Past the end of K x is the last piece's again: 0 times an infinity there would be NaN. (bf16: it is NaN in
          // its own place already.)
          const bool on = BF || (round + n) * WS + ks < pieces;
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = __builtin_fmaf(s, BF ? dd[c] + oo[c] : (on ? dd[c] : 0.0f), acc[c]);
        }
      });
      round += kBatch;
      if (round < rounds) return;
      // y of the tiles of the set: a thread (of the wave, or of the workgroup) finishes eight outputs of a row
      constexpr int TPR = SW ? 1 : 2;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lds.sum[wave][4 * g + c][r] = acc[c];
        acc[c] = 0.0f;
      }
      if constexpr (WS > 1) lds_barrier();
      else __builtin_amdgcn_wave_barrier();
      const int v = WS > 1 ? tid : lane;
      const int tile = WS > 1 ? v / (kRows * TPR) : wave, row = v / TPR % kRows, h = SW ? 0 : 8 * (v % TPR);
      const int c0 = (set * WN + tile) * cols + h;
      if (v < (WS > 1 ? WN : 1) * kRows * TPR && row < (int)M && c0 < a.N) {
        const Raw8<T> add = linear_add8<T>(a, r0 + row, c0);
        float s[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = u[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < WS; ++k) {
          float f[8];
          load8(&lds.sum[tile * WS + k][row][h], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] += f[i];
          if constexpr (SW) {
            load8(&lds.sum[tile * WS + k][row][8], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += f[i];
          }
        }
        q4_finish<T, SW>(a, a.bias != nullptr ? a.bias + t.g * P : nullptr, qa.epi, r0 + row, c0, s, u, add);
      }
      if constexpr (WS > 1) lds_barrier();
      else __builtin_amdgcn_wave_barrier();
      round = 0;
      ++set;
      if constexpr (staged) buf_round = XR;  // the next set begins with the first stage
    };

    Batch b0, b1;
    rows_l();
    load(b0);
    lds_barrier();  // the rows before these are done with
    if (staged) {
      load_x(0);
      store_x(0);
      load_x(1);
    } else {
#pragma unroll 2
      for (uint32_t i = wave; i < M * sb; i += kWaves) put_x(lds.x, i, sb, sv, get_x(0, i, sb));
    }
    lds_barrier();
    const auto stream = [&](auto stagedc) __attribute__((always_inline)) {
      while (true) {
        load(b1);
        work(stagedc, b0);
        if (set > last) break;
        load(b0);
        work(stagedc, b1);
        if (set > last) break;
      }
    };
    if (staged) stream(std::true_type());
    else stream(std::false_type());
  }
}

// A tile of w for each wave where they are enough for the chip's 256 CUs, else more waves on one.
template <typename T, bool SW, int G>
void run_few(const Q4Args& a, hipStream_t s) {
  const int64_t nt = SW ? a.l.N / 8 : (a.l.N + 15) / 16, mt = q4_tiles_bound(a, kRows);
  const auto go = [&](auto ws) {
    constexpr int WS = decltype(ws)::value, WN = kWaves / WS;
    const int64_t sets = mt * ((nt + WN - 1) / WN);
    hipLaunchKernelGGL((q4_few_kernel<T, SW, G, WS>), dim3((unsigned)std::min<int64_t>(sets, 256)), dim3(64 * kWaves), 0,
                       s, a);
  };
  if (nt * mt >= 4096) go(std::integral_constant<int, 1>());
  else if (nt * mt >= 1024) go(std::integral_constant<int, 2>());
  else go(std::integral_constant<int, 8>());
}

template <typename T, bool SW>
void run_few(const Q4Args& a, hipStream_t s) {
  if (a.group == 32) run_few<T, SW, 32>(a, s);
  else if (a.group == 64) run_few<T, SW, 64>(a, s);
  else run_few<T, SW, 128>(a, s);
}

}  // namespace

hipError_t launch_q4_few(const Q4Args& a, int act, hipStream_t s) {
  const bool sw = a.epi == MOK_EPI_SWIGLU;
  if (act == MOK_F32) {
    if (sw) run_few<float, true>(a, s);
    else run_few<float, false>(a, s);
  } else {
    if (sw) run_few<bf16, true>(a, s);
    else run_few<bf16, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace mok
