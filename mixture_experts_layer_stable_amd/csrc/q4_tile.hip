// Products with 4-bit weights for many rows of x a group (prompts).
//
// A workgroup multiplies BM rows of x by 128 rows of w. x and the codes with their scales and zero points
// come into LDS by direct loads; while the matrix units work on one K-tile (128 bytes of a row of x) the
// codes of the next are written into LDS as matrix operands. bf16: the operand is q - z, exact in bf16,
// and at each group's end its sums take their scale in fp32, so w is never rounded; that costs as
// many accumulators again, and a multiplication for each, and bounds the tile to 256 x 128 (wave tiles of
// 128 x 64). fp32: the operand is s (q - z), rounded once.
#include "linear_dense.h"
#include "q4.h"

namespace mok {

namespace {

// 4 bytes a lane into LDS at lds + 4 lane (see load_lds_sv for the distances).
__device__ __forceinline__ void dma4_any(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}

template <typename T, class Tl, bool SW>
struct Q4Tile {
  using OA = DenseK<T, Tl::BM, Tl::FM, Tl::NW>;
  static constexpr int BN = 128;
  static constexpr int kA = 3, kRaw = 4;                  // stages
  static constexpr int RAW = 4096 + 1024 + 1024;          // codes, scales, zero points of a K-tile
  static constexpr int A0 = 0, B0 = kA * OA::BYTES, R0 = B0 + 2 * BN * 128, LDS = R0 + kRaw * RAW;
  static constexpr int NL = OA::NI + 3;                   // loads of a wave and K-tile
  static_assert(Tl::BN == BN && Tl::NT == 256 && Tl::FN == 2, "tile");
};

template <typename T, class Tl, bool SW, int G>
__global__ __launch_bounds__(Tl::NT) void q4_tile_kernel(Q4Args qa) {
  using C = Q4Tile<T, Tl, SW>;
  constexpr bool BF = std::is_same<T, bf16>::value;
  constexpr int ES = sizeof(T), BK = 128 / ES;      // values of a K-tile
  constexpr int GP = BK / G > 0 ? BK / G : 1;       // scales of a row in a K-tile
  __shared__ __align__(1024) char smem[C::LDS];
  static_assert(C::LDS <= 160 << 10 && Tl::NW * 32 * kDensePatch * 4 <= C::LDS, "LDS");
  LinearArgs a = qa.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Tl::WN, wn = wave % Tl::WN;
  const int64_t P = SW ? 2 * (int64_t)a.N : a.N;
  constexpr int BNO = SW ? 64 : 128;  // outputs of a tile's columns
  const int NT = (a.N + BNO - 1) / BNO;
  GroupTile t;
  int mt, nt;
  if (qa.off == nullptr) {
    const int MT = (int)((a.M + Tl::BM - 1) / Tl::BM);
    t = {0, 0, (int)a.M, 0, MT};
    band_walk(xcd_logical(blockIdx.x, gridDim.x), MT, NT, mt, nt);
  } else {
    GroupScan scan;
    scan.init(qa.off, qa.E, a.M, Tl::BM);
    const int tiles = scan.total * NT;
    if ((int)blockIdx.x >= tiles) return;
    const int L = xcd_logical(blockIdx.x, tiles);
    t = scan.find(L / NT, Tl::BM);
    band_walk(L - t.first * NT, t.tiles, NT, mt, nt);
  }
  const int64_t m0 = t.lo + (int64_t)mt * Tl::BM;
  const int n0 = nt * BNO, rows = (int)min<int64_t>(t.hi - m0, Tl::BM);
  const uint32_t K = (uint32_t)a.K, KG = K / G;
  // first output column of tile column j, and its row of w (columns past N re-read the last one)
  const auto col = [&](int j) { return SW ? n0 + (j / 64) * 32 + (j & 31) : n0 + j; };
  const auto wrow = [&](int j) { return t.g * P + min(col(j), a.N - 1) + (SW && (j & 32) ? a.N : 0); };

  const auto frow_a = [&](int f) { return wm * Tl::WTM + f * 32; };
  typename C::OA oa;
  oa.init((const T*)a.a + m0 * K, 0, K, [&](int row) { return (uint32_t)min(row, rows - 1) * (uint32_t)(ES * K); }, frow_a,
          wave, lane);
  // Raw loads of this lane: 16 bytes of codes of row tid / 2 (bf16: half tid % 2 of its K-tile; fp32: a row is 16
  // bytes, rows tid % 128); scale and zero point of row tid / 2 (group tid % 2 of the K-tile, if it has two).
  const uint8_t* wq = (const uint8_t*)a.b + wrow(BF ? tid >> 1 : tid & 127) * (K / 2);
  const uint64_t sg = (uint64_t)wrow(tid >> 1) * KG;
  const uint32_t lds = lds_offset(smem);
  const auto issue_raw = [&](uint32_t kt) {
    const uint32_t to = lds + C::R0 + kt % C::kRaw * C::RAW + wave * 1024;
    const uint32_t part = BF ? 16 * (tid & 1) : 0;
    C::OA::dma16_any((const char*)wq + min(kt * (BK / 2) + part, K / 2 - 16), to);
    const uint64_t i = sg + min(kt * BK / G + (GP > 1 ? tid & 1 : 0), KG - 1);
    const uint32_t ts = lds + C::R0 + kt % C::kRaw * C::RAW + 4096 + wave * 256;
    dma4_any((const char*)qa.s + (i * ES & ~3ull), ts);
    dma4_any(qa.z + (i & ~3ull), ts + 1024);
  };
  // The codes of K-tile kt as operands in B's stage: this thread's 32 (fp32: 16) of row tid / 2.
  const uint32_t sg_lo = (uint32_t)sg;
  const int brow = tid >> 1, part = tid & 1;
  const auto operand = [&](uint32_t kt) {
    const char* raw = smem + C::R0 + kt % C::kRaw * C::RAW;
    char* to = smem + C::B0 + (kt & 1) * (C::BN * 128) + brow * 128;
    const uint32_t i = sg_lo + min(kt * BK / G + (GP > 1 ? part : 0), KG - 1);
    const uint32_t zr = *reinterpret_cast<const uint32_t*>(raw + 4096 + 1024 + 4 * tid);
    const float z = qa.zeros ? (float)(zr >> ((i & 3) * 8) & 0xFFu) : 8.0f;
    if constexpr (BF) {
      const uint4 w = *reinterpret_cast<const uint4*>(raw + 16 * tid);
      const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t lo = wd[u] & 0x0F0F0F0Fu, hi = wd[u] >> 4 & 0x0F0F0F0Fu;
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = (float)((c & 1 ? hi : lo) >> (8 * (c / 2)) & 0xFFu) - z;
        *reinterpret_cast<uint4*>(to + 16 * ((4 * part + u) ^ swz_k(brow))) = pack(f, (bf16*)nullptr);
      }
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(raw + 16 * brow + 8 * part);
      const float s = *reinterpret_cast<const float*>(raw + 4096 + 4 * tid);
      const uint32_t wd[2] = {w.x, w.y};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float f[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = s * ((float)(wd[u / 2] >> (16 * (u % 2) + 4 * c) & 15u) - z);
        *reinterpret_cast<uint4*>(to + 16 * ((4 * part + u) ^ swz_k(brow))) = pack(f, (float*)nullptr);
      }
    }
  };
  uint32_t foff[2][4];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int row = wn * Tl::WTN + f * 32 + (lane & 31);
      foff[f][ks] = row * 128 + 16 * ((2 * ks + (lane >> 5)) ^ swz_k(row));
    }

  f32x16_t acc[Tl::FM][2], grp[Tl::FM][2];  // fp32: grp is not used
  zero_acc<Tl>(acc);
  if constexpr (BF) zero_acc<Tl>(grp);
  const uint32_t KT = (K + BK - 1) / BK;
  // acc += scale * grp for the group that ends in K-tile kt (group h of it)
  const auto flush = [&](uint32_t kt, int h) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int j = wn * Tl::WTN + f * 32 + (lane & 31);
      const uint32_t i = (uint32_t)wrow(j) * KG + min(kt * BK / G + h, KG - 1);
      const uint32_t sr = *reinterpret_cast<const uint32_t*>(smem + C::R0 + kt % C::kRaw * C::RAW + 4096 + 4 * (2 * j + h));
      const float s = __uint_as_float(sr >> ((i & 1) * 16) << 16);
#pragma unroll
      for (int m = 0; m < Tl::FM; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          acc[m][f][r] = __builtin_fmaf(s, grp[m][f][r], acc[m][f][r]);
          grp[m][f][r] = 0.0f;
        }
    }
  };

  // Loads of K-tile kt: x two K-tiles ahead, codes three (past the end: again the last ones, which no one reads).
  const auto issue = [&](uint32_t kt_a, uint32_t kt_raw) {
    const uint32_t to = lds + C::A0 + kt_a % C::kA * C::OA::BYTES;
    oa.template issue<false>(min(kt_a, KT - 1), to, wave);
    issue_raw(kt_raw);
  };
  issue_raw(0);
  issue(0, 1);
  issue(1, 2);
  wait_vmcnt<2 * C::NL>();
  ring_barrier();
  operand(0);
  for (uint32_t kt = 0; kt < KT; ++kt) {
    wait_vmcnt<C::NL>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    issue(kt + 2, kt + 3);
    const char* sa = smem + C::A0 + kt % C::kA * C::OA::BYTES;
    const char* sb = smem + C::B0 + (kt & 1) * (C::BN * 128);
    operand(kt + 1);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint4 fa[Tl::FM], fb[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) fb[f] = *reinterpret_cast<const uint4*>(sb + foff[f][ks]);
#pragma unroll
      for (int m = 0; m < Tl::FM; ++m) fa[m] = oa.frag(sa, m, ks);
#pragma unroll
      for (int m = 0; m < Tl::FM; ++m)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          if constexpr (BF) Mma<T>::run(grp[m][f], fa[m], fb[f]);
          else Mma<T>::run(acc[m][f], fa[m], fb[f]);
        }
      if constexpr (BF && G == 32)
        if (ks == 1) flush(kt, 0);
    }
    if constexpr (BF) {
      if (G == 32) flush(kt, 1);
      else if (((kt + 1) * BK) % G == 0 || kt + 1 == KT) flush(kt, 0);
    }
  }
  wait_vmcnt<0>();
  __syncthreads();

  // A lane holds 16 rows of a column: through a patch of LDS to eight columns of a row.
  float* patch = reinterpret_cast<float*>(smem) + wave * (32 * kDensePatch);
  constexpr int LPR = SW ? 4 : 8;
  const float* bias = a.bias != nullptr ? a.bias + t.g * P : nullptr;
#pragma unroll
  for (int m = 0; m < Tl::FM; ++m) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        patch[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * kDensePatch + 32 * f + (lane & 31)] = acc[m][f][r];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < LPR / 2; ++i) {
      const int row = lane / LPR + (64 / LPR) * i, c = (lane % LPR) * 8;
      const int mm = wm * Tl::WTM + m * 32 + row, cc = col(wn * Tl::WTN + c);
      if (mm < rows && cc < a.N) {
        const Raw8<T> add = linear_add8<T>(a, m0 + mm, cc);
        float p[8], u[8];
        load8(patch + row * kDensePatch + c, p);
        if constexpr (SW) load8(patch + row * kDensePatch + 32 + c, u);
        q4_finish<T, SW>(a, bias, qa.epi, m0 + mm, cc, p, u, add);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, class Tl, bool SW>
void run_tile(const Q4Args& a, hipStream_t s) {
  const int bno = SW ? 64 : 128;
  const dim3 grid((unsigned)(q4_tiles_bound(a, Tl::BM) * ((a.l.N + bno - 1) / bno)));
  if (a.group == 32) hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 32>), grid, dim3(Tl::NT), 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 64>), grid, dim3(Tl::NT), 0, s, a);
  else hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 128>), grid, dim3(Tl::NT), 0, s, a);
}

template <typename T, class Tl>
void run_tile(const Q4Args& a, hipStream_t s) {
  if (a.epi == MOK_EPI_SWIGLU) run_tile<T, Tl, true>(a, s);
  else run_tile<T, Tl, false>(a, s);
}

}  // namespace

hipError_t launch_q4_tile(const Q4Args& a, int act, int bm, hipStream_t s) {
  if (act == MOK_F32) run_tile<float, Tiling<128, 128, 2, 2>>(a, s);
  else if (bm == 256) run_tile<bf16, Tiling<256, 128, 2, 2>>(a, s);
  else run_tile<bf16, Tiling<128, 128, 2, 2>>(a, s);
  return hipGetLastError();
}

}  // namespace mok
