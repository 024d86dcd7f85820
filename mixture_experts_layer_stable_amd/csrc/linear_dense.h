// Matrix product on direct global->LDS loads, for the products of linear.hip (bf16, fp32).
//
// A workgroup multiplies one BM x BN tile, each wave its part of it; both operands of a K-tile (128
// bytes of K: 64 bf16, 32 fp32) arrive in LDS stages by global_load_lds_dwordx4 (gemm2.h's tile
// layouts, with ragged edges). With 256 x 256 tiles a SIMD holds one wave (256 fp32 accumulators per
// lane), so nothing but the order of its own instructions hides its loads: every LDS read and DMA of
// the loop has its place between two MFMAs (see dense_tile). fp32 is bound by its MFMAs, at 64 cycles
// each (8192 x 4096 x 4096: 143 TFLOP/s; staged through registers 128).
#pragma once
#include "gemm2.h"
#include "linear.h"

namespace mok {

// LDS byte offset of a shared array (wave-uniform).
__device__ __forceinline__ uint32_t lds_offset(const char* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)p);
}

static __device__ uint4 g_zero_16 = {};  // what is read past the end of K

// K-contiguous operand: tile row r starts at sbase + voff(r); K-tile kt is its bytes
// 128 kt .. +127, chunks at or past K read zeros.
// SW: 32-row blocks of the tile come in turn from the rows at sbase and from those at sbase + up
// (gate and up rows of w); a DMA instruction's 8 rows lie in one block.
template <typename T, int ROWS, int NF, int NW, bool SW = false>
struct DenseK {
  static constexpr int BYTES = ROWS * 128;
  static constexpr int NI = ROWS / (8 * NW);  // DMA instructions per wave per stage (8 rows each)
  static_assert(ROWS % (8 * NW) == 0, "rows");
  const char* sbase;
  int64_t up, kbytes;  // of a row's K
  uint32_t voff[NI];
  uint32_t foff[NF][4];

  // rowoff(row): byte offset of the row from its base (below 4 GiB); frow(f): first tile row of
  // fragment f.
  template <class F, class G>
  __device__ __forceinline__ void init(const void* base, int64_t up_, int64_t K, F rowoff, G frow, int wave, int lane) {
    sbase = reinterpret_cast<const char*>(base);
    up = up_;
    kbytes = (int64_t)sizeof(T) * K;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = 8 * (wave + NW * j) + (lane >> 3);
      voff[j] = rowoff(row) + 16u * (uint32_t)((lane & 7) ^ swz_k(row));
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int row = frow(f) + (lane & 31);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) foff[f][ks] = row * 128 + 16 * ((2 * ks + (lane >> 5)) ^ swz_k(row));
    }
  }
  __device__ __forceinline__ int64_t full() const { return kbytes / 128; }  // K-tiles that have all of their K
  __device__ __forceinline__ const char* base(int64_t kt, int j, int wave) const {
    const char* b = sbase + kt * 128;
    if constexpr (SW) b += ((wave + NW * j) >> 2) & 1 ? up : 0;
    return b;
  }
  // DMA instructions j0 .. j1-1 of K-tile kt into the stage at LDS offset lds; FULL: kt < full()
  template <bool FULL>
  __device__ __forceinline__ void issue(int64_t kt, uint32_t lds, int wave, int j0 = 0, int j1 = NI) const {
    if (FULL || (kt + 1) * 128 <= kbytes) {
#pragma unroll
      for (int j = j0; j < j1; ++j)
        load_lds_sv<16>(uniform_ptr(base(kt, j, wave)), voff[j], lds + (wave + NW * j) * 1024);
    } else {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int j = j0; j < j1; ++j) {
        const int row = 8 * (wave + NW * j) + (lane >> 3);
        const int ch = (lane & 7) ^ swz_k(row);
        const char* p = kt * 128 + 16 * ch < kbytes ? base(kt, j, wave) + voff[j]
                                                    : reinterpret_cast<const char*>(&g_zero_16);
        dma16_any(p, lds + (wave + NW * j) * 1024);
      }
    }
  }
  __device__ __forceinline__ static void dma16_any(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 ::"s"(lds), "v"(p) : "memory", "m0");
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    return *reinterpret_cast<const uint4*>(stage + foff[f][ks]);
  }
};

// MN-contiguous operand: k-row k of the tile starts at sbase + k * ld bytes; KR k-rows of ROWS
// elements per stage. Rows at or past K read zeros, 16-byte column chunks at or past `cols` read the
// row's first chunk (their results are not stored).
template <typename T, int ROWS, int NF, int NW>
struct DenseMN {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int KR = kRowBytes / (int)sizeof(T), VE = Elem<T>::VE;
  static constexpr int PITCH = ROWS * (int)sizeof(T);
  static constexpr int BYTES = KR * PITCH;
  static constexpr int NI = BYTES / (1024 * NW);
  static_assert(BYTES % (1024 * NW) == 0 && PITCH <= 1024, "tile");
  // chunk c of k-row k lies at chunk c ^ swz(k). bf16: the four rows that a transposing read covers are
  // on distinct banks (rows of 64 bytes are by themselves, of 128 bytes every other one). fp32: so are
  // the 32 columns of rows k and k + 4 that a fragment's 4-byte read takes.
  static __device__ __forceinline__ int swz(int k) {
    if constexpr (F32) return ROWS >= 64 ? 2 * (k & 4) : 0;
    return ROWS >= 128 ? 4 * (k & 3) : (ROWS == 64 ? 2 * (k & 2) : 0);
  }
  const char* sbase;
  int64_t ld, K;
  uint32_t voff[NI];
  uint32_t foff[NF];

  template <class G>
  __device__ __forceinline__ void init(const void* base, int64_t ld_bytes, int64_t K_, int64_t cols, G fcol, int wave,
                                       int lane) {
    sbase = reinterpret_cast<const char*>(base);
    ld = ld_bytes;
    K = K_;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int o = (wave + NW * j) * 1024 + 16 * lane, kr = o / PITCH;
      const int ch = ((o % PITCH) >> 4) ^ swz(kr);
      voff[j] = (uint32_t)(kr * ld_bytes) + (VE * ch < cols ? 16u * (uint32_t)ch : 0u);
    }
    const int g = lane >> 4, i = lane & 15;
    const int k0 = F32 ? 4 * (lane >> 5) : 8 * (g >> 1) + (i >> 2);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int mn = fcol(f) + (F32 ? lane & 31 : 16 * (g & 1) + 4 * (i & 3));
      foff[f] = k0 * PITCH + 16 * ((mn / VE) ^ swz(k0)) + (int)sizeof(T) * (mn % VE);
    }
  }
  __device__ __forceinline__ int64_t full() const { return K / KR; }
  template <bool FULL>
  __device__ __forceinline__ void issue(int64_t kt, uint32_t lds, int wave, int j0 = 0, int j1 = NI) const {
    const int64_t k0 = kt * KR;
    if (FULL || k0 + KR <= K) {
      const char* b = uniform_ptr(sbase + k0 * ld);
#pragma unroll
      for (int j = j0; j < j1; ++j) load_lds_sv<16>(b, voff[j], lds + (wave + NW * j) * 1024);
    } else {
#pragma unroll
      for (int j = j0; j < j1; ++j) {
        const int kr = ((wave + NW * j) * 1024 + 16 * (int)(threadIdx.x & 63)) / PITCH;
        const char* p = k0 + kr < K ? sbase + k0 * ld + voff[j] : reinterpret_cast<const char*>(&g_zero_16);
        DenseK<T, 32 * NW, 1, NW>::dma16_any(p, lds + (wave + NW * j) * 1024);
      }
    }
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    const char* a = stage + foff[f] + ks * (KR / 4) * PITCH;
    if constexpr (F32) {
      const auto at = [&](int k) { return *reinterpret_cast<const uint32_t*>(a + k * PITCH); };
      return make_uint4(at(0), at(1), at(2), at(3));
    } else {
      return tr_pair(a, a + 4 * PITCH);
    }
  }
};

// LDS stages: two of A, and of B two, or three where they fit the workgroup's share (256 x 256 tiles:
// all 160 KB), whose third lets B be loaded a K-tile earlier.
template <class OA, class OB, int BST>
struct DenseRing {
  static constexpr int BYTES = 2 * OA::BYTES + BST * OB::BYTES;
  char* smem;
  uint32_t lds;
  int a0 = 0, b0 = 0;  // stages of the current K-tile
  __device__ __forceinline__ int a_off(int d) const { return (a0 ^ (d & 1)) * OA::BYTES; }
  __device__ __forceinline__ int b_off(int d) const {  // d < BST
    const int q = b0 + d;
    return 2 * OA::BYTES + (q >= BST ? q - BST : q) * OB::BYTES;
  }
  __device__ __forceinline__ void next() {
    a0 ^= 1;
    b0 = b0 + 1 == BST ? 0 : b0 + 1;
  }
};

// One K-tile, whose first fragments are in a[0], b[0]. A step of a quarter of it is NM MFMAs (of
// 16 k; fp32: four times as many of 2 k); behind each of its
// first ones goes a fragment read of the next step. At the last step the wave holds every fragment
// that it needs of the K-tile: it waits for its own loads of K-tile kt+1 and for the workgroup, then
// reads that tile's first fragments and loads kt+2's A into the stage that has become free, between
// the step's MFMAs. B's loads (of kt+2, or of kt+1 with two stages) go out in another step, so the
// memory system sees two smaller bursts. sched_barrier keeps each where it is put: left to itself the
// compiler gathers reads before the MFMAs (16384 x 4096 x 7168: 860 us, 810 placed; an MFMA takes 32
// cycles, room for its neighbour's few scalar and address instructions). B's third stage: 748 ->
// 738 us, 387 -> 379 for the weight gradient. FULL: kt + 2 lies below the operands' full(), so no
// condition stays in the loop (with conditions around the loads: 990 us). 16 x 16 x 32 MFMAs need
// twice the fragments, and spill.
template <typename T, class Tl, bool FULL, int BST, class OA, class OB>
__device__ __forceinline__ void dense_tile(const OA& oa, const OB& ob, int64_t kt, int64_t kt1,
                                           const DenseRing<OA, OB, BST>& ring, int wave, uint4 (&a)[2][Tl::FM],
                                           uint4 (&b)[2][Tl::FN], f32x16_t (&acc)[Tl::FM][Tl::FN]) {
  constexpr int NM = Tl::FM * Tl::FN, NR = Tl::FM + Tl::FN, RS = (NR + NM - 1) / NM;
  constexpr int HALF = NM > 1 ? NM / 2 : 1;         // MFMA slots that an operand's loads are spread over
  constexpr int BKS = BST == 3 ? 1 : 0, BS0 = BST == 3 ? 0 : NM / 4;  // step and slot of B's first load
  const bool more1 = FULL || kt + 1 < kt1, more2 = FULL || kt + 2 < kt1, moreb = BST == 3 ? more2 : more1;
  static_for<0, 4>([&](auto kc) {
    constexpr int ks = decltype(kc)::value, c = ks & 1;
    if constexpr (ks == 3) {
      if (BST == 3 && more2) wait_vmcnt<OB::NI>();  // all but B of kt+2
      else wait_vmcnt<0>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    const char* fa = ring.smem + ring.a_off(ks == 3);
    const char* fb = ring.smem + ring.b_off(ks == 3);
    static_for<0, NM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      Mma<T>::run(acc[i / Tl::FN][i % Tl::FN], b[c][i % Tl::FN], a[c][i / Tl::FN]);
      if (ks < 3 || more1) {
        static_for<RS * i, (RS * (i + 1) < NR ? RS * (i + 1) : NR)>([&](auto rc) {
          constexpr int r = decltype(rc)::value;
          if constexpr (r < Tl::FN) b[c ^ 1][r] = ob.frag(fb, r, (ks + 1) & 3);
          else a[c ^ 1][r - Tl::FN] = oa.frag(fa, r - Tl::FN, (ks + 1) & 3);
        });
      }
      constexpr int sa = i - (NM - HALF), sb = i - BS0;
      if constexpr (ks == 3 && sa >= 0)
        if (more2)
          oa.template issue<FULL>(kt + 2, ring.lds + ring.a_off(0), wave, sa * OA::NI / HALF, (sa + 1) * OA::NI / HALF);
      if constexpr (ks == BKS && sb >= 0 && sb < HALF)
        if (moreb)
          ob.template issue<FULL>(kt + BST - 1, ring.lds + ring.b_off(BST - 1), wave, sb * OB::NI / HALF,
                                  (sb + 1) * OB::NI / HALF);
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// acc += the products of K-tiles kt0 .. kt1-1 (kt1 > kt0). smem: the ring. The MFMA operands are
// swapped (transposed blocks): a lane then holds 16 columns of one row.
template <typename T, class Tl, int BST, class OA, class OB>
__device__ __forceinline__ void dense_loop(const OA& oa, const OB& ob, int64_t kt0, int64_t kt1, char* smem, int wave,
                                           f32x16_t (&acc)[Tl::FM][Tl::FN]) {
  DenseRing<OA, OB, BST> ring{smem, lds_offset(smem)};
  oa.template issue<false>(kt0, ring.lds + ring.a_off(0), wave);
  ob.template issue<false>(kt0, ring.lds + ring.b_off(0), wave);
  if (kt0 + 1 < kt1) {
    oa.template issue<false>(kt0 + 1, ring.lds + ring.a_off(1), wave);
    if (BST == 3) ob.template issue<false>(kt0 + 1, ring.lds + ring.b_off(1), wave);
    wait_vmcnt<OA::NI + (BST == 3 ? OB::NI : 0)>();
  } else {
    wait_vmcnt<0>();
  }
  ring_barrier();
  uint4 a[2][Tl::FM], b[2][Tl::FN];
#pragma unroll
  for (int fm = 0; fm < Tl::FM; ++fm) a[0][fm] = oa.frag(smem + ring.a_off(0), fm, 0);
#pragma unroll
  for (int fn = 0; fn < Tl::FN; ++fn) b[0][fn] = ob.frag(smem + ring.b_off(0), fn, 0);
  int64_t kt = kt0;
  for (const int64_t full = min(kt1, oa.full()); kt + 2 < full; ++kt, ring.next())
    dense_tile<T, Tl, true, BST>(oa, ob, kt, kt1, ring, wave, a, b, acc);
#pragma unroll 1
  for (; kt < kt1; ++kt, ring.next()) dense_tile<T, Tl, false, BST>(oa, ob, kt, kt1, ring, wave, a, b, acc);
  __syncthreads();
}

// Hands the transposed blocks of dense_loop back through a per-wave LDS patch, every lane owning
// eight consecutive columns of a row: store(pair, row, col, g, u, add), pair the index of its 64
// columns in the wave's tile, row and col in the workgroup's; with SW, u are the same columns of the
// up block 32 to the right. add is what load(row, col) gave, called kAhead block pairs earlier: alone
// on its SIMD a wave would wait out each load's latency (8192 x 7168 x 4096 with an addend: 467 us,
// 422 ahead). The patch's row pitch keeps the 16-byte writes of the 32 rows on distinct banks; a
// wave's LDS operations run in order. Wave tiles of 32 columns go block by block.
constexpr int kDensePatch = 68;  // floats
template <class Tl, bool SW>
constexpr int kDenseLanes = SW || Tl::FN % 2 ? 4 : 8;  // lanes of a row

template <class Tl, bool SW, class L, class F>
__device__ __forceinline__ void dense_epilogue(f32x16_t (&acc)[Tl::FM][Tl::FN], char* smem, int wave, int wm, int wn,
                                               int lane, L&& load, F&& store) {
  constexpr int NB = Tl::FN % 2 ? 1 : 2;                              // blocks at a time
  static_assert(!SW || NB == 2, "gate and up blocks side by side");
  constexpr int NP = Tl::FM * Tl::FN / NB, kAhead = NP < 3 ? NP : 3;  // block pairs
  constexpr int LPR = kDenseLanes<Tl, SW>, NI = LPR / 2;              // passes of a pair
  float* patch = reinterpret_cast<float*>(smem) + wave * (32 * kDensePatch);
  const int m = lane & 31, h = lane >> 5;
  const int r0 = wm * Tl::WTM + lane / LPR, c0 = (lane % LPR) * 8;
  decltype(load(0, 0)) raw[kAhead][NI];
  const auto fetch = [&](auto pc) {
    constexpr int p = decltype(pc)::value, fm = NB * p / Tl::FN, fn = NB * p % Tl::FN;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      raw[p % kAhead][i] = load(r0 + fm * 32 + (64 / LPR) * i, wn * Tl::WTN + fn * 32 + c0);
  };
  static_for<0, kAhead>([&](auto pc) { fetch(pc); });
  static_for<0, NP>([&](auto pc) {
    constexpr int p = decltype(pc)::value, fm = NB * p / Tl::FN, fn = NB * p % Tl::FN;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(patch + m * kDensePatch + 32 * b + 8 * g + 4 * h) =
            make_float4(acc[fm][fn + b][4 * g], acc[fm][fn + b][4 * g + 1], acc[fm][fn + b][4 * g + 2],
                        acc[fm][fn + b][4 * g + 3]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float* q = patch + (lane / LPR + (64 / LPR) * i) * kDensePatch + c0;
      float g8[8], u8[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(q + 4 * k);
        const float4 u = SW ? *reinterpret_cast<const float4*>(q + 32 + 4 * k) : v;
        g8[4 * k] = v.x; g8[4 * k + 1] = v.y; g8[4 * k + 2] = v.z; g8[4 * k + 3] = v.w;
        u8[4 * k] = u.x; u8[4 * k + 1] = u.y; u8[4 * k + 2] = u.z; u8[4 * k + 3] = u.w;
      }
      store(std::integral_constant<int, fn / NB>(), r0 + fm * 32 + (64 / LPR) * i, wn * Tl::WTN + fn * 32 + c0, g8, u8,
            raw[p % kAhead][i]);
    }
    if constexpr (p + kAhead < NP) fetch(std::integral_constant<int, p + kAhead>());
  });
}

constexpr int kBand = 8;  // tile rows of a band of the tile walk

// PART: the tile's sums over this slice of K go to a.part; linear_join_kernel adds the slices.
template <typename T, class Tl, int KIND, int EPI, typename TO, bool PART>
__global__ __launch_bounds__(Tl::NT) void linear_dense_kernel(LinearArgs a) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  // 256 x 256 tiles belong to outputs that no cache keeps: stored past L2, they leave it to the
  // operands' bands (16384 x (2 x 2048) x 7168: 818 -> 745 us)
  constexpr bool NTS = Tl::BM * Tl::BN >= 256 * 256;
  using OA = std::conditional_t<KIND == LIN_DW, DenseMN<T, Tl::BM, Tl::FM, Tl::NW>, DenseK<T, Tl::BM, Tl::FM, Tl::NW>>;
  using OB =
      std::conditional_t<KIND == LIN_FWD, DenseK<T, Tl::BN, Tl::FN, Tl::NW, SW>, DenseMN<T, Tl::BN, Tl::FN, Tl::NW>>;
  constexpr int64_t ES = sizeof(T), BKE = kRowBytes / ES;
  constexpr int PATCH = Tl::NW * 32 * kDensePatch * 4;
  // B's third LDS stage where as many workgroups of it fit a CU's 160 KB as of two stages (fp32 64 x 64
  // tiles, 1 x 4096 x 4096: 33 -> 25 us; with fewer workgroups it costs more than it gives)
  constexpr int kCuLds = 160 << 10;
  constexpr int BST = kCuLds / DenseRing<OA, OB, 3>::BYTES == kCuLds / DenseRing<OA, OB, 2>::BYTES ? 3 : 2;
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
  const int64_t KT = (a.K + BKE - 1) / BKE, kt0 = KT * slice / a.split, kt1 = KT * (slice + 1) / a.split;

  const auto frow_a = [&](int f) { return wm * Tl::WTM + f * 32; };
  const auto frow_b = [&](int f) { return wn * Tl::WTN + f * 32; };
  // first output column of tile column j (SWIGLU: 32-column blocks of gate and up in turn)
  const auto col = [&](int j) { return SW ? n0 + (j / 64) * 32 + (j & 31) : n0 + j; };
  const T* A = (const T*)a.a;
  const T* B = (const T*)a.b;
  OA oa;
  OB ob;
  if constexpr (KIND == LIN_DW) {
    oa.init(A + m0, ES * a.M, a.K, a.M - m0, frow_a, wave, lane);
  } else {
    const int last = (int)min<int64_t>(a.M - 1 - m0, Tl::BM - 1);  // rows past M re-read the last one
    oa.init(A + m0 * a.K, 0, a.K, [&](int row) { return (uint32_t)min(row, last) * (uint32_t)(ES * a.K); }, frow_a, wave,
            lane);
  }
  if constexpr (KIND == LIN_FWD) {
    ob.init(B + (int64_t)n0 * a.K, ES * a.N * a.K, a.K,
            [&](int j) { return (uint32_t)(min(col(j), a.N - 1) - n0) * (uint32_t)(ES * a.K); }, frow_b, wave, lane);
  } else {
    ob.init(B + n0, ES * a.N, a.K, a.N - n0, frow_b, wave, lane);
  }
  f32x16_t acc[Tl::FM][Tl::FN];
  zero_acc<Tl>(acc);
  if (kt1 > kt0) dense_loop<T, Tl, BST>(oa, ob, kt0, kt1, smem, wave, acc);

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
  constexpr int LPR = kDenseLanes<Tl, SW>, NB = (Tl::FN + 1) / 2;
  float bg[NB][8], bu[NB][8];
#pragma unroll
  for (int p = 0; p < NB; ++p) {
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
        if (in(row, j)) linear_store8<KIND, EPI, TO, T, NTS>(a, m0 + row, col(j), g, u, add);
      });
}

template <typename T, class Tl, int KIND, int EPI, typename TO>
void run_dense(const LinearArgs& a, hipStream_t s) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  const int bn = SW ? Tl::BN / 2 : Tl::BN;
  const int64_t tiles = (int64_t)((a.N + bn - 1) / bn) * ((a.M + Tl::BM - 1) / Tl::BM);
  const dim3 grid((unsigned)(tiles * a.split)), block(Tl::NT);
  if (a.split == 1) {
    hipLaunchKernelGGL((linear_dense_kernel<T, Tl, KIND, EPI, TO, false>), grid, block, 0, s, a);
    return;
  }
  hipLaunchKernelGGL((linear_dense_kernel<T, Tl, KIND, SW ? MOK_EPI_SWIGLU : MOK_EPI_NONE, T, true>), grid, block, 0, s,
                     a);
  linear_join<KIND, EPI, TO, T>(a, s);
}

// The forward passes of a tile.
template <typename T, class Tl>
void run_dense_fwd(const LinearArgs& a, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_dense<T, Tl, LIN_FWD, MOK_EPI_NONE, T>(a, s);
  else if (epi == MOK_EPI_SILU) run_dense<T, Tl, LIN_FWD, MOK_EPI_SILU, T>(a, s);
  else if (epi == MOK_EPI_GELU) run_dense<T, Tl, LIN_FWD, MOK_EPI_GELU, T>(a, s);
  else if constexpr (Tl::FN % 2 == 0) run_dense<T, Tl, LIN_FWD, MOK_EPI_SWIGLU, T>(a, s);  // gate and up side by side
}

}  // namespace mok
