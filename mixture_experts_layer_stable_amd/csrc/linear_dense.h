// bf16 matrix product on direct global->LDS loads, for the products of linear.hip.
//
// A workgroup multiplies one BM x BN tile, each wave its part of it; both operands
// of a 64-element K-tile arrive in LDS stages by global_load_lds_dwordx4 (gemm2.h's tile layouts,
// with ragged edges). With 256 x 256 tiles a SIMD holds one wave (256 fp32
// accumulators per lane), so nothing but the order of its own instructions hides its loads: every
// LDS read and DMA of the loop has its place between two MFMAs (see dense_tile).
#pragma once
#include "gemm2.h"
#include "linear.h"

namespace mok {

// LDS byte offset of a shared array (wave-uniform).
__device__ __forceinline__ uint32_t lds_offset(const char* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)p);
}

__device__ __forceinline__ void dma16_at(const char* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(sbase) : "memory", "m0");
}

static __device__ uint4 g_zero_16 = {};  // what is read past the end of K

// K-contiguous operand: tile row r starts at sbase + voff(r); K-tile kt is its bytes
// 128 kt .. +127, chunks at or past K read zeros.
// SW: 32-row blocks of the tile come in turn from the rows at sbase and from those at sbase + up
// (gate and up rows of w); a DMA instruction's 8 rows lie in one block.
template <int ROWS, int NF, int NW, bool SW = false>
struct DenseK {
  static constexpr int BYTES = ROWS * 128;
  static constexpr int NI = ROWS / (8 * NW);  // DMA instructions per wave per stage (8 rows each)
  static_assert(ROWS % (8 * NW) == 0, "rows");
  const char* sbase;
  int64_t up, kbytes;  // kbytes = 2 K
  uint32_t voff[NI];
  uint32_t foff[NF][4];

  // rowoff(row): byte offset of the row from its base (below 4 GiB); frow(f): first tile row of
  // fragment f.
  template <class F, class G>
  __device__ __forceinline__ void init(const void* base, int64_t up_, int64_t K, F rowoff, G frow, int wave, int lane) {
    sbase = reinterpret_cast<const char*>(base);
    up = up_;
    kbytes = 2 * K;
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
      for (int j = j0; j < j1; ++j) dma16_at(uniform_ptr(base(kt, j, wave)), voff[j], lds + (wave + NW * j) * 1024);
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
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    return *reinterpret_cast<const uint4*>(stage + foff[f][ks]);
  }
};

// MN-contiguous operand: k-row k of the tile starts at sbase + k * ld bytes; 64 k-rows x ROWS
// bf16 per stage. Rows at or past K read zeros, 16-byte column chunks at or past `cols` read the
// row's first chunk (their results are not stored).
template <int ROWS, int NF, int NW>
struct DenseMN {
  static constexpr int PITCH = ROWS * 2;
  static constexpr int BYTES = 64 * PITCH;
  static constexpr int NI = BYTES / (1024 * NW);
  static_assert(BYTES % (1024 * NW) == 0 && PITCH <= 1024, "tile");
  // chunk c of k-row k lies at chunk c ^ swz(k): the four rows that a transposing read covers are
  // on distinct banks (rows of 64 bytes are by themselves, of 128 bytes every other one)
  static __device__ __forceinline__ int swz(int k) { return ROWS >= 128 ? 4 * (k & 3) : (ROWS == 64 ? 2 * (k & 2) : 0); }
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
      voff[j] = (uint32_t)(kr * ld_bytes) + (8 * ch < cols ? 16u * (uint32_t)ch : 0u);
    }
    const int g = lane >> 4, i = lane & 15;
    const int k0 = 8 * (g >> 1) + (i >> 2);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int mn = fcol(f) + 16 * (g & 1) + 4 * (i & 3);
      foff[f] = k0 * PITCH + 16 * ((mn >> 3) ^ swz(k0)) + 2 * (mn & 7);
    }
  }
  __device__ __forceinline__ int64_t full() const { return K / 64; }
  template <bool FULL>
  __device__ __forceinline__ void issue(int64_t kt, uint32_t lds, int wave, int j0 = 0, int j1 = NI) const {
    const int64_t k0 = kt * 64;
    if (FULL || k0 + 64 <= K) {
      const char* b = uniform_ptr(sbase + k0 * ld);
#pragma unroll
      for (int j = j0; j < j1; ++j) dma16_at(b, voff[j], lds + (wave + NW * j) * 1024);
    } else {
#pragma unroll
      for (int j = j0; j < j1; ++j) {
        const int kr = ((wave + NW * j) * 1024 + 16 * (int)(threadIdx.x & 63)) / PITCH;
        const char* p = k0 + kr < K ? sbase + k0 * ld + voff[j] : reinterpret_cast<const char*>(&g_zero_16);
        DenseK<32 * NW, 1, NW>::dma16_any(p, lds + (wave + NW * j) * 1024);
      }
    }
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    const char* a = stage + foff[f] + ks * 16 * PITCH;
    return tr_pair(a, a + 4 * PITCH);
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

// One K-tile, whose first fragments are in a[0], b[0]. A 16-k step is NM MFMAs; behind each of its
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
template <class Tl, bool FULL, int BST, class OA, class OB>
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
      Mma<bf16>::run(acc[i / Tl::FN][i % Tl::FN], b[c][i % Tl::FN], a[c][i / Tl::FN]);
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
template <class Tl, int BST, class OA, class OB>
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
    dense_tile<Tl, true, BST>(oa, ob, kt, kt1, ring, wave, a, b, acc);
#pragma unroll 1
  for (; kt < kt1; ++kt, ring.next()) dense_tile<Tl, false, BST>(oa, ob, kt, kt1, ring, wave, a, b, acc);
  __syncthreads();
}

// Hands the transposed blocks of dense_loop back through a per-wave LDS patch, every lane owning
// eight consecutive columns of a row: store(pair, row, col, g, u, add), pair the index of its 64
// columns in the wave's tile, row and col in the workgroup's; with SW, u are the same columns of the up block 32 to the right. add is what load(row, col)
// gave, called kAhead block pairs earlier: alone on its SIMD a wave would wait out each load's
// latency (8192 x 7168 x 4096 with an addend: 467 us, 422 ahead). The patch's row pitch keeps the
// 16-byte writes of the 32 rows on distinct banks; a wave's LDS operations run in order.
constexpr int kDensePatch = 68;  // floats

template <class Tl, bool SW, class L, class F>
__device__ __forceinline__ void dense_epilogue(f32x16_t (&acc)[Tl::FM][Tl::FN], char* smem, int wave, int wm, int wn,
                                               int lane, L&& load, F&& store) {
  static_assert(Tl::FN % 2 == 0, "blocks are handed back in horizontal pairs");
  constexpr int NP = Tl::FM * Tl::FN / 2, kAhead = NP < 3 ? NP : 3;  // block pairs
  constexpr int LPR = SW ? 4 : 8, NI = LPR / 2;                      // lanes of a row, passes of a pair
  float* patch = reinterpret_cast<float*>(smem) + wave * (32 * kDensePatch);
  const int m = lane & 31, h = lane >> 5;
  const int r0 = wm * Tl::WTM + lane / LPR, c0 = (lane % LPR) * 8;
  decltype(load(0, 0)) raw[kAhead][NI];
  const auto fetch = [&](auto pc) {
    constexpr int p = decltype(pc)::value, fm = 2 * p / Tl::FN, fn = 2 * p % Tl::FN;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      raw[p % kAhead][i] = load(r0 + fm * 32 + (64 / LPR) * i, wn * Tl::WTN + fn * 32 + c0);
  };
  static_for<0, kAhead>([&](auto pc) { fetch(pc); });
  static_for<0, NP>([&](auto pc) {
    constexpr int p = decltype(pc)::value, fm = 2 * p / Tl::FN, fn = 2 * p % Tl::FN;
#pragma unroll
    for (int b = 0; b < 2; ++b)
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
      store(std::integral_constant<int, fn / 2>(), r0 + fm * 32 + (64 / LPR) * i, wn * Tl::WTN + fn * 32 + c0, g8, u8, raw[p % kAhead][i]);
    }
    if constexpr (p + kAhead < NP) fetch(std::integral_constant<int, p + kAhead>());
  });
}

}  // namespace mok
