// bf16 matrix product on direct global->LDS loads, for the products of linear.hip.
//
// A workgroup multiplies one BM x BN tile; both operands of a 64-element K-tile arrive in one
// of two LDS stages by global_load_lds_dwordx4 (gemm2.h's tile layouts, with ragged edges).
// A fragment is read one 16-k step ahead of its MFMAs, across the stage change too: at the last
// step of a K-tile a wave holds all fragments it still needs, so the barrier there frees the
// stage for K-tile kt+2's loads while the step's MFMAs still run, and those cover the first
// fragment reads of K-tile kt+1.
#pragma once
#include "gemm2.h"
#include "linear.h"

namespace mok {

static __device__ uint4 g_zero_16 = {};  // what is read past the end of K

// K-contiguous operand: tile row r starts at sbase + voff(r); K-tile kt is its bytes
// 128 kt .. +127, chunks at or past K read the zero block.
// SW: 32-row blocks of the tile come in turn from the rows at sbase and from those at sbase + up
// (gate and up rows of w); an instruction's 8 rows lie in one block.
template <int ROWS, int NF, int NW, bool SW = false>
struct DenseK {
  static constexpr int BYTES = ROWS * 128;
  static constexpr int NI = ROWS / (8 * NW);  // DMA instructions per wave per stage (8 rows each)
  static_assert(ROWS % (8 * NW) == 0, "rows");
  const char* sbase;
  uint32_t voff[NI];
  uint32_t foff[NF][4];
  int64_t kbytes;  // 2 K
  int64_t up;

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
  __device__ __forceinline__ const char* base(int64_t kt, int j, int wave) const {
    const char* b = sbase + kt * 128;
    if constexpr (SW) b += ((wave + NW * j) >> 2) & 1 ? up : 0;
    return b;
  }
  __device__ __forceinline__ void issue(int64_t kt, char* stage, int wave) const {
    if ((kt + 1) * 128 <= kbytes) {
#pragma unroll
      for (int j = 0; j < NI; ++j) dma16_sv(uniform_ptr(base(kt, j, wave)), voff[j], stage + (wave + NW * j) * 1024);
    } else {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int row = 8 * (wave + NW * j) + (lane >> 3);
        const int ch = (lane & 7) ^ swz_k(row);
        const char* p = kt * 128 + 16 * ch < kbytes ? base(kt, j, wave) + voff[j] : reinterpret_cast<const char*>(&g_zero_16);
        dma16(p, stage + (wave + NW * j) * 1024);
      }
    }
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    return *reinterpret_cast<const uint4*>(stage + foff[f][ks]);
  }
};

// MN-contiguous operand: k-row k of the tile starts at sbase + k * ld bytes; 64 k-rows x ROWS
// bf16 per stage. Rows at or past K read the zero block, 16-byte column chunks at or past
// `cols` read the row's first chunk (their results are not stored).
template <int ROWS, int NF, int NW>
struct DenseMN {
  static constexpr int PITCH = ROWS * 2;
  static constexpr int BYTES = 64 * PITCH;
  static constexpr int NI = BYTES / (1024 * NW);
  static_assert(BYTES % (1024 * NW) == 0 && PITCH <= 1024, "tile");
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
      const int ch = ((o % PITCH) >> 4) ^ swz_mn(kr);
      voff[j] = (uint32_t)(kr * ld_bytes) + (8 * ch < cols ? 16u * (uint32_t)ch : 0u);
    }
    const int g = lane >> 4, i = lane & 15;
    const int k0 = 8 * (g >> 1) + (i >> 2);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int mn = fcol(f) + 16 * (g & 1) + 4 * (i & 3);
      foff[f] = k0 * PITCH + 16 * ((mn >> 3) ^ swz_mn(k0)) + 2 * (mn & 7);
    }
  }
  __device__ __forceinline__ void issue(int64_t kt, char* stage, int wave) const {
    const int64_t k0 = kt * 64;
    if (k0 + 64 <= K) {
      const char* b = uniform_ptr(sbase + k0 * ld);
#pragma unroll
      for (int j = 0; j < NI; ++j) dma16_sv(b, voff[j], stage + (wave + NW * j) * 1024);
    } else {
      const char* b = sbase + k0 * ld;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int kr = ((wave + NW * j) * 1024 + 16 * (int)(threadIdx.x & 63)) / PITCH;
        const char* p = k0 + kr < K ? b + voff[j] : reinterpret_cast<const char*>(&g_zero_16);
        dma16(p, stage + (wave + NW * j) * 1024);
      }
    }
  }
  __device__ __forceinline__ uint4 frag(const char* stage, int f, int ks) const {
    const char* a = stage + foff[f] + ks * 16 * PITCH;
    return tr_pair(a, a + 4 * PITCH);
  }
};

// acc += the products of K-tiles kt0 .. kt1-1 (kt1 > kt0). smem: two stages. The MFMA operands
// are swapped (transposed blocks): a lane then holds 16 columns of one row.
template <class Tl, class OA, class OB>
__device__ __forceinline__ void dense_loop(const OA& oa, const OB& ob, int64_t kt0, int64_t kt1, char* smem, int wave,
                                           f32x16_t (&acc)[Tl::FM][Tl::FN]) {
  constexpr int SB = OA::BYTES + OB::BYTES;
  zero_acc<Tl>(acc);
  oa.issue(kt0, smem, wave);
  ob.issue(kt0, smem + OA::BYTES, wave);
  if (kt0 + 1 < kt1) {
    oa.issue(kt0 + 1, smem + SB, wave);
    ob.issue(kt0 + 1, smem + SB + OA::BYTES, wave);
    wait_vmcnt<OA::NI + OB::NI>();
  } else {
    wait_vmcnt<0>();
  }
  ring_barrier();
  uint4 a[2][Tl::FM], b[2][Tl::FN];
#pragma unroll
  for (int fm = 0; fm < Tl::FM; ++fm) a[0][fm] = oa.frag(smem, fm, 0);
#pragma unroll
  for (int fn = 0; fn < Tl::FN; ++fn) b[0][fn] = ob.frag(smem + OA::BYTES, fn, 0);
  int cur = 0;
  for (int64_t kt = kt0; kt < kt1; ++kt) {
    char* st = smem + cur * SB;
    char* nx = smem + (cur ^ 1) * SB;
    static_for<0, 4>([&](auto kc) {
      constexpr int ks = decltype(kc)::value, c = ks & 1;
      if constexpr (ks < 3) {
#pragma unroll
        for (int fm = 0; fm < Tl::FM; ++fm) a[c ^ 1][fm] = oa.frag(st, fm, ks + 1);
#pragma unroll
        for (int fn = 0; fn < Tl::FN; ++fn) b[c ^ 1][fn] = ob.frag(st + OA::BYTES, fn, ks + 1);
      } else if (kt + 1 < kt1) {
        // every fragment of this stage is in registers and this wave's loads of the next stage
        // have landed: after the barrier both hold for the whole workgroup
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kt + 2 < kt1) {
          oa.issue(kt + 2, st, wave);
          ob.issue(kt + 2, st + OA::BYTES, wave);
        }
#pragma unroll
        for (int fm = 0; fm < Tl::FM; ++fm) a[c ^ 1][fm] = oa.frag(nx, fm, 0);
#pragma unroll
        for (int fn = 0; fn < Tl::FN; ++fn) b[c ^ 1][fn] = ob.frag(nx + OA::BYTES, fn, 0);
      }
#pragma unroll
      for (int fm = 0; fm < Tl::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < Tl::FN; ++fn) Mma<bf16>::run(acc[fm][fn], b[c][fn], a[c][fm]);
    });
    cur ^= 1;
  }
  __syncthreads();
}

// Hands the transposed blocks of dense_loop back through a per-wave LDS patch, every lane owning
// eight consecutive columns of a row: f(row, col, g, u), row and col in the workgroup's tile; with
// SW, u are the same columns of the up block 32 to the right. The patch's row pitch keeps the
// 16-byte writes of the 32 rows on distinct banks; a wave's LDS operations run in order.
constexpr int kDensePatch = 68;  // floats

template <class Tl, bool SW, class F>
__device__ __forceinline__ void dense_epilogue(f32x16_t (&acc)[Tl::FM][Tl::FN], char* smem, int wave, int wm, int wn,
                                               int lane, F&& f) {
  static_assert(Tl::FN % 2 == 0, "blocks are handed back in horizontal pairs");
  float* patch = reinterpret_cast<float*>(smem) + wave * (32 * kDensePatch);
  const int m = lane & 31, h = lane >> 5;
  constexpr int LPR = SW ? 4 : 8;  // lanes of a row
  const int r0 = lane / LPR, c0 = (lane % LPR) * 8;
#pragma unroll
  for (int fm = 0; fm < Tl::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < Tl::FN; fn += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(patch + m * kDensePatch + 32 * b + 8 * g + 4 * h) =
              make_float4(acc[fm][fn + b][4 * g], acc[fm][fn + b][4 * g + 1], acc[fm][fn + b][4 * g + 2],
                          acc[fm][fn + b][4 * g + 3]);
#pragma unroll
      for (int i = 0; i < LPR / 2; ++i) {
        const int row = r0 + (64 / LPR) * i;
        const float* p = patch + row * kDensePatch + c0;
        float g8[8], u8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          g8[q] = p[q];
          u8[q] = SW ? p[32 + q] : 0.0f;
        }
        f(wm * Tl::WTM + fm * 32 + row, wn * Tl::WTN + fn * 32 + c0, g8, u8);
      }
    }
}

}  // namespace mok
