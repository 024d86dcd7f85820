// Products with 4-bit weights for many rows of x a group (prompts).
//
// A workgroup multiplies 128 rows of x by 128 rows of w, two workgroups a CU. x and the codes with their
// scales and zero points come into LDS by direct loads; while the matrix units work on one K-tile (128 bytes
// of a row of x) the codes of the next are written into LDS as matrix operands. bf16: the operand is q - z,
// exact in bf16, and the sums of each K-tile (of each group of 32, where a scale ends inside it) take their
// scale in fp32, so w is never rounded. fp32: the operand is s (q - z), rounded once.
// What bounds it is vector instructions beside the MFMAs: the codes' conversion, which every row tile
// does again, and the sums' scaling: the MFMAs are busy a third of the time. 4096 rows, 2 x 2048 x 7168: 322 to 342 us
// over several cards (703 to 747 TFLOP/s); 7168 x 2048: 169 to 178, in groups of 32 189 to 193 (twice the scalings; with last
// K-tiles that branched around their loads, and spilled, 192 and 307 where these took 169 and 189). The sums are as many
// registers again as the accumulators: 256 x 128 tiles spill (387 for 333 on that card), 128 x 128 with one workgroup a CU
// take 0.79 us a K-tile where two take 1.45 for both. fp32, 4096 rows, 2048 x 2048: 311 to 313 us (110 TFLOP/s).
// Few tiles of a dense product take slices of K, joined by linear_join (128 rows, 2 x 2048 x 7168: 101 -> 36 us).
#include "linear_dense.h"
#include "q4.h"

namespace mok {

namespace {

// 4 bytes a lane into LDS at lds + 4 lane (see load_lds_sv for the distances).
__device__ __forceinline__ void dma4_any(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}

template <typename T, class Tl>
struct Q4Tile {
  using OA = DenseK<T, Tl::BM, Tl::FM, Tl::NW>;
  static constexpr int BN = 128;
  static constexpr bool BF = std::is_same<T, bf16>::value;
  static constexpr int kA = BF ? 2 : 3, kRaw = BF ? 2 : 4;  // stages
  static constexpr int RAW = 4096 + 1024 + 1024;          // codes, scales, zero points of a K-tile
  static constexpr int B0 = kA * OA::BYTES, R0 = B0 + 2 * BN * 128, LDS = R0 + kRaw * RAW;
  static constexpr int NL = OA::NI + 3;                   // loads of a wave and K-tile
  static_assert(Tl::BN == BN && Tl::NT == 256 && Tl::FN == 2, "tile");
};

template <typename T, class Tl, bool SW, int G>
__global__ __launch_bounds__(Tl::NT, sizeof(T) == 2 ? 2 : 1) void q4_tile_kernel(Q4Args qa) {
  using C = Q4Tile<T, Tl>;
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
  int mt, nt, slice = 0;
  if (qa.off == nullptr) {
    const int MT = (int)((a.M + Tl::BM - 1) / Tl::BM), L = xcd_logical(blockIdx.x, gridDim.x);
    t = {0, 0, (int)a.M, 0, MT};
    slice = L / (MT * NT);
    band_walk(L - slice * MT * NT, MT, NT, mt, nt);
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
  // this slice of K: whole pieces of 128 from k0 on
  const uint32_t KF = (uint32_t)a.K, pieces = (KF + 127) / 128;
  const uint32_t k0 = (uint32_t)((uint64_t)pieces * slice / a.split) * 128;
  const uint32_t K = min(KF, (uint32_t)((uint64_t)pieces * (slice + 1) / a.split) * 128) - k0, KG = K / G;
  // first output column of tile column j, and its row of w (columns past N re-read the last one)
  const auto col = [&](int j) { return SW ? n0 + (j / 64) * 32 + (j & 31) : n0 + j; };
  const auto wrow = [&](int j) { return t.g * P + min(col(j), a.N - 1) + (SW && (j & 32) ? a.N : 0); };

  const auto frow_a = [&](int f) { return wm * Tl::WTM + f * 32; };
  typename C::OA oa;
  oa.init((const T*)a.a + m0 * KF + k0, 0, K, [&](int row) { return (uint32_t)min(row, rows - 1) * (uint32_t)(ES * KF); },
          frow_a, wave, lane);
  // Raw loads of this lane: 16 bytes of codes of row tid / 2 (bf16: half tid % 2 of its K-tile; fp32: a row is 16
  // bytes, rows tid % 128); scale and zero point of row tid / 2 (group tid % 2 of the K-tile, if it has two).
  const uint8_t* wq = (const uint8_t*)a.b + wrow(BF ? tid >> 1 : tid & 127) * (KF / 2) + k0 / 2;
  const uint64_t sg = (uint64_t)wrow(tid >> 1) * (KF / G) + k0 / G;
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

  f32x16_t acc[Tl::FM][2];
  zero_acc<Tl>(acc);
  const uint32_t KT = (K + BK - 1) / BK;
  if constexpr (!BF) {
    // Loads of K-tile kt: x two K-tiles ahead, codes three (past the end: again the last ones, which no one reads).
    const auto issue = [&](uint32_t kt_a, uint32_t kt_raw) {
      oa.template issue<false>(min(kt_a, KT - 1), lds + kt_a % C::kA * C::OA::BYTES, wave);
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
      const char* sa = smem + kt % C::kA * C::OA::BYTES;
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
          for (int f = 0; f < 2; ++f) Mma<T>::run(acc[m][f], fa[m], fb[f]);
      }
    }
  } else {
    // Two waves a SIMD, of two workgroups: everything has its place between two matrix instructions, as in dense_tile. At a
    // K-tile's last step the wave holds its fragments of it: it waits for its loads of the next and for
    // the workgroup, reads the next one's first fragments and loads x two, codes three K-tiles ahead. In
    // the other steps the next K-tile's codes become operands. A group's sums go to acc where the next
    // group's first products would overwrite them.
    constexpr int NM = Tl::FM * 2, NR = Tl::FM + 2;
    static_assert(NM == 4, "slots 1 to 8 lie before the step that reads the operands");
    f32x16_t grp[Tl::FM][2];
    zero_acc<Tl>(grp);
    uint4 fa[2][Tl::FM], fb[2][2];
    uint32_t sr[2][2] = {{0, 0}, {0, 0}};  // [half of the K-tile][f]: scales as loaded, of the group that ends there
    uint32_t sh[2] = {0, 0};               // [f]: low bits of the index of column f's first scale
#pragma unroll
    for (int f = 0; f < 2; ++f) sh[f] = (uint32_t)wrow(wn * Tl::WTN + f * 32 + (lane & 31)) * (KF / G) + k0 / G;
    float s[2] = {0.0f, 0.0f};  // of the group that ended last
    const auto read_scales = [&](const char* raw, uint32_t (&to)[2][2]) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const char* p = raw + 4096 + 8 * (wn * Tl::WTN + f * 32 + (lane & 31));
        to[0][f] = *reinterpret_cast<const uint32_t*>(p);
        if constexpr (G == 32) to[1][f] = *reinterpret_cast<const uint32_t*>(p + 4);
      }
    };
    const auto flush = [&](auto ic) {
      constexpr int i = decltype(ic)::value, m = i / 2, f = i % 2;
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][f][r] = __builtin_fmaf(s[f], grp[m][f][r], acc[m][f][r]);
    };
    const auto scale = [&](uint32_t kt, int half) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint32_t ix = sh[f] + kt * BK / G + half;
        s[f] = __uint_as_float(sr[half][f] >> ((ix & 1) * 16) << 16);
      }
    };
    // The step's loads have no branch, around which the sums would be spilled: past the end they take the last K-tile
    // again, and the second half of half a K-tile (G = 32) is the first one once more, which no one reads.
    const auto upper = [&](int j) { return ((lane & 7) ^ swz_k(8 * (wave + Tl::NW * j) + (lane >> 3))) >> 2 & 1; };
    static_assert(Tl::NW == 4, "upper(j) goes by j % 2");
    const uint32_t odd = G == 32 && KT * BK != K ? 64 : 0, hs[2] = {odd * upper(0), odd * upper(1)};
    const auto step = [&](uint32_t kt) {
      const uint32_t nk = kt + 1;
      const char* raw = smem + C::R0 + nk % C::kRaw * C::RAW;
      char* to = smem + C::B0 + (nk & 1) * (C::BN * 128) + brow * 128;
      uint4 w;
      uint32_t zr = 0;
      float z = 0.0f;
      uint32_t lo = 0, hi = 0;
      uint32_t op[4], srn[2][2];
      const uint32_t kd = kt + 2, dst = lds + kd % C::kA * C::OA::BYTES;
      static_for<0, 4>([&](auto kc) {
        constexpr int ks = decltype(kc)::value, c = ks & 1;
        constexpr bool first = G == 32 ? ks % 2 == 0 : ks == 0;  // of a group, or of half of one of 128
        if constexpr (ks == 3) {
          wait_vmcnt<0>();
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        const char* sa = smem + (ks == 3 ? nk : kt) % C::kA * C::OA::BYTES;
        const char* sb = smem + C::B0 + ((ks == 3 ? nk : kt) & 1) * (C::BN * 128);
        static_for<0, NM>([&](auto ic) {
          constexpr int i = decltype(ic)::value, m = i / 2, f = i % 2, slot = ks * NM + i;
          if constexpr (first) {
            flush(ic);
            const f32x16_t zero = {};
            grp[m][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa[c][m]),
                                                                __builtin_bit_cast(bf16x8_t, fb[c][f]), zero, 0, 0, 0);
          } else {
            Mma<T>::run(grp[m][f], fa[c][m], fb[c][f]);
          }
          if constexpr (i < NR) {
            if constexpr (i < 2) fb[c ^ 1][i] = *reinterpret_cast<const uint4*>(sb + foff[i][(ks + 1) & 3]);
            else fa[c ^ 1][i - 2] = oa.frag(sa, i - 2, (ks + 1) & 3);
          }
          // the next K-tile's operands: 32 codes in slots 1 to 8, four in each
          if constexpr (slot == 0) {
            w = *reinterpret_cast<const uint4*>(raw + 16 * tid);
            zr = *reinterpret_cast<const uint32_t*>(raw + 4096 + 1024 + 4 * tid);
          }
          constexpr int kFirst = 1, kPer = 2;  // first slot, pairs a slot
          if constexpr (slot == kFirst) {
            const uint32_t ix = sg_lo + min(nk * BK / G + (GP > 1 ? part : 0), KG - 1);
            z = qa.zeros ? (float)(zr >> ((ix & 3) * 8) & 0xFFu) : 8.0f;
          }
          if constexpr (slot >= kFirst && slot < kFirst + 16 / kPer) {
            static_for<0, kPer>([&](auto pc) {
              constexpr int pair = (slot - kFirst) * kPer + decltype(pc)::value, u = pair / 4, q = pair % 4;
              if constexpr (q == 0) {
                const uint32_t wd = u == 0 ? w.x : (u == 1 ? w.y : (u == 2 ? w.z : w.w));
                lo = wd & 0x0F0F0F0Fu;
                hi = wd >> 4 & 0x0F0F0F0Fu;
                asm("" : "+v"(lo), "+v"(hi));  // bytes: one conversion each
              }
              op[q] = bf16x2_rne((float)(lo >> (8 * q) & 0xFFu) - z, (float)(hi >> (8 * q) & 0xFFu) - z);
              if constexpr (q == 3)
                *reinterpret_cast<uint4*>(to + 16 * ((4 * part + u) ^ swz_k(brow))) = make_uint4(op[0], op[1], op[2], op[3]);
            });
          }
          // scales of the groups that end in the next K-tile; of the group that has just ended
          if constexpr (slot == NM) read_scales(raw, srn);
          if constexpr (i == NM - 1 && (ks == 3 || (G == 32 && ks == 1))) scale(kt, G == 32 && ks == 3);
          if constexpr (slot == 4 * NM - 1) {
#pragma unroll
            for (int h = 0; h < (G == 32 ? 2 : 1); ++h)
#pragma unroll
              for (int ff = 0; ff < 2; ++ff) sr[h][ff] = srn[h][ff];
          }
          if constexpr (ks == 3) {
            constexpr int NI = C::OA::NI;
            const uint32_t kl = min(kd, KT - 1), end = G == 32 && kl == KT - 1 ? ~0u : 0u;
            static_for<i * NI / NM, (i + 1) * NI / NM>([&](auto jc) {
              constexpr int j = decltype(jc)::value;
              load_lds_sv<16>(uniform_ptr(oa.base(kl, j, wave)), oa.voff[j] - (hs[j & 1] & end), dst + (wave + Tl::NW * j) * 1024);
            });
            if constexpr (i == NM - 1) issue_raw(kt + 3);
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    };
    issue_raw(0);
    issue_raw(1);
    oa.template issue<false>(0, lds, wave);
    wait_vmcnt<0>();
    ring_barrier();
    operand(0);
    read_scales(smem + C::R0, sr);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    oa.template issue<false>(min(1u, KT - 1), lds + C::OA::BYTES, wave);
    issue_raw(2);
#pragma unroll
    for (int m = 0; m < Tl::FM; ++m) fa[0][m] = oa.frag(smem, m, 0);
#pragma unroll
    for (int f = 0; f < 2; ++f) fb[0][f] = *reinterpret_cast<const uint4*>(smem + C::B0 + foff[f][0]);
    for (uint32_t kt = 0; kt < K / BK; ++kt) step(kt);
    static_for<0, NM>([&](auto ic) { flush(ic); });
    if (G == 32 && KT * BK != K) {  // half a K-tile: one group
      const char* sa = smem + (KT - 1) % C::kA * C::OA::BYTES;
      const char* sb = smem + C::B0 + ((KT - 1) & 1) * (C::BN * 128);
      zero_acc<Tl>(grp);
      static_for<0, NM>([&](auto ic) { Mma<T>::run(grp[ic / 2][ic % 2], fa[0][ic / 2], fb[0][ic % 2]); });
#pragma unroll
      for (int m = 0; m < Tl::FM; ++m) fa[1][m] = oa.frag(sa, m, 1);
#pragma unroll
      for (int f = 0; f < 2; ++f) fb[1][f] = *reinterpret_cast<const uint4*>(sb + foff[f][1]);
      static_for<0, NM>([&](auto ic) { Mma<T>::run(grp[ic / 2][ic % 2], fa[1][ic / 2], fb[1][ic % 2]); });
      scale(KT - 1, 0);
      static_for<0, NM>([&](auto ic) { flush(ic); });
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
#pragma unroll 1
    for (int i = 0; i < LPR / 2; ++i) {
      const int row = lane / LPR + (64 / LPR) * i, c = (lane % LPR) * 8;
      const int mm = wm * Tl::WTM + m * 32 + row, cc = col(wn * Tl::WTN + c);
      if (mm < rows && cc < a.N && a.part != nullptr) {
        float p[8];
        float* to = a.part + ((int64_t)slice * a.M + m0 + mm) * P + cc;
        load8(patch + row * kDensePatch + c, p);
        store8(to, p);
        if constexpr (SW) {
          load8(patch + row * kDensePatch + 32 + c, p);
          store8(to + a.N, p);
        }
      } else if (mm < rows && cc < a.N) {
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
  const dim3 grid((unsigned)(q4_tiles_bound(a, Tl::BM) * ((a.l.N + bno - 1) / bno) * a.l.split));
  if (a.group == 32) hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 32>), grid, dim3(Tl::NT), 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 64>), grid, dim3(Tl::NT), 0, s, a);
  else hipLaunchKernelGGL((q4_tile_kernel<T, Tl, SW, 128>), grid, dim3(Tl::NT), 0, s, a);
}

template <typename T, class Tl>
void run_tile(const Q4Args& a, hipStream_t s) {
  if (a.epi == MOK_EPI_SWIGLU) run_tile<T, Tl, true>(a, s);
  else run_tile<T, Tl, false>(a, s);
}

template <typename T>
void run_join(const Q4Args& a, hipStream_t s) {
  if (a.epi == MOK_EPI_SWIGLU) linear_join<LIN_FWD, MOK_EPI_SWIGLU, T, T>(a.l, s);
  else if (a.epi == MOK_EPI_SILU) linear_join<LIN_FWD, MOK_EPI_SILU, T, T>(a.l, s);
  else if (a.epi == MOK_EPI_GELU) linear_join<LIN_FWD, MOK_EPI_GELU, T, T>(a.l, s);
  else linear_join<LIN_FWD, MOK_EPI_NONE, T, T>(a.l, s);
}

}  // namespace

hipError_t launch_q4_tile(const Q4Args& a, int act, hipStream_t s) {
  if (act == MOK_F32) run_tile<float, Tiling<128, 128, 2, 2>>(a, s);
  else run_tile<bf16, Tiling<128, 128, 2, 2>>(a, s);
  if (a.l.split > 1) {
    if (act == MOK_F32) run_join<float>(a, s);
    else run_join<bf16>(a, s);
  }
  return hipGetLastError();
}

}  // namespace mok
