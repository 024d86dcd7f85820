// Products with 4-bit weights for a few rows of x a group (decoded tokens).
//
//   p[m][n] = sum over groups j of K of s[n][j] (sum_k x[m][k] (16 + q[n][k]) - (16 + z[n][j]) sum_k x[m][k])
//
// What bounds them is the codes' way from HBM and its latency, so a workgroup takes 16 rows of w (8 gate
// and 8 up rows for SWIGLU) over all of K, as linear_few.hip, and its eight waves take 128 codes of K
// of each row in turn. A code becomes a matrix operand without arithmetic: 16 + q in bf16 is
// 0x4180 | q << 3, two of a dword at a time; the products are exact in fp32, a multiplication by ones
// gives the sums of x that the offset brought in, in the lanes that hold the results, and a group's
// result takes its scale in fp32. So w is never rounded to bf16. fp32 x: codes as fp32 numbers q - z.
#include "linear_few.h"
#include "q4.h"

namespace mok {

namespace {

constexpr int kPiece = 128;  // codes of a row that a wave takes at a time

// Lanes l, l + 16, l + 32, l + 48 hold four units each: unit d of lane group g <-> unit g of lane group d.
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
template <int W>
__device__ __forceinline__ void group_transpose(uint32_t (&u)[4][W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    swap32(u[0][i], u[2][i]);
    swap32(u[1][i], u[3][i]);
    swap16(u[0][i], u[1][i]);
    swap16(u[2][i], u[3][i]);
  }
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

// RT: tiles of 16 rows of x; G: codes that share a scale
template <typename T, int EPI, int RT, int G>
__global__ __launch_bounds__(64 * kFewWaves) void q4_few_kernel(Q4Args qa) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU, BF = std::is_same<T, bf16>::value;
  constexpr int BM = 16 * RT, XV = sizeof(T) / 2;  // 16-byte vectors of eight values of x
  constexpr int GP = kPiece / G;                   // scales of a piece
  constexpr int NB = RT == 1 && BF ? 4 : 2;        // pieces that a wave loads at a time
  __shared__ __align__(16) float s_sum[kFewWaves][BM][kFewLd];
  LinearArgs a = qa.l;
  const int NT = SW ? a.N / 8 : (a.N + 15) / 16;
  int L;
  GroupTile t;
  if (!q4_tile(qa, BM, NT, L, t)) return;
  const int i0 = L - t.first * NT, mt = i0 % t.tiles, nt = i0 / t.tiles;
  const int64_t r0 = t.lo + (int64_t)mt * BM, P = SW ? 2 * (int64_t)a.N : a.N;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = nt * (SW ? 8 : 16), K = (int)a.K, M = (int)min<int64_t>(BM, t.hi - r0), KG = K / G;
  // row of w of this lane (rows past N re-read the last one)
  const int64_t wr = t.g * P + (SW ? (r < 8 ? n0 + r : (int64_t)a.N + n0 + r - 8) : min(n0 + r, a.N - 1));
  const uint8_t* wq = (const uint8_t*)a.b + wr * (K / 2);
  const T* ws = (const T*)qa.s + wr * KG;
  const uint8_t* wz = qa.z != nullptr ? qa.z + wr * KG : nullptr;
  // x: register j of a lane is of row 4 (r / 4) + j until quad_transpose, as in linear_few.hip
  const T* x[RT][4];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = 16 * q + (r & 12) + j;
      x[q][j] = m < M ? (const T*)a.a + (r0 + m) * K : nullptr;
    }

  struct Batch {
    uint4 w[NB];
    uint4 x[NB][RT][XV][4];
    float s[GP], z[GP];  // of piece (lane group) of the batch
  };
  const int pieces = (K + kPiece - 1) / kPiece, rounds = (pieces + kFewWaves - 1) / kFewWaves;
  const int first = (int)((nt >> 3 & 31) * (unsigned)pieces >> 5);  // workgroups start all over K
  // first code of piece `i` of this wave, or K for none
  const auto at = [&](int i) {
    int q = i * kFewWaves + wave;
    if (q >= pieces) return K;
    q += first;
    return (q >= pieces ? q - pieces : q) * kPiece;
  };
  const auto load = [&](int i, Batch& b) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int k = at(i + n) + 32 * g;
      b.w[n] = k < K ? ldg16(wq + k / 2) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < RT; ++q)
#pragma unroll
        for (int h = 0; h < XV; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = k + (BF ? 8 * (r & 3) : 16 * h + 4 * (r & 3));
            b.x[n][q][h][j] = k < K && x[q][j] != nullptr ? ldg16(x[q][j] + e) : make_uint4(0, 0, 0, 0);
          }
    }
    const int k = g < NB ? at(i + g) : K;
#pragma unroll
    for (int p = 0; p < GP; ++p) {
      const bool in = k + p * G < K;
      b.s[p] = in ? Elem<T>::get(ws, k / G + p) : 0.0f;
      b.z[p] = in && wz != nullptr ? (float)wz[k / G + p] : 8.0f;
    }
  };
  f32x4_t acc[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) acc[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const auto mma = [&](Batch& b) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      uint32_t w[4][1] = {{b.w[n].x}, {b.w[n].y}, {b.w[n].z}, {b.w[n].w}};
      if constexpr (GP > 1) group_transpose(w);
      float sc[GP], zp[GP];
#pragma unroll
      for (int p = 0; p < GP; ++p) {
        sc[p] = __shfl(b.s[p], r + 16 * n);
        zp[p] = __shfl(b.z[p], r + 16 * n);
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        uint32_t u[4][4 * XV];
#pragma unroll
        for (int h = 0; h < XV; ++h) {
          quad_transpose(b.x[n][q][h]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // bf16: vector j is unit j; fp32: vectors 2 (j % 2) .. of half h are unit 2 h + j / 2
            const uint4& v = b.x[n][q][h][j];
            const int d = BF ? j : 2 * h + j / 2, o = BF ? 0 : 4 * (j % 2);
            u[d][o] = v.x;
            u[d][o + 1] = v.y;
            u[d][o + 2] = v.z;
            u[d][o + 3] = v.w;
          }
        }
        if constexpr (GP > 1) group_transpose(u);
#pragma unroll
        for (int p = 0; p < GP; ++p) {
          f32x4_t d = zero, o = zero;
#pragma unroll
          for (int e = p * (4 / GP); e < (p + 1) * (4 / GP); ++e) {
            if constexpr (BF) {
              const uint4 xv = order_bf16(make_uint4(u[e][0], u[e][1], u[e][2], u[e][3]));
              const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
              d = mma16<bf16>(xv, codes_bf16(w[e][0]), d);
              o = mma16<bf16>(xv, one, o);
            } else {
              const uint32_t lo = w[e][0] & 0x0F0F0F0Fu, hi = w[e][0] >> 4 & 0x0F0F0F0Fu;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float wv = (float)((c & 1 ? hi : lo) >> (8 * (c / 2)) & 0xFFu) - zp[p];
                d = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(u[e][c % (4 * XV)]), wv, d, 0, 0, 0);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[q][i] = __builtin_fmaf(sc[p], BF ? __builtin_fmaf(-16.0f - zp[p], o[i], d[i]) : d[i], acc[q][i]);
        }
      }
    }
  };
  Batch b0, b1;
  load(0, b0);
  // what this lane stores in the end: eight outputs of a row, and what is added to them
  const int row = SW ? tid : tid >> 1, c = n0 + (SW ? 0 : 8 * (tid & 1));
  const bool out = row < M && c < a.N;
  Raw8<T> add{};
  float bg[8], bu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bg[i] = bu[i] = 0.0f;
  if (a.bias != nullptr) a.bias += t.g * P;
  if (out) {
    add = linear_add8<T>(a, r0 + row, c);
    linear_bias8<EPI>(a, c, bg, bu);
  }
  for (int i = 0; i < rounds; i += 2 * NB) {
    if (i + NB < rounds) load(i + NB, b1);
    mma(b0);
    if (i + NB >= rounds) break;
    if (i + 2 * NB < rounds) load(i + 2 * NB, b0);
    mma(b1);
  }
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[wave][16 * q + 4 * g + i][r] = acc[q][i];
  __syncthreads();
  if (tid < 256 * RT) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kFewWaves; ++i) v += s_sum[i][tid >> 4][tid & 15];
    s_sum[0][tid >> 4][tid & 15] = v;
  }
  __syncthreads();
  if (!out) return;
  float p[8], u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = s_sum[0][row][(SW ? 0 : c - n0) + i] + bg[i];
    u[i] = SW ? s_sum[0][row][8 + i] + bu[i] : 0.0f;
  }
  linear_store8<LIN_FWD, EPI, T, T>(a, r0 + row, c, p, u, add);
}

template <typename T, int EPI, int RT>
void run_few(const Q4Args& a, hipStream_t s) {
  const int cols = EPI == MOK_EPI_SWIGLU ? 8 : 16;
  const dim3 grid((unsigned)(q4_tiles_bound(a, 16 * RT) * ((a.l.N + cols - 1) / cols))), block(64 * kFewWaves);
  if (a.group == 32) hipLaunchKernelGGL((q4_few_kernel<T, EPI, RT, 32>), grid, block, 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((q4_few_kernel<T, EPI, RT, 64>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((q4_few_kernel<T, EPI, RT, 128>), grid, block, 0, s, a);
}

template <typename T, int RT>
void run_few(const Q4Args& a, int epi, hipStream_t s) {
  if (epi == MOK_EPI_NONE) run_few<T, MOK_EPI_NONE, RT>(a, s);
  else if (epi == MOK_EPI_SILU) run_few<T, MOK_EPI_SILU, RT>(a, s);
  else if (epi == MOK_EPI_GELU) run_few<T, MOK_EPI_GELU, RT>(a, s);
  else run_few<T, MOK_EPI_SWIGLU, RT>(a, s);
}

}  // namespace

hipError_t launch_q4_few(const Q4Args& a, int rt, int act, int epi, hipStream_t s) {
  if (act == MOK_F32) {
    if (rt == 1) run_few<float, 1>(a, epi, s);
    else run_few<float, 2>(a, epi, s);
  } else {
    if (rt == 1) run_few<bf16, 1>(a, epi, s);
    else run_few<bf16, 2>(a, epi, s);
  }
  return hipGetLastError();
}

}  // namespace mok
