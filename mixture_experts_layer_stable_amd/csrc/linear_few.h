// The few-row product of linear_few.hip: one workgroup's part, for the dense and the grouped kernels.
//
// What bounds them is w's way from HBM, and what they wait for is latency: a workgroup takes 16 rows
// of w (8 gate and 8 up rows for SWIGLU) over all of K, so that no second launch has to join slices of
// K. Its eight waves take 256-byte pieces of K in turn, each loads its fragments straight into
// registers, the next piece's ahead of the MFMAs, and the waves' sums are added in LDS in wave order.
#pragma once
#include "linear.h"

namespace mok {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
constexpr int kFewWaves = 8;
constexpr int kFewLd = 20;  // floats of a row of sums

// The quad's 4 x 4 matrix (register, lane) of 16-byte elements, transposed.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
  const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
  const auto swap = [](uint32_t& x, uint32_t& y, bool odd, auto ctrl) {
    constexpr int C = decltype(ctrl)::value;
    const uint32_t dx = __builtin_amdgcn_mov_dpp(x, C, 0xf, 0xf, true), dy = __builtin_amdgcn_mov_dpp(y, C, 0xf, 0xf, true);
    x = odd ? dy : x;
    y = odd ? y : dx;
  };
  const auto swap4 = [&](uint4& x, uint4& y, bool odd, auto ctrl) {
    swap(x.x, y.x, odd, ctrl);
    swap(x.y, y.y, odd, ctrl);
    swap(x.z, y.z, odd, ctrl);
    swap(x.w, y.w, odd, ctrl);
  };
  const std::integral_constant<int, 0xb1> by1;  // lanes 1 0 3 2
  const std::integral_constant<int, 0x4e> by2;  // lanes 2 3 0 1
  swap4(v[0], v[1], b0, by1);
  swap4(v[2], v[3], b0, by1);
  swap4(v[0], v[2], b1, by2);
  swap4(v[1], v[3], b1, by2);
}

// acc += A B^T of 16 rows each: lane l holds 16 bytes of K of row l % 16, group l / 16. Which k they
// are does not matter as long as both operands agree.
template <typename T>
__device__ __forceinline__ f32x4_t mma16(const uint4& a, const uint4& b, f32x4_t acc) {
  if constexpr (std::is_same<T, bf16>::value) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc,
                                                   0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), acc, 0, 0, 0);
  }
}

// The workgroup's 16 rows of w (8 and 8 for SWIGLU), the nt-th, and all rows of x. RT: tiles of 16 of those.
template <typename T, int EPI, int RT>
__device__ __forceinline__ void few_work(const LinearArgs& a, int nt, float (&s_sum)[kFewWaves][RT * 16][kFewLd]) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  constexpr int VE = Elem<T>::VE, PIECE = 16 * VE;  // elements of 16 and of 256 bytes
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = nt * (SW ? 8 : 16), K = (int)a.K, M = (int)a.M;
  // Four lanes load 64 consecutive bytes of a row, as the address unit takes them together: register j
  // of a lane is of row 4 (r / 4) + j, bytes 64 g + 16 (r % 4) of the piece, until quad_transpose
  // makes it the lane's own row r, bytes 64 g + 16 j (a lane a row: 66 cycles a load; 16 x (2 x 2048)
  // x 7168 19.2 us). Columns past N re-read the last one, rows past M are zeros.
  const T *w[4], *x[RT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int q = (r & 12) + j;
    w[j] = (const T*)a.b + (SW ? (q < 8 ? n0 + q : (int64_t)a.N + n0 + q - 8) : min(n0 + q, a.N - 1)) * K;
#pragma unroll
    for (int t = 0; t < RT; ++t) x[t][j] = 16 * t + q < M ? (const T*)a.a + (int64_t)(16 * t + q) * K : nullptr;
  }

  uint4 wf[2][4], xf[2][RT][4];
  const int pieces = (K + PIECE - 1) / PIECE, rounds = (pieces + kFewWaves - 1) / kFewWaves;
  // The workgroups of an XCD start all over K: rows of a pitch of many KB meet in one memory channel
  // (1 x 4096 x 4096 fp32: 19.0 us, 15.3).
  const int first = (int)((nt >> 3 & 31) * (unsigned)pieces >> 5);
  const auto load = [&](int round, uint4 (&wv)[4], uint4 (&xv)[RT][4]) {
    int q = round * kFewWaves + wave;
    const bool live = q < pieces;
    q += first;
    q -= q >= pieces ? pieces : 0;
    const int k = q * PIECE + (4 * g + (r & 3)) * VE;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wv[j] = live && k < K ? ldg16(w[j] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < RT; ++t) xv[t][j] = live && k < K && x[t][j] != nullptr ? ldg16(x[t][j] + k) : make_uint4(0, 0, 0, 0);
    }
  };
  f32x4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const auto mma = [&](uint4 (&wv)[4], uint4 (&xv)[RT][4]) {
    quad_transpose(wv);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      quad_transpose(xv[t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t] = mma16<T>(xv[t][j], wv[j], acc[t]);
    }
  };
  load(0, wf[0], xf[0]);
  // what this lane stores in the end: eight outputs of a row, and what is added to them
  const int row = SW ? tid : tid >> 1, c = n0 + (SW ? 0 : 8 * (tid & 1));
  const bool out = row < M && c < a.N;
  Raw8<T> add{};
  float bg[8], bu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bg[i] = bu[i] = 0.0f;
  if (out) {
    add = linear_add8<T>(a, row, c);
    linear_bias8<EPI>(a, c, bg, bu);
  }
  for (int i = 0; i < rounds; i += 2) {
    if (i + 1 < rounds) load(i + 1, wf[1], xf[1]);
    mma(wf[0], xf[0]);
    if (i + 1 >= rounds) break;
    if (i + 2 < rounds) load(i + 2, wf[0], xf[0]);
    mma(wf[1], xf[1]);
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[wave][16 * t + 4 * g + i][r] = acc[t][i];
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
  linear_store8<LIN_FWD, EPI, T, T>(a, row, c, p, u, add);
}

}  // namespace mok
