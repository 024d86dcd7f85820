// Epilogue of the matrix products (linear.hip): what happens to eight consecutive fp32 results
// of a row before they are rounded and stored.
#pragma once
#include "block.h"
#include "gemm.h"

namespace mok {

// Eight consecutive elements of a row as floats / stored from floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (std::is_same<T, bf16>::value) {
    unpack(ldg16(p), v, (bf16*)nullptr);
  } else {
    float a[4], b[4];
    unpack(ldg16(p), a, (float*)nullptr);
    unpack(ldg16(p + 4), b, (float*)nullptr);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  }
}
// NT: a non-temporal store, for outputs that no cache would keep anyway.
template <bool NT>
__device__ __forceinline__ void put16(void* p, const uint4& v) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (NT) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
  else stg16(p, v);
}
template <bool NT = false, typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (std::is_same<T, bf16>::value) {
    put16<NT>(p, pack(v, (bf16*)nullptr));
  } else {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) { a[i] = v[i]; b[i] = v[4 + i]; }
    put16<NT>(p, pack(a, (float*)nullptr));
    put16<NT>(p + 4, pack(b, (float*)nullptr));
  }
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.0f / (1.0f + expf(-z)); }
// The same to 2^-20 by the hardware's exp2 and reciprocal, for results that are rounded to bf16:
// a wave that has its SIMD to itself waits for every instruction of an epilogue (16384 x (2 x 2048)
// x 7168 SWIGLU: 10 us less).
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
template <typename T>
__device__ __forceinline__ float sigmoid_t(float z) {
  return std::is_same<T, bf16>::value ? sigmoid_fast(z) : sigmoid_f(z);
}
__device__ __forceinline__ float phi_f(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

// What is added to columns c .. c+7 of row m, as it lies in memory (zeros without an addend).
template <typename T>
struct Raw8 {
  uint4 v[std::is_same<T, bf16>::value ? 1 : 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> linear_add8(const LinearArgs& a, int64_t m, int c) {
  Raw8<T> r;
#pragma unroll
  for (auto& v : r.v) v = make_uint4(0, 0, 0, 0);
  if (a.add != nullptr) {
    const T* p = (const T*)a.add + m * a.N + c;
    r.v[0] = ldg16(p);
    if constexpr (!std::is_same<T, bf16>::value) r.v[1] = ldg16(p + 4);
  }
  return r;
}

// Columns c .. c+7 (c a multiple of 8, in range) of row m: g = the products and bias, u = those of
// the up columns (SWIGLU only), add = linear_add8's. T: type of add, out; TP: of pre. NT:
// non-temporal stores.
template <int KIND, int EPI, typename T, typename TP, bool NT = false>
__device__ __forceinline__ void linear_store8(const LinearArgs& a, int64_t m, int c, float (&g)[8], float (&u)[8],
                                              const Raw8<T>& add) {
  if constexpr (KIND == LIN_FWD) {
    const int P = EPI == MOK_EPI_SWIGLU ? 2 * a.N : a.N;
    if (a.pre != nullptr) {
      TP* p = (TP*)a.pre + m * P + c;
      store8<NT>(p, g);
      if constexpr (EPI == MOK_EPI_SWIGLU) store8<NT>(p + a.N, u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (EPI == MOK_EPI_SILU || EPI == MOK_EPI_SWIGLU) g[i] *= sigmoid_t<T>(g[i]);
      if constexpr (EPI == MOK_EPI_SWIGLU) g[i] *= u[i];
      if constexpr (EPI == MOK_EPI_GELU) g[i] *= phi_f(g[i]);
    }
  }
  if (a.add != nullptr) {
    float r[8];
    load8(reinterpret_cast<const T*>(&add.v[0]), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += r[i];
  }
  store8<NT>((T*)a.out + m * a.N + c, g);
}

// g += bias of columns c .. c+7 (u: of the up columns)
template <int EPI>
__device__ __forceinline__ void linear_bias8(const LinearArgs& a, int c, float (&g)[8], float (&u)[8]) {
  if (a.bias == nullptr) return;
  float b[8];
  load8(a.bias + c, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] += b[i];
  if constexpr (EPI == MOK_EPI_SWIGLU) {
    load8(a.bias + a.N + c, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] += b[i];
  }
}

// d = dy of eight columns, p = pre of them (u: of the up columns) -> d = dp (u: of the up columns).
template <typename T, int EPI>
__device__ __forceinline__ void linear_dpre8(float (&d)[8], const float (&p)[8], float (&u)[8]) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (EPI == MOK_EPI_SILU || SW) {
      const float s = sigmoid_t<T>(p[i]), f = s * (1.0f + p[i] * (1.0f - s));
      if constexpr (SW) {
        const float up = d[i] * p[i] * s;
        d[i] *= u[i] * f;
        u[i] = up;
      } else {
        d[i] *= f;
      }
    } else if constexpr (EPI == MOK_EPI_GELU) {
      d[i] *= phi_f(p[i]) + p[i] * 0.39894228040143268f * expf(-0.5f * p[i] * p[i]);
    }
  }
}

// out = f(sum of the slices' partial products + bias) + add. A wave takes 64 / SL groups of eight
// columns; SL lanes a group read every SL-th slice each and add their sums in a tree, so that few rows
// do not wait for one slice after the other (5 x 4096 of 16 slices: 9.7 us with a lane for all of
// them, 5.3 with 8). T: type of the operands.
template <int KIND, int EPI, typename TO, typename T, int SL>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a) {
  constexpr bool SW = EPI == MOK_EPI_SWIGLU;
  constexpr int CG = 64 / SL;
  const int lane = threadIdx.x & 63, sl = lane / CG;
  const int64_t nv = a.N / 8, i = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * CG + lane % CG;
  const bool in = i < a.M * nv;
  const int64_t m = in ? i / nv : 0, P = SW ? 2 * a.N : a.N;
  const int c = in ? (int)(i - m * nv) * 8 : 0;
  Raw8<TO> add{};
  if (sl == 0) add = linear_add8<TO>(a, m, c);
  float g[8], u[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) g[q] = u[q] = 0.0f;
#pragma unroll 4
  for (int s = sl; s < a.split; s += SL) {
    const float* p = a.part + ((int64_t)s * a.M + m) * P + c;
    float v[8];
    load8(p, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) g[q] += v[q];
    if constexpr (SW) {
      load8(p + a.N, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) u[q] += v[q];
    }
  }
#pragma unroll
  for (int o = CG; o < 64; o <<= 1)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] += __shfl_xor(g[q], o);
      if constexpr (SW) u[q] += __shfl_xor(u[q], o);
    }
  if (!in || sl != 0) return;
  if constexpr (KIND == LIN_FWD) linear_bias8<EPI>(a, c, g, u);
  linear_store8<KIND, EPI, TO, T>(a, m, c, g, u, add);
}

template <int KIND, int EPI, typename TO, typename T>
inline void linear_join(const LinearArgs& a, hipStream_t s) {
  const int64_t groups = a.M * (a.N / 8);
  const auto grid = [&](int sl) { return dim3((unsigned)((groups * sl + 255) / 256)); };
  if (a.split >= 8) hipLaunchKernelGGL((linear_join_kernel<KIND, EPI, TO, T, 8>), grid(8), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear_join_kernel<KIND, EPI, TO, T, 2>), grid(2), dim3(256), 0, s, a);
}

}  // namespace mok
