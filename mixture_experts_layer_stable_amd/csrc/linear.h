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
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (std::is_same<T, bf16>::value) {
    stg16(p, pack(v, (bf16*)nullptr));
  } else {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) { a[i] = v[i]; b[i] = v[4 + i]; }
    stg16(p, pack(a, (float*)nullptr));
    stg16(p + 4, pack(b, (float*)nullptr));
  }
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.0f / (1.0f + expf(-z)); }
__device__ __forceinline__ float phi_f(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

// Columns c .. c+7 (c a multiple of 8, in range) of row m: g = the products, u = those of the
// up columns (SWIGLU only). T: type of add, out; TP: of pre.
template <int KIND, int EPI, typename T, typename TP>
__device__ __forceinline__ void linear_store8(const LinearArgs& a, int64_t m, int c, float (&g)[8], float (&u)[8]) {
  if constexpr (KIND == LIN_FWD) {
    const int P = EPI == MOK_EPI_SWIGLU ? 2 * a.N : a.N;
    if (a.bias != nullptr) {
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
    if (a.pre != nullptr) {
      TP* p = (TP*)a.pre + m * P + c;
      store8(p, g);
      if constexpr (EPI == MOK_EPI_SWIGLU) store8(p + a.N, u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (EPI == MOK_EPI_SILU) g[i] *= sigmoid_f(g[i]);
      if constexpr (EPI == MOK_EPI_GELU) g[i] *= phi_f(g[i]);
      if constexpr (EPI == MOK_EPI_SWIGLU) g[i] *= sigmoid_f(g[i]) * u[i];
    }
  }
  const int64_t o = m * a.N + c;
  if (a.add != nullptr) {
    float r[8];
    load8((const T*)a.add + o, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += r[i];
  }
  store8((T*)a.out + o, g);
}

}  // namespace mok
