// Rows to the experts' order and back (dispatch, combine) and their gradients. HBM-bound: each row is
// read once by 16-byte vectors and written once. A slot or row whose index is outside its range
// (-1: dropped, padding) counts as none.
#include "permute.h"

namespace mok {

namespace {

// Rows of more than 16 MB an array are stored past the caches, which could not keep them for a reader.
constexpr int64_t kNtBytes = 16 << 20;

template <bool NT>
__device__ __forceinline__ void put_row(void* p, const uint4& v) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (NT) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
  else stg16(p, v);
}

// out[r] = in[perm[r] / k], zeros for no slot. A thread copies one vector of a row.
template <bool NT>
__global__ __launch_bounds__(256) void dispatch_kernel(PermuteArgs a, int row_vecs) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.R * row_vecs; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / row_vecs;
    const int v = (int)(i - r * row_vecs), s = a.perm[r];
    uint4 x = make_uint4(0, 0, 0, 0);
    if (s >= 0 && s < a.T * a.k) x = ldg16((const char*)a.in + ((int64_t)(s / a.k) * row_vecs + v) * 16);
    put_row<NT>((char*)a.out + i * 16, x);
  }
}

// out[t] = add[t] + sum_j gate[t][j] in[inv[t][j]], slots in order.
template <typename T, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(PermuteArgs a) {
  constexpr int VE = Elem<T>::VE;
  const int row_vecs = a.H / VE;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.T * row_vecs; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / row_vecs;
    const int c = (int)(i - t * row_vecs) * VE;
    float acc[VE];
#pragma unroll
    for (int q = 0; q < VE; ++q) acc[q] = 0.0f;
    if (a.add != nullptr) unpack(ldg16((const T*)a.add + t * a.H + c), acc, (T*)nullptr);
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int r = a.inv[t * a.k + j];
      if (r < 0 || r >= a.R) continue;
      const float g = a.gate != nullptr ? a.gate[t * a.k + j] : 1.0f;
      float f[VE];
      unpack(ldg16((const T*)a.in + (int64_t)r * a.H + c), f, (T*)nullptr);
#pragma unroll
      for (int q = 0; q < VE; ++q) acc[q] = __builtin_fmaf(g, f[q], acc[q]);
    }
    put_row<NT>((T*)a.out + t * a.H + c, pack(acc, (T*)nullptr));
  }
}

// A wave takes a slot: out[r] = gate dy[t], dgate = <dy[t], o[r]>. Behind the T k slots come the R rows,
// of which those of no slot are zeroed.
template <typename T, bool NT>
__global__ __launch_bounds__(256) void combine_bwd_kernel(PermuteArgs a) {
  constexpr int VE = Elem<T>::VE;
  const int lane = threadIdx.x & 63;
  const int64_t S = a.T * a.k, waves = S + (a.perm != nullptr ? a.R : 0);
  for (int64_t s = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); s < waves; s += (int64_t)gridDim.x * 4) {
    if (s >= S) {
      const int64_t r = s - S;
      const int q = a.perm[r];
      if (q >= 0 && q < S) continue;
      for (int c = lane * VE; c < a.H; c += 64 * VE) put_row<NT>((T*)a.out + r * a.H + c, make_uint4(0, 0, 0, 0));
      continue;
    }
    const int64_t t = s / a.k;
    const int r = a.inv[s];
    if (r < 0 || r >= a.R) {
      if (lane == 0 && a.dgate != nullptr) a.dgate[s] = 0.0f;
      continue;
    }
    const float g = a.gate != nullptr ? a.gate[s] : 1.0f;
    float sum = 0.0f;
    for (int c = lane * VE; c < a.H; c += 64 * VE) {
      float d[VE], o[VE];
      unpack(ldg16((const T*)a.in + t * a.H + c), d, (T*)nullptr);
      if (a.dgate != nullptr) {
        unpack(ldg16((const T*)a.o + (int64_t)r * a.H + c), o, (T*)nullptr);
#pragma unroll
        for (int q = 0; q < VE; ++q) sum = __builtin_fmaf(d[q], o[q], sum);
      }
#pragma unroll
      for (int q = 0; q < VE; ++q) d[q] *= g;
      put_row<NT>((T*)a.out + (int64_t)r * a.H + c, pack(d, (T*)nullptr));
    }
    if (a.dgate == nullptr) continue;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) a.dgate[s] = sum;
  }
}

unsigned blocks_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 22); }

template <typename T>
hipError_t run_combine(const PermuteArgs& a, hipStream_t s) {
  const int64_t n = a.T * (a.H / Elem<T>::VE);
  const bool nt = (int64_t)sizeof(T) * a.T * a.H > kNtBytes;
  const dim3 grid(blocks_of((n + 255) / 256)), block(256);
  if (nt) hipLaunchKernelGGL((combine_kernel<T, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_kernel<T, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_combine_bwd(const PermuteArgs& a, hipStream_t s) {
  const bool nt = (int64_t)sizeof(T) * a.R * a.H > kNtBytes;
  const int64_t waves = a.T * a.k + (a.perm != nullptr ? a.R : 0);
  const dim3 grid(blocks_of((waves + 3) / 4)), block(256);
  if (nt) hipLaunchKernelGGL((combine_bwd_kernel<T, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_bwd_kernel<T, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(const PermuteArgs& a, int act, hipStream_t s) {
  const int row_vecs = a.H / (act == MOK_F32 ? 4 : 8);
  const int64_t n = a.R * row_vecs;
  const dim3 grid(blocks_of((n + 255) / 256)), block(256);
  if (16 * n > kNtBytes) hipLaunchKernelGGL((dispatch_kernel<true>), grid, block, 0, s, a, row_vecs);
  else hipLaunchKernelGGL((dispatch_kernel<false>), grid, block, 0, s, a, row_vecs);
  return hipGetLastError();
}

hipError_t launch_combine(const PermuteArgs& a, int act, hipStream_t s) {
  return act == MOK_F32 ? run_combine<float>(a, s) : run_combine<bf16>(a, s);
}

hipError_t launch_combine_bwd(const PermuteArgs& a, int act, hipStream_t s) {
  return act == MOK_F32 ? run_combine_bwd<float>(a, s) : run_combine_bwd<bf16>(a, s);
}

}  // namespace mok
