// Rows to the experts' order and back (dispatch, combine) and their gradients. HBM-bound: each row is
// read once by 16-byte vectors and written once. A slot or row whose index is outside its range
// (-1: dropped, padding) counts as none.
#include "permute.h"

namespace mok {

namespace {

// Bytes of the rows that a call reads and writes, from which on it stores past the caches. The last one holds 256 MiB, and
// what was written stays there for its reader where it fits beside what was read. Through the caches and past them, k = 8,
// H = 7168, 16 experts: dispatch and the grouped product with 256 columns that reads xs, 22 MB of xs 66 and 92 us, 59 MB
// 73 and 102, 117 MB 92 and 118, 176 MB (198 in all) 130 and 137, 235 MB (264 in all) 172 and 163, 1.9 GB 1189 and 1140;
// combine's backward and its reader, 117 MB of d_o (250 in all) 123 and 135, 176 MB (375 in all) 173 and 169. The writer
// alone takes up to 2 us less past the caches.
constexpr int64_t kNtBytes = 256000000;

template <bool NT>
__device__ __forceinline__ void put_row(void* p, const uint4& v) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (NT) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
  else stg16(p, v);
}

// out[r] = in[perm[r] / k], zeros for no slot. 2^lanes lanes copy a row, four vectors of it in flight. 16384 x 8
// x 7168: 488 to 512 us over several cards (through the caches 557). The experts' order reads every row of x eight times,
// far apart, and x (235 MB) stays in the last cache for some of them only: 1.38 GB come from memory and 1.88 GB go
// there (traffic counters), 6.6 TB/s.
template <bool NT>
__global__ __launch_bounds__(256) void dispatch_kernel(PermuteArgs a, int row_vecs, int lanes) {
  const int step = 1 << lanes, v0 = threadIdx.x & (step - 1);
  const int64_t rows = (int64_t)gridDim.x << (8 - lanes);
  for (int64_t r = ((int64_t)blockIdx.x << (8 - lanes)) + (threadIdx.x >> lanes); r < a.R; r += rows) {
    const int s = a.perm[r];
    const bool on = s >= 0 && s < a.T * a.k;
    const char* src = (const char*)a.in + (int64_t)(on ? s / a.k : 0) * row_vecs * 16;
    char* dst = (char*)a.out + r * row_vecs * 16;
    if (on) {
#pragma unroll 4
      for (int v = v0; v < row_vecs; v += step) put_row<NT>(dst + (int64_t)v * 16, ldg16(src + (int64_t)v * 16));
    } else {
      for (int v = v0; v < row_vecs; v += step) put_row<NT>(dst + (int64_t)v * 16, make_uint4(0, 0, 0, 0));
    }
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

// 2^lanes lanes take a slot: out[r] = gate dy[t], dgate = <dy[t], o[r]>. Behind the T k slots come the R
// rows, of which those of no slot are zeroed.
template <typename T, bool NT>
__global__ __launch_bounds__(256) void combine_bwd_kernel(PermuteArgs a, int lanes) {
  constexpr int VE = Elem<T>::VE;
  const int step = 1 << lanes, c0 = (threadIdx.x & (step - 1)) * VE;
  const int64_t S = a.T * a.k, all = S + (a.perm != nullptr ? a.R : 0), items = (int64_t)gridDim.x << (8 - lanes);
  for (int64_t s = ((int64_t)blockIdx.x << (8 - lanes)) + (threadIdx.x >> lanes); s < all; s += items) {
    if (s >= S) {
      const int64_t r = s - S;
      const int q = a.perm[r];
      if (q >= 0 && q < S) continue;
      for (int c = c0; c < a.H; c += step * VE) put_row<NT>((T*)a.out + r * a.H + c, make_uint4(0, 0, 0, 0));
      continue;
    }
    const int64_t t = (uint32_t)s / (uint32_t)a.k;  // T k < 2^31
    const int r = a.inv[s];
    if (r < 0 || r >= a.R) {
      if (c0 == 0 && a.dgate != nullptr) a.dgate[s] = 0.0f;
      continue;
    }
    const float g = a.gate != nullptr ? a.gate[s] : 1.0f;
    float sum = 0.0f;
#pragma unroll 2
    for (int c = c0; c < a.H; c += step * VE) {
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
    for (int o = 1; o < step; o <<= 1) sum += __shfl_xor(sum, o);  // the lanes of a slot go through here together
    if (c0 == 0) a.dgate[s] = sum;
  }
}

// Lanes of a row of n vectors, as a power of two up to a wave.
int row_lanes(int n) {
  int lanes = 0;
  while (lanes < 6 && (1 << lanes) < n) ++lanes;
  return lanes;
}

unsigned blocks_of(int64_t n) { return (unsigned)std::min<int64_t>(n, 1 << 22); }

template <typename T>
hipError_t run_combine(const PermuteArgs& a, hipStream_t s) {
  const int64_t n = a.T * (a.H / Elem<T>::VE);
  const bool nt = (int64_t)sizeof(T) * (a.R + a.T) * a.H > kNtBytes;
  const dim3 grid(blocks_of((n + 255) / 256)), block(256);
  if (nt) hipLaunchKernelGGL((combine_kernel<T, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_kernel<T, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_combine_bwd(const PermuteArgs& a, hipStream_t s) {
  const bool nt = (int64_t)sizeof(T) * (a.R * (a.dgate != nullptr ? 2 : 1) + a.T) * a.H > kNtBytes;
  const int lanes = row_lanes(a.H / Elem<T>::VE);
  const int64_t items = a.T * a.k + (a.perm != nullptr ? a.R : 0), per = 256 >> lanes;
  const dim3 grid(blocks_of((items + per - 1) / per)), block(256);
  if (nt) hipLaunchKernelGGL((combine_bwd_kernel<T, true>), grid, block, 0, s, a, lanes);
  else hipLaunchKernelGGL((combine_bwd_kernel<T, false>), grid, block, 0, s, a, lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(const PermuteArgs& a, int act, hipStream_t s) {
  const int row_vecs = a.H / (act == MOK_F32 ? 4 : 8);
  const int lanes = row_lanes(row_vecs);
  const int64_t per = 256 >> lanes;
  const dim3 grid(blocks_of((a.R + per - 1) / per)), block(256);
  if (16 * (a.R + a.T) * row_vecs > kNtBytes) hipLaunchKernelGGL((dispatch_kernel<true>), grid, block, 0, s, a, row_vecs, lanes);
  else hipLaunchKernelGGL((dispatch_kernel<false>), grid, block, 0, s, a, row_vecs, lanes);
  return hipGetLastError();
}

hipError_t launch_combine(const PermuteArgs& a, int act, hipStream_t s) {
  return act == MOK_F32 ? run_combine<float>(a, s) : run_combine<bf16>(a, s);
}

hipError_t launch_combine_bwd(const PermuteArgs& a, int act, hipStream_t s) {
  return act == MOK_F32 ? run_combine_bwd<float>(a, s) : run_combine_bwd<bf16>(a, s);
}

}  // namespace mok
