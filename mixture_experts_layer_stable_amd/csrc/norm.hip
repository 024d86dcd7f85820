// RMS norm with the residual's addition: forward (optionally with the MX rows of the result)
// and backward, and the column sum of partial rows.
//
// One pass: a group of G lanes holds a whole row in registers (up to VPT 16-byte vectors per
// lane), sums v^2 (backward: g * xh) over the row, and writes the outputs from the registers,
// so each input is read once and each output written once. Bound by HBM.
#include "block.h"
#include "mx.h"

namespace mok {
// Row stores of big arrays go past the caches, which could not keep them for a reader (more than
// kNtBytes an output: 2048 x 7168 with MX rows 33 -> 25 us, 16384 x 7168 166 -> 159 us).
constexpr int64_t kNtBytes = 16 << 20;

template <bool NT>
__device__ __forceinline__ void row_store(void* p, const uint4& v) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  if constexpr (NT) __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_t*>(p));
  else stg16(p, v);
}

// Sum over a group of G lanes (a power of two up to 64, or whole waves of one workgroup),
// in a fixed order; every lane gets it. s_red: one per wave. All lanes of the
// workgroup call it.
template <typename V>
__device__ __forceinline__ V group_sum(V v, int G, V* s_red) {
  const int w = G < 64 ? G : 64;
  for (int o = 1; o < w; o <<= 1) v += __shfl_xor(v, o);
  if (G <= 64) return v;
  const int wave = threadIdx.x >> 6, gw = G >> 6, w0 = wave / gw * gw;
  if ((threadIdx.x & 63) == 0) s_red[wave] = v;
  __syncthreads();
  V t = 0;
  for (int i = 0; i < gw; ++i) t += s_red[w0 + i];
  __syncthreads();
  return t;
}

// 1 / sqrt(x) to half a step: the hardware's estimate and one Newton step on its exact residual. The
// estimate takes a subnormal x for 0: it is formed of x 2^24, which is exact, as is the factor 2^12 after.
__device__ __forceinline__ float rsqrt_round(float mean) {
  const bool tiny = mean < 0x1p-126f;
  const float x = tiny ? mean * 0x1p24f : mean;
  const float r = __builtin_amdgcn_rsqf(x), h = x * r;
  const float e = __builtin_fmaf(-h, r, 1.0f) - __builtin_fmaf(x, r, -h) * r;  // 1 - x r^2
  const float y = x > 0.0f && x < INFINITY ? __builtin_fmaf(0.5f * r, e, r) : r;
  return tiny ? y * 0x1p12f : y;
}

// Lanes per row, rows per workgroup and vectors per lane for rows of nv vectors: small rows
// share a workgroup of 256 lanes, a row of more than 256 vectors has one of its own.
struct NormShape {
  int G, rows, vpt;
};
inline NormShape norm_shape(int H, int act) {
  const int nv = H / (act == MOK_F32 ? 4 : 8);
  if (nv <= 256) {
    int G = 16;
    while (G < nv) G <<= 1;
    return {G, 256 / G, 1};
  }
  const int vpt = nv <= 2048 ? 2 : (nv <= 4096 ? 4 : 8);
  return {(nv + 64 * vpt - 1) / (64 * vpt) * 64, 1, vpt};
}

template <typename T, int VPT, int Q, bool NT>  // Q: 0 none, 1 MXFP8, 2 MXFP4
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormArgs a, int G) {
  constexpr int VE = Elem<T>::VE;
  __shared__ double s_red[16];
  const int g = threadIdx.x / G, l = threadIdx.x - g * G, nv = a.H / VE;
  const int rows = blockDim.x / G;
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += (int64_t)gridDim.x * rows) {
    const int64_t t = t0 + g;
    const bool on = t < a.T;
    const int64_t base = t * a.H;
    float v[VPT][VE];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = l + j * G;
#pragma unroll
      for (int e = 0; e < VE; ++e) v[j][e] = 0.0f;
      if (on && i < nv) {
        unpack(ldg16((const T*)a.x + base + i * VE), v[j], (T*)nullptr);
        if (a.res != nullptr) {
          float f[VE];
          unpack(ldg16((const T*)a.res + base + i * VE), f, (T*)nullptr);
#pragma unroll
          for (int e = 0; e < VE; ++e) v[j][e] += f[e];
        }
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) ss = __builtin_fmaf(v[j][e], v[j][e], ss);
    }
    // An error of rstd moves a whole row, and with it every y next to a rounding border of bf16 or of
    // the MX elements: the lanes' sums are added in fp64 and the root is right to half a step (of 14.7 M
    // elements of y 75 are not the nearest bf16; the double rounding through fp32 alone gives 70).
    const float rstd = rsqrt_round((float)(group_sum((double)ss, G, s_red) / a.H + (double)a.eps));
    if (on && l == 0 && a.rstd != nullptr) a.rstd[t] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = l + j * G;
      const bool in = on && i < nv;
      float f[VE];
      if (in) {
        if (a.r != nullptr) row_store<NT>((T*)a.r + base + i * VE, pack(v[j], (T*)nullptr));
        unpack(ldg16((const T*)a.w + i * VE), f, (T*)nullptr);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = v[j][e] * rstd * f[e];
        const uint4 o = pack(f, (T*)nullptr);
        if (a.y != nullptr) row_store<NT>((T*)a.y + base + i * VE, o);
        if constexpr (Q != 0) unpack(o, f, (T*)nullptr);  // the quantiser's input is the stored bf16 value
      }
      if constexpr (Q != 0) {
        // H is a multiple of 128: the 16 lanes of a K-tile (four blocks of four lanes) are all
        // in or all out of the row
        float m = 0.0f;
        if (in) {
#pragma unroll
          for (int e = 0; e < VE; ++e) m = fmaxf(m, fabsf(f[e]));
        }
        m = fmaxf(m, __shfl_xor(m, 1));
        m = fmaxf(m, __shfl_xor(m, 2));
        const uint32_t sb = Q == 1 ? mx_scale_byte(m) : mx4_scale_byte(m);
        const float inv = mx_inv_scale(sb);
        uint32_t sw = sb << (8 * ((l >> 2) & 3));
        sw |= __shfl_xor(sw, 4);
        sw |= __shfl_xor(sw, 8);
        if (in) {
          if constexpr (Q == 1) {
            *reinterpret_cast<uint2*>(a.q + base + i * VE) =
                make_uint2(mx_pack4(f[0], f[1], f[2], f[3], inv), mx_pack4(f[4], f[5], f[6], f[7], inv));
          } else {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < VE; ++e) w |= e2m1_code(f[e] * inv) << (4 * e);
            *reinterpret_cast<uint32_t*>(a.q + (base + i * VE) / 2) = w;
          }
          if ((i & 15) == 0) *reinterpret_cast<uint32_t*>(a.s + ((int64_t)(i >> 4) * a.T + t) * 4) = sw;
        }
      }
    }
  }
}

template <typename T, int VPT, bool NT>
static void norm_fwd_q(const NormArgs& a, int quant, const NormShape& n, hipStream_t s) {
  // a workgroup a row group, up to the 2^32 threads that a launch can have
  const dim3 grid((unsigned)std::min<int64_t>((a.T + n.rows - 1) / n.rows, 1 << 21)), block(n.G * n.rows);
  if constexpr (std::is_same<T, bf16>::value) {
    if (quant == MOK_MXFP8) {
      hipLaunchKernelGGL((norm_fwd_kernel<T, VPT, 1, NT>), grid, block, 0, s, a, n.G);
      return;
    }
    if (quant == MOK_MXFP4) {
      hipLaunchKernelGGL((norm_fwd_kernel<T, VPT, 2, NT>), grid, block, 0, s, a, n.G);
      return;
    }
  }
  hipLaunchKernelGGL((norm_fwd_kernel<T, VPT, 0, NT>), grid, block, 0, s, a, n.G);
}

template <typename T, bool NT>
static void norm_fwd_t(const NormArgs& a, int quant, const NormShape& n, hipStream_t s) {
  if (n.vpt == 1) norm_fwd_q<T, 1, NT>(a, quant, n, s);
  else if (n.vpt == 2) norm_fwd_q<T, 2, NT>(a, quant, n, s);
  else if (n.vpt == 4) norm_fwd_q<T, 4, NT>(a, quant, n, s);
  else norm_fwd_q<T, 8, NT>(a, quant, n, s);
}

hipError_t launch_norm_fwd(const NormArgs& a, int act, int quant, hipStream_t s) {
  const NormShape n = norm_shape(a.H, act);
  const bool nt = a.T * a.H * (act == MOK_F32 ? 4 : 2) > kNtBytes;
  if (act == MOK_F32) nt ? norm_fwd_t<float, true>(a, quant, n, s) : norm_fwd_t<float, false>(a, quant, n, s);
  else nt ? norm_fwd_t<bf16, true>(a, quant, n, s) : norm_fwd_t<bf16, false>(a, quant, n, s);
  return hipGetLastError();
}

// Backward: a workgroup takes row groups blockIdx, blockIdx + grid, ... and keeps its columns'
// share of dw in registers, in fp32, one row after the other (T / 512 of them; fewer where rows lie
// side by side); the row groups of a workgroup are added in LDS in group order and written as one
// partial row. dr is loaded with dy and r, ahead of the row's sum (16384 x 7168: 202 -> 172 us, 5.5
// TB/s; the next row's loads ahead of the sum too: 265, its registers spill); 512 workgroups, two per
// CU (768: 205 us, 1024: 180, 256: 321).
template <typename T, int VPT, bool NT>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormArgs a, int G) {
  constexpr int VE = Elem<T>::VE;
  __shared__ float s_red[16];
  extern __shared__ float s_dw[];  // [rows per workgroup][H] when it has more than one row group
  const int rows = blockDim.x / G, g = threadIdx.x / G, l = threadIdx.x - g * G, nv = a.H / VE;
  const int64_t groups = (a.T + rows - 1) / rows;
  float dw[VPT][VE];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = 0.0f;
  for (int64_t b = blockIdx.x; b < groups; b += gridDim.x) {
    const int64_t t = b * rows + g, base = t * a.H;
    const bool on = t < a.T;
    const float rstd = on ? a.rstd[t] : 0.0f;
    float gv[VPT][VE], xh[VPT][VE];
    uint4 dr[VPT];
    float c = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = l + j * G;
#pragma unroll
      for (int e = 0; e < VE; ++e) gv[j][e] = xh[j][e] = 0.0f;
      if (on && i < nv) {
        float w[VE];
        unpack(ldg16((const T*)a.dy + base + i * VE), gv[j], (T*)nullptr);
        unpack(ldg16((const T*)a.r + base + i * VE), xh[j], (T*)nullptr);
        unpack(ldg16((const T*)a.w + i * VE), w, (T*)nullptr);
        dr[j] = a.dr != nullptr ? ldg16((const T*)a.dr + base + i * VE) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          xh[j][e] *= rstd;
          dw[j][e] = __builtin_fmaf(gv[j][e], xh[j][e], dw[j][e]);
          gv[j][e] *= w[e];
          c = __builtin_fmaf(gv[j][e], xh[j][e], c);
        }
      }
    }
    c = group_sum(c, G, s_red) / (float)a.H;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = l + j * G;
      if (on && i < nv) {
        float f[VE];
        unpack(dr[j], f, (T*)nullptr);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = __builtin_fmaf(rstd, gv[j][e] - xh[j][e] * c, f[e]);
        row_store<NT>((T*)a.dx + base + i * VE, pack(f, (T*)nullptr));
      }
    }
  }
  if (a.part == nullptr) return;
  float* out = a.part + (int64_t)blockIdx.x * a.H;
  if (rows == 1) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = l + j * G;
      if (i < nv)
#pragma unroll
        for (int e = 0; e < VE; ++e) out[i * VE + e] = dw[j][e];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = l + j * G;
    if (i < nv)
#pragma unroll
      for (int e = 0; e < VE; ++e) s_dw[g * a.H + i * VE + e] = dw[j][e];
  }
  __syncthreads();
  for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
    float v = 0.0f;
    for (int q = 0; q < rows; ++q) v += s_dw[q * a.H + h];
    out[h] = v;
  }
}

int norm_parts(int64_t T, int H, int act) {
  const NormShape n = norm_shape(H, act);
  const int64_t groups = (T + n.rows - 1) / n.rows;
  return (int)std::min<int64_t>(groups, 512);
}

template <typename T, bool NT>
static void norm_bwd_t(const NormArgs& a, const NormShape& n, int grid, hipStream_t s) {
  const size_t lds = n.rows > 1 ? 4 * (size_t)n.rows * a.H : 0;
  const dim3 block(n.G * n.rows);
  if (n.vpt == 1) hipLaunchKernelGGL((norm_bwd_kernel<T, 1, NT>), dim3(grid), block, lds, s, a, n.G);
  else if (n.vpt == 2) hipLaunchKernelGGL((norm_bwd_kernel<T, 2, NT>), dim3(grid), block, lds, s, a, n.G);
  else if (n.vpt == 4) hipLaunchKernelGGL((norm_bwd_kernel<T, 4, NT>), dim3(grid), block, lds, s, a, n.G);
  else hipLaunchKernelGGL((norm_bwd_kernel<T, 8, NT>), dim3(grid), block, lds, s, a, n.G);
}

hipError_t launch_norm_bwd(const NormArgs& a, int act, hipStream_t s) {
  const NormShape n = norm_shape(a.H, act);
  const int grid = norm_parts(a.T, a.H, act);
  const bool nt = a.T * a.H * (act == MOK_F32 ? 4 : 2) > kNtBytes;
  if (act == MOK_F32) nt ? norm_bwd_t<float, true>(a, n, grid, s) : norm_bwd_t<float, false>(a, n, grid, s);
  else nt ? norm_bwd_t<bf16, true>(a, n, grid, s) : norm_bwd_t<bf16, false>(a, n, grid, s);
  return hipGetLastError();
}

// Workgroup: 64 columns, 16 waves; wave w adds partial rows w, w + 16, ..., then the waves'
// sums are added in wave order.
__global__ __launch_bounds__(1024) void col_sum_kernel(const float* __restrict__ part, int P, int H, void* out,
                                                       bool f32) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (h < H) {
#pragma unroll 8
    for (int p = wave; p < P; p += 16) v += part[(int64_t)p * H + h];
  }
  s_sum[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || h >= H) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) t += s_sum[i][lane];
  if (f32) reinterpret_cast<float*>(out)[h] = t;
  else reinterpret_cast<bf16*>(out)[h] = (bf16)f32_to_bf16(t);
}

hipError_t launch_col_sum(const float* part, int P, int H, void* out, bool f32, hipStream_t s) {
  hipLaunchKernelGGL(col_sum_kernel, dim3((H + 63) / 64), dim3(1024), 0, s, part, P, H, out, f32);
  return hipGetLastError();
}

}  // namespace mok
