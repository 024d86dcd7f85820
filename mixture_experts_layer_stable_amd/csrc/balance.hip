// Balance loss of the router: scores, per-expert counts and sums over ragged segments, and the
// gradient by the logits.
//
// Forward, two launches: (1) a workgroup takes a chunk of consecutive tokens; a group of G lanes
// holds one token's logits in registers (one read, the next token's on their way), forms its
// scores and adds them to the lanes' own per-expert sums; slots are counted with integer LDS
// atomics; where a segment ends inside the chunk the sums are written out as the partial row of
// (chunk, segment). (2) one workgroup per (64 experts, segment) adds the segment's partial rows;
// the last of them adds the parts of the loss. Batches of up to 2^14 logits take one launch of one
// workgroup for all of it. No float atomics: the sums depend on T, E and the segments only. Bound
// by HBM (logits read once) or, for small batches, by the launches.
// Backward: one launch, one read of the logits and one write of their gradient.
#include <cmath>

#include "api.h"
#include "block.h"

namespace mok {

namespace {

constexpr int kThreadsB = 256;
// Four workgroups per CU, as long as a chunk keeps 32 rows.
constexpr int kBalanceChunks = 1024, kBalanceRows = 32;
constexpr int64_t kBalanceSmall = 1 << 14;  // logits of a batch for one workgroup
constexpr int kBalanceSmallSegs = 64;

// Logits of one token over G lanes: J vectors of VEC per lane (vector j*G + lane), at most 16
// values. VEC = 4 where the rows are 16-byte aligned (E a multiple of 4).
struct RowShape {
  int G, J, vec;
};
RowShape row_shape(int E) {
  const int vec = E % 4 == 0 ? 4 : 1, nv = E / vec, most = 16 / vec;
  int G = 1;
  while (G < 64 && G * most < nv) G <<= 1;
  int J = (nv + G - 1) / G;
  if (vec == 1) {  // instantiated for powers of two
    int p = 1;
    while (p < J) p <<= 1;
    J = p;
  }
  return {G, J, vec};
}

template <int VEC, int J>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, int G, float fill,
                                         float (&v)[J * VEC]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = (l + j * G) * VEC;
    if constexpr (VEC == 4) {
      const float4 f = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(fill, fill, fill, fill);
      v[4 * j] = f.x;
      v[4 * j + 1] = f.y;
      v[4 * j + 2] = f.z;
      v[4 * j + 3] = f.w;
    } else {
      v[j] = e < E ? row[e] : fill;
    }
  }
}

__device__ __forceinline__ float lanes_sum(float v, int G) {
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float lanes_max(float v, int G) {
  for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// exp(x) for x <= 0 to two steps of fp32: the hardware's exp2 of the rounded product, corrected
// by the product's own rounding error. Below -150 it is 0 (a NaN stays one); the library's expf,
// for every range, made these kernels vector-ALU bound (131072 x 256 sigmoid forward 96 us).
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
  const float y = x < -150.0f ? -150.0f : x;
  const float t = y * kLog2e, lo = __builtin_fmaf(y, kLog2e, -t);
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * kLn2, lo, e);
}

// A token's scores up to a common factor, from its logits z and their maximum m over the group:
// exp(z - m), or sig(z) exp(-min(m, 0)) -- normalised sigmoid scores do not change by the factor,
// and a token whose every logit is far below 0 keeps its digits. Without a finite logit they are 0
// (a NaN stays one). shift is subtracted in the softmax's exponent (the backward's normaliser);
// slope (when asked for) receives 1 - sig(z), without a cancellation.
template <bool SIG, bool SLOPE, int NV>
__device__ __forceinline__ void scores(float (&z)[NV], float m, float shift, float (&slope)[NV]) {
  if (m == -INFINITY) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      z[i] = z[i] == -INFINITY ? 0.0f : z[i];
      if constexpr (SLOPE) slope[i] = 0.0f;
    }
  } else if constexpr (!SIG) {
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] = exp_neg((z[i] - m) - shift);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float e = exp_neg(-fabsf(z[i])), d = __builtin_amdgcn_rcpf(1.0f + e);
      if constexpr (SLOPE) slope[i] = z[i] > 0.0f ? e * d : d;
      // with a logit above 0 the factor is 1: sig(z) = d or e d
      z[i] = (m >= 0.0f ? (z[i] > 0.0f ? 1.0f : e) : exp_neg(z[i] - m)) * d;
    }
  }
}

// Segment bounds, clamped to the token range.
__device__ __forceinline__ int64_t seg_at(const BalanceArgs& a, int s) {
  if (a.seg == nullptr) return s == 0 ? 0 : a.T;
  const int64_t v = a.seg[s];
  return v < 0 ? 0 : (v > a.T ? a.T : v);
}

// First segment that ends after token t (S if there is none).
__device__ __forceinline__ int seg_of(const BalanceArgs& a, int64_t t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (seg_at(a, m + 1) <= t) lo = m + 1; else hi = m;
  }
  return lo;
}

template <int NT>
__device__ __forceinline__ double block_sum(double v, double* s_w) {
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < NT / 64; ++i) v += s_w[i];
  return v;
}

// The loss from the sum l of its segments' parts, the sum z of lse^2, and the segments' tokens.
template <int NT>
__device__ void finish_loss(const BalanceArgs& a, double l, double z, double* s_w) {
  double n = 0.0, full = 0.0;
  for (int i = threadIdx.x; i < a.S; i += NT) {
    const int t = __hip_atomic_load(a.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    n += t;
    full += t > 0;
  }
  l = block_sum<NT>(l, s_w);
  z = block_sum<NT>(z, s_w);
  n = block_sum<NT>(n, s_w);
  full = block_sum<NT>(full, s_w);
  if (threadIdx.x != 0) return;
  a.loss[0] = full > 0.0 ? (float)((double)a.coef / full * l) : 0.0f;
  a.loss[1] = n > 0.0 && a.zcoef != 0.0f ? (float)((double)a.zcoef / n * z) : 0.0f;
  a.tokens[a.S] = (int)full;
  a.tokens[a.S + 1] = (int)n;
}

// ALL: one workgroup takes every token and writes the results itself.
template <int NT, bool ALL, bool SIG, int VEC, int J>
__global__ __launch_bounds__(NT) void balance_rows_kernel(BalanceArgs a, int G) {
  constexpr int NV = VEC * J;
  constexpr int NW = NT / 64;
  __shared__ float s_q[NW * (NV > 4 ? 1024 : 256)];  // [waves][E]; E <= 64 NV, and G >= E / 16
  __shared__ int s_c[1024];
  __shared__ int s_n;
  __shared__ double s_w[NT / 64];
  const int tid = threadIdx.x, g = tid / G, l = tid - g * G, groups = NT / G;
  const int64_t c0 = ALL ? 0 : (int64_t)blockIdx.x * a.rows, c1 = ALL ? a.T : min(a.T, c0 + a.rows);
  float zsum = 0.0f;
  double loss = 0.0;
  if (!ALL && blockIdx.x == 0 && tid == 0) *a.done = 0;
  for (int s = ALL ? 0 : seg_of(a, c0); s < a.S; ++s) {
    const int64_t s0 = seg_at(a, s), s1 = seg_at(a, s + 1);
    if (!ALL && s0 >= c1) break;
    const int64_t t0 = max(s0, c0), t1 = min(s1, c1);
    if (!ALL && t1 <= t0) continue;
    const auto counts = [&](int64_t t) { return t < t1 && (a.mask == nullptr || a.mask[t] != 0); };
    float z[NV], zn[NV];  // this token's logits, the next one's
    int64_t t = t0 + g;
    bool on = counts(t);
    if (on) load_row<VEC, J>(a.logits + t * a.E, a.E, l, G, -INFINITY, zn);
    for (int e = tid; e < a.E; e += NT) s_c[e] = 0;
    if (tid == 0) s_n = 0;
    __syncthreads();
    // slots
    int n = 0;
    for (int64_t u = t0 + tid; u < t1; u += NT) {
      if (!counts(u)) continue;
      const int32_t* ids = a.idx + u * a.k;
      for (int j = 0; j < a.k; ++j) {
        const int e = ids[j];
        if (e >= 0 && e < a.E) atomicAdd(&s_c[e], 1);
      }
      ++n;
    }
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    if ((tid & 63) == 0 && n != 0) atomicAdd(&s_n, n);
    // scores
    float q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = 0.0f;
    for (int64_t b = t0; b < t1; b += groups, t += groups) {
      const bool cur = on;
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] = cur ? zn[i] : 0.0f;
      on = counts(t + groups);
      if (on) load_row<VEC, J>(a.logits + (t + groups) * a.E, a.E, l, G, -INFINITY, zn);
      float sum = 0.0f;
      float m = z[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, z[i]);
      m = lanes_max(m, G);
      scores<SIG, false, NV>(z, m, 0.0f, z);
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += z[i];
      sum = lanes_sum(sum, G);
      if constexpr (SIG) {
        if (cur && l == 0) a.stat[t] = sum;
      } else {
        // stat is the log of the sum relative to the maximum: added to a large maximum it
        // would lose its digits, and the backward's scores with them
        if (cur && l == 0) {
          const float st = sum == 0.0f ? 0.0f : logf(sum), lse = m + st;
          a.stat[t] = st;
          if (sum != 0.0f) zsum = __builtin_fmaf(lse, lse, zsum);
        }
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (cur) {
#pragma unroll
        for (int i = 0; i < NV; ++i) q[i] = __builtin_fmaf(z[i], inv, q[i]);
      }
    }
    // the groups of a wave, then the waves in order
#pragma unroll
    for (int i = 0; i < NV; ++i)
      for (int o = G; o < 64; o <<= 1) q[i] += __shfl_xor(q[i], o);
    if ((tid & 63) < G) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const int e = (l + j * G) * VEC + v;
          if (e < a.E) s_q[(tid >> 6) * a.E + e] = q[j * VEC + v];
        }
    }
    __syncthreads();
    const int ns = s_n;
    for (int e = tid; e < a.E; e += NT) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) v += s_q[i * a.E + e];
      if constexpr (ALL) {
        a.counts[(int64_t)s * a.E + e] = s_c[e];
        a.prob[(int64_t)s * a.E + e] = ns > 0 ? v / (float)ns : 0.0f;
        if (ns > 0) loss += (double)s_c[e] * v * ((double)a.E / ((double)a.k * ns * ns));
      } else {
        const int64_t at = (int64_t)blockIdx.x + s;
        a.wq[at * a.E + e] = v;
        a.wc[at * a.E + e] = s_c[e];
      }
    }
    if (tid == 0) {
      if constexpr (ALL) a.tokens[s] = ns;
      else a.wn[(int64_t)blockIdx.x + s] = ns;
    }
    __syncthreads();
  }
  if constexpr (ALL) {
    finish_loss<NT>(a, loss, zsum, s_w);
  } else {
    const double z = block_sum<NT>(zsum, s_w);
    if (tid == 0) a.wz[blockIdx.x] = (float)z;
  }
}

// Workgroup (64 experts, segment): wave w adds the partial rows w, w + 16, ... of the segment.
__global__ __launch_bounds__(1024) void balance_seg_kernel(BalanceArgs a) {
  __shared__ double s_q[16][64];
  __shared__ int s_c[16][64];
  __shared__ int s_n[16];
  __shared__ double s_w[16];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane, s = blockIdx.y;
  const int64_t s0 = seg_at(a, s), s1 = seg_at(a, s + 1);
  const int lo = (int)(s0 / a.rows), hi = s1 > s0 ? (int)((s1 - 1) / a.rows) + 1 : lo;
  double q = 0.0;
  int c = 0, n = 0;
  if (e < a.E) {
#pragma unroll 16
    for (int i = lo + wave; i < hi; i += 16) {
      const int64_t at = ((int64_t)i + s) * a.E + e;
      q += (double)a.wq[at];
      c += a.wc[at];
    }
  }
  for (int i = lo + (int)threadIdx.x; i < hi; i += 1024) n += a.wn[i + s];
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  s_q[wave][lane] = q;
  s_c[wave][lane] = c;
  if (lane == 0) s_n[wave] = n;
  __syncthreads();
  if (wave == 0) {
    q = 0.0;
    c = n = 0;
    for (int i = 0; i < 16; ++i) {
      q += s_q[i][lane];
      c += s_c[i][lane];
      n += s_n[i];
    }
    double part = 0.0;
    if (e < a.E) {
      a.counts[(int64_t)s * a.E + e] = c;
      a.prob[(int64_t)s * a.E + e] = n > 0 ? (float)(q / n) : 0.0f;
      if (n > 0) part = (double)c * q * ((double)a.E / ((double)a.k * n * n));
    }
    for (int o = 1; o < 64; o <<= 1) part += __shfl_xor(part, o);
    if (lane == 0) {
      __hip_atomic_store(a.wl + (int64_t)s * gridDim.x + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (blockIdx.x == 0) __hip_atomic_store(a.tokens + s, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // Both stores go past the XCD's L2 and have arrived before this workgroup is counted; the last
      // one counted reads them all past its L2. (A release would write the whole L2 back: 5 us.)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const int parts = gridDim.x * gridDim.y;
      s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  double l = 0.0, z = 0.0;
  for (int i = threadIdx.x; i < (int)(gridDim.x * gridDim.y); i += 1024)
    l += __hip_atomic_load(a.wl + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = threadIdx.x; i < a.chunks; i += 1024) z += (double)a.wz[i];
  finish_loss<1024>(a, l, z, s_w);
}

template <typename TO, bool SIG, int VEC, int J>
__global__ __launch_bounds__(kThreadsB) void balance_grad_kernel(BalanceArgs a, int G, int64_t rows) {
  constexpr int NV = VEC * J;
  const int tid = threadIdx.x, g = tid / G, l = tid - g * G, groups = kThreadsB / G;
  const int64_t c0 = (int64_t)blockIdx.x * rows, c1 = min(a.T, c0 + rows);
  const int full = a.tokens[a.S], N = a.tokens[a.S + 1];
  const float gz = N > 0 ? a.dloss[1] * a.zcoef * 2.0f / (float)N : 0.0f;
  int64_t s0 = 0, s1 = -1;  // bounds of the segment that c[] belongs to
  float c[NV], gs = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = 0.0f;
  for (int64_t t = c0 + g; t < c1; t += groups) {
    if (t >= s1) {
      const int s = seg_of(a, t);
      if (s < a.S) {
        s0 = seg_at(a, s);
        s1 = seg_at(a, s + 1);
        const float n = (float)a.tokens[s];
        gs = n > 0.0f ? a.dloss[0] * a.coef * (float)a.E / ((float)full * (float)a.k * n * n) : 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const int e = (l + j * G) * VEC + v;
            c[j * VEC + v] = e < a.E ? (float)a.counts[(int64_t)s * a.E + e] : 0.0f;
          }
      } else {
        s0 = s1 = a.T;  // no segment from here on
      }
    }
    const bool on = t >= s0 && t < s1 && (a.mask == nullptr || a.mask[t] != 0);
    float z[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] = 0.0f;
    if (on) {
      load_row<VEC, J>(a.logits + t * a.E, a.E, l, G, -INFINITY, z);
      const float st = a.stat[t];
      float m = z[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, z[i]);
      m = lanes_max(m, G);
      float dot = 0.0f, slope[NV];
      scores<SIG, SIG, NV>(z, m, SIG ? 0.0f : st, slope);
      if constexpr (SIG) {
        const float inv = st == 0.0f ? 0.0f : 1.0f / st;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          z[i] *= inv;
          dot = __builtin_fmaf(z[i], c[i], dot);
        }
        dot = lanes_sum(dot, G);
#pragma unroll
        for (int i = 0; i < NV; ++i) z[i] = z[i] * slope[i] * (gs * (c[i] - dot));
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) dot = __builtin_fmaf(z[i], c[i], dot);
        dot = lanes_sum(dot, G);
        const float h = m == -INFINITY || gz == 0.0f ? 0.0f : gz * (m + st);
#pragma unroll
        for (int i = 0; i < NV; ++i) z[i] *= __builtin_fmaf(gs, c[i] - dot, h);
      }
    }
    TO* out = reinterpret_cast<TO*>(a.dlogits) + t * a.E;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = (l + j * G) * VEC;
      if (e >= a.E) continue;
      if constexpr (VEC == 4 && std::is_same<TO, float>::value) {
        *reinterpret_cast<float4*>(out + e) = make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
      } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(out + e) =
            make_uint2(bf16x2_rne(z[4 * j], z[4 * j + 1]), bf16x2_rne(z[4 * j + 2], z[4 * j + 3]));
      } else {
        Elem<TO>::put(out, e, z[j]);
      }
    }
  }
}

// f(std::integral_constant VEC, std::integral_constant J) for a row shape
template <class F>
void with_shape(const RowShape& r, F&& f) {
  using std::integral_constant;
  if (r.vec == 4) {
    const integral_constant<int, 4> v;
    if (r.J == 1) f(v, integral_constant<int, 1>());
    else if (r.J == 2) f(v, integral_constant<int, 2>());
    else if (r.J == 3) f(v, integral_constant<int, 3>());
    else f(v, integral_constant<int, 4>());
  } else {
    const integral_constant<int, 1> v;
    if (r.J == 1) f(v, integral_constant<int, 1>());
    else if (r.J == 2) f(v, integral_constant<int, 2>());
    else if (r.J == 4) f(v, integral_constant<int, 4>());
    else if (r.J == 8) f(v, integral_constant<int, 8>());
    else f(v, integral_constant<int, 16>());
  }
}

}  // namespace

BalanceWs balance_ws(int64_t T, int E, int S) {
  BalanceWs w;
  w.rows = (int)std::max<int64_t>(kBalanceRows, (T + kBalanceChunks - 1) / kBalanceChunks);
  w.chunks = (int)std::max<int64_t>(1, (T + w.rows - 1) / w.rows);
  const size_t pairs = (size_t)w.chunks + S;
  size_t o = 0;
  w.q = o; o = up(o + 4 * pairs * E);
  w.c = o; o = up(o + 4 * pairs * E);
  w.n = o; o = up(o + 4 * pairs);
  w.z = o; o = up(o + 4 * (size_t)w.chunks);
  w.done = o; o = up(o + 4);
  w.loss = o; o = up(o + 8 * (size_t)S * ((E + 63) / 64));
  w.bytes = o;
  return w;
}

hipError_t launch_balance_fwd(const BalanceArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.E);
  const bool all = a.T * a.E <= kBalanceSmall && a.S <= kBalanceSmallSegs;
  with_shape(r, [&](auto v, auto j) {
    constexpr int V = decltype(v)::value, JJ = decltype(j)::value;
    const auto go = [&](auto sig) {
      constexpr bool SIG = decltype(sig)::value;
      if (all)
        hipLaunchKernelGGL((balance_rows_kernel<1024, true, SIG, V, JJ>), dim3(1), dim3(1024), 0, s, a, r.G);
      else
        hipLaunchKernelGGL((balance_rows_kernel<kThreadsB, false, SIG, V, JJ>), dim3(a.chunks), dim3(kThreadsB), 0, s, a,
                           r.G);
    };
    if (a.sigmoid) go(std::true_type());
    else go(std::false_type());
  });
  if (!all) hipLaunchKernelGGL(balance_seg_kernel, dim3((a.E + 63) / 64, a.S), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.E);
  const int groups = kThreadsB / r.G;
  // consecutive tokens per workgroup: 2048 workgroups at most, at least one pass of the groups
  const int64_t rows = std::max<int64_t>(groups, (a.T + 2047) / 2048);
  const int grid = (int)((a.T + rows - 1) / rows);
  with_shape(r, [&](auto v, auto j) {
    constexpr int V = decltype(v)::value, JJ = decltype(j)::value;
    const auto go = [&](auto sig) {
      constexpr bool SIG = decltype(sig)::value;
      if (a.bf16_grad)
        hipLaunchKernelGGL((balance_grad_kernel<bf16, SIG, V, JJ>), dim3(grid), dim3(kThreadsB), 0, s, a, r.G, rows);
      else
        hipLaunchKernelGGL((balance_grad_kernel<float, SIG, V, JJ>), dim3(grid), dim3(kThreadsB), 0, s, a, r.G, rows);
    };
    if (a.sigmoid) go(std::true_type());
    else go(std::false_type());
  });
  return hipGetLastError();
}

}  // namespace mok
