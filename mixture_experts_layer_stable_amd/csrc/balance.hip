// Balance loss of the router: scores, per-expert counts and sums over ragged segments, and the
// gradient by the logits.
//
// Forward, two launches: (1) a workgroup takes a chunk of consecutive tokens; a group of G lanes
// holds one token's logits in registers (one read, the next token's on their way), forms its
// scores and adds them to the lanes' own per-expert sums; slots are counted with integer LDS
// atomics; where a segment ends inside the chunk the sums are written out as the partial row of
// (chunk, segment). (2) one workgroup per (64 experts, segment), or per 16 where a segment has many
// partial rows, adds the segment's partial rows; the last of them, by a count on one word (13 ns a
// workgroup: 60000 segments take 0.8 ms), adds the parts of the loss. Small batches take one launch
// of one workgroup for all of it (kBalanceSmall). No float atomics: the sums depend on T, E and the
// segments only. Bound by its loads (131072 x 256: 45 us, 3.1 TB/s, and 11 for the 16 workgroups of the
// second launch); for small batches by the launches, for short segments by the walk over a chunk's.
// Backward: one launch, one read of the logits and one write of their gradient.
#include <cmath>

#include "api.h"
#include "block.h"

namespace mok {

namespace {

constexpr int kThreadsB = 256;
// Four workgroups per CU, as long as a chunk keeps 16 rows (T = 16384, E = 384, 37 segments: 64 rows
// 51.8 us, 32 rows 46, 16 rows 43.9) and one for each group of lanes.
constexpr int kBalanceChunks = 1024, kBalanceRows = 16;
// One workgroup for the whole batch: up to 2^14 logits of one segment (E = 8, us against two launches: 64
// tokens 9.6, 11.5; 2048 tokens 11.7, 12.5). It walks its segments one after the other, 3 to 6 us each, as
// does the workgroup of each chunk: a batch of one chunk gains the launch up to four of them (64 tokens, E = 8, 4
// segments: 23.9, 26.0; 16: 81, 79), a batch of more chunks nothing (2048 tokens, E = 8, 2 segments: 16.1,
// 13.5; 256 tokens, E = 64, 64 segments: 415, 103).
constexpr int64_t kBalanceSmall = 1 << 14;
constexpr int kBalanceSmallSegs = 4;
constexpr int kSegExperts = 16;  // of a workgroup of the second launch, at least

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

// exp(x) by the hardware's exp2: off by |x| 2^-24 of its value and a step, so by 2^-20 for the
// scores down to e^-16 that a sum of them in fp32 can see. The library's expf, to half a step over
// every range, made these kernels vector-ALU bound (131072 x 256 sigmoid forward 96 us).
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

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
  } else if (m >= 0.0f) {  // with a logit above 0 the factor is 1 (and a sig below 2^-126 is 0 beside it)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float e = exp_neg(-z[i]), d = __builtin_amdgcn_rcpf(1.0f + e);
      if constexpr (SLOPE) slope[i] = fminf(e, 3e38f) * d;  // an infinite e has d = 0
      z[i] = d;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float e = exp_neg(-fabsf(z[i])), d = __builtin_amdgcn_rcpf(1.0f + e);
      if constexpr (SLOPE) slope[i] = d;
      z[i] = exp_neg(z[i] - m) * d;
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

// The same for a wave-uniform t, all lanes calling: 64 segment ends are looked at together, so 64
// segments take one load's latency and 65535 three.
__device__ __forceinline__ int seg_of_wave(const BalanceArgs& a, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.S;  // the answer lies in lo .. hi
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64, i = lo + (lane + 1) * step;  // segments below i
    const bool past = i <= hi && seg_at(a, i) <= t;                    // all of those end by t
    const int n = __popcll(__ballot(past));
    hi = min(hi, lo + (n + 1) * step - 1);
    lo += n * step;
  }
  return lo;
}

// The loss from the sums over threads of l, its segments' parts, of z, lse^2, of n, counted tokens,
// and of full, segments with some.
template <int NT>
__device__ void finish_loss(const BalanceArgs& a, double l, double z, double n, double full) {
  __shared__ double s_w[NT / 64][4];
  for (int o = 1; o < 64; o <<= 1) {
    l += __shfl_xor(l, o);
    z += __shfl_xor(z, o);
    n += __shfl_xor(n, o);
    full += __shfl_xor(full, o);
  }
  if ((threadIdx.x & 63) == 0) {
    double* w = s_w[threadIdx.x >> 6];
    w[0] = l;
    w[1] = z;
    w[2] = n;
    w[3] = full;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  l = z = n = full = 0.0;
  for (int i = 0; i < NT / 64; ++i) {
    l += s_w[i][0];
    z += s_w[i][1];
    n += s_w[i][2];
    full += s_w[i][3];
  }
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
  __shared__ float s_z[NW];
  const int tid = threadIdx.x, g = tid / G, l = tid - g * G, groups = NT / G;
  const int64_t c0 = ALL ? 0 : (int64_t)blockIdx.x * a.rows, c1 = ALL ? a.T : min(a.T, c0 + a.rows);
  float zsum = 0.0f;
  double loss = 0.0, all_n = 0.0, all_full = 0.0;
  if (!ALL && blockIdx.x == 0 && tid == 0) *a.done = 0;
  // The token that this group has on its way and its logits: loaded before anything is known of
  // segments and mask (a token that does not count is dropped later), so that one latency covers
  // the search, the mask and the logits.
  float zn[NV];
  int64_t tn = c0 + g;
  const auto fetch = [&](int64_t t, int64_t end) {
    tn = t < end ? t : -1;
    if (t < end) load_row<VEC, J>(a.logits + t * a.E, a.E, l, G, -INFINITY, zn);
  };
  fetch(tn, c1);
  for (int s = ALL ? 0 : seg_of_wave(a, c0); s < a.S; ++s) {
    const int64_t s0 = seg_at(a, s), s1 = seg_at(a, s + 1);
    if (!ALL && s0 >= c1) break;
    const int64_t t0 = max(s0, c0), t1 = min(s1, c1);
    if (!ALL && t1 <= t0) {  // one of a run of empty segments, maybe: on with the one that holds token t0
      s = max(s, seg_of_wave(a, t0) - 1);
      continue;
    }
    if (tn != t0 + g) fetch(t0 + g, t1);
    bool on = t0 + g < t1 && (a.mask == nullptr || a.mask[t0 + g] != 0);
    for (int e = tid; e < a.E; e += NT) s_c[e] = 0;
    if (tid == 0) s_n = 0;
    __syncthreads();
    // slots
    int n = 0;
    const uint32_t slots = (uint32_t)(t1 - t0) * (uint32_t)a.k;  // a thread a slot: one latency for 256 of them
    for (uint32_t i = tid; t1 > t0 && i < slots; i += NT) {
      const uint32_t u = i / (uint32_t)a.k;
      const int e = a.idx[t0 * a.k + i];
      const bool counted = a.mask == nullptr || a.mask[t0 + u] != 0;
      if (counted && e >= 0 && e < a.E) atomicAdd(&s_c[e], 1);
      n += counted && u * (uint32_t)a.k == i;
    }
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    if ((tid & 63) == 0 && n != 0) atomicAdd(&s_n, n);
    // scores
    float q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = 0.0f;
    for (int64_t b = t0; b < t1; b += groups) {
      const int64_t t = b + g;
      const bool cur = on;
      float z[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] = cur ? zn[i] : 0.0f;
      fetch(t + groups, t1);
      on = t + groups < t1 && (a.mask == nullptr || a.mask[t + groups] != 0);
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
      std::conditional_t<ALL, double, float> v = 0;  // ALL: the waves' sums are the partial rows
#pragma unroll
      for (int i = 0; i < NW; ++i) v += s_q[i * a.E + e];
      if constexpr (ALL) {
        a.counts[(int64_t)s * a.E + e] = s_c[e];
        a.prob[(int64_t)s * a.E + e] = ns > 0 ? (float)(v / ns) : 0.0f;
        if (ns > 0) loss += (double)s_c[e] * v * ((double)a.E / ((double)a.k * ns * ns));
      } else {
        const int64_t at = (int64_t)blockIdx.x + s;
        a.wq[at * a.E + e] = v;
        a.wc[at * a.E + e] = s_c[e];
      }
    }
    if (tid == 0) {
      if constexpr (ALL) {
        a.tokens[s] = ns;
        all_n += ns;
        all_full += ns > 0;
      } else {
        a.wn[(int64_t)blockIdx.x + s] = ns;
      }
    }
    __syncthreads();
  }
  if constexpr (ALL) {
    finish_loss<NT>(a, loss, zsum, all_n, all_full);
  } else {
    zsum = lanes_sum(zsum, 64);
    if ((tid & 63) == 0) s_z[tid >> 6] = zsum;
    __syncthreads();
    if (tid == 0) {
      float v = 0.0f;
      for (int i = 0; i < NW; ++i) v += s_z[i];
      a.wz[blockIdx.x] = v;
    }
  }
}

// Workgroup (X experts, segment): thread (row lane, expert) adds every (NT / X)th partial row of the
// segment, then the row lanes are added in order.
template <int NT, int X>
__global__ __launch_bounds__(NT) void balance_seg_kernel(BalanceArgs a) {
  constexpr int R = NT / X;
  __shared__ double s_q[R][X];
  __shared__ int s_c[R][X];
  __shared__ int s_n[NT / 64];
  __shared__ bool s_last;
  const int tid = threadIdx.x, x = tid % X, r = tid / X, e = blockIdx.x * X + x, s = blockIdx.y;
  const int64_t s0 = seg_at(a, s), s1 = seg_at(a, s + 1);
  const int lo = (int)(s0 / a.rows), hi = s1 > s0 ? (int)((s1 - 1) / a.rows) + 1 : lo;
  double q = 0.0;
  int c = 0, n = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int i = lo + r; i < hi; i += R) {
      const int64_t at = ((int64_t)i + s) * a.E + e;
      q += (double)a.wq[at];
      c += a.wc[at];
    }
  }
  for (int i = lo + tid; i < hi; i += NT) n += a.wn[i + s];
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
  s_q[r][x] = q;
  s_c[r][x] = c;
  if ((tid & 63) == 0) s_n[tid >> 6] = n;
  __syncthreads();
  if (tid < 64) {
    q = 0.0;
    c = n = 0;
    if (tid < X) {
      for (int i = 0; i < R; ++i) {
        q += s_q[i][x];
        c += s_c[i][x];
      }
    }
    for (int i = 0; i < NT / 64; ++i) n += s_n[i];
    double part = 0.0;
    if (tid < X && e < a.E) {
      a.counts[(int64_t)s * a.E + e] = c;
      a.prob[(int64_t)s * a.E + e] = n > 0 ? (float)(q / n) : 0.0f;
      if (n > 0) part = (double)c * q * ((double)a.E / ((double)a.k * n * n));
    }
    for (int o = 1; o < 64; o <<= 1) part += __shfl_xor(part, o);
    if (tid == 0) {
      __hip_atomic_store(a.wl + (int64_t)s * gridDim.x + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (blockIdx.x == 0) __hip_atomic_store(a.tokens + s, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // Both stores go past the XCD's L2 and have arrived before this workgroup is counted; the last
      // one counted reads them all past its L2. (A release would write the whole L2 back.)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const int parts = gridDim.x * gridDim.y;
      s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  double l = 0.0, z = 0.0, nn = 0.0, full = 0.0;
  for (int i = tid; i < (int)(gridDim.x * gridDim.y); i += NT)
    l += __hip_atomic_load(a.wl + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < a.chunks; i += NT) z += (double)a.wz[i];
  for (int i = tid; i < a.S; i += NT) {
    const int t = __hip_atomic_load(a.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    nn += t;
    full += t > 0;
  }
  finish_loss<NT>(a, l, z, nn, full);
}

template <typename TO, bool SIG, int VEC, int J>
__global__ __launch_bounds__(kThreadsB) void balance_grad_kernel(BalanceArgs a, int G, int64_t rows) {
  constexpr int NV = VEC * J;
  const int tid = threadIdx.x, g = tid / G, l = tid - g * G, groups = kThreadsB / G;
  const int64_t c0 = (int64_t)blockIdx.x * rows, c1 = min(a.T, c0 + rows);
  const int full = a.tokens[a.S], N = a.tokens[a.S + 1];
  const float gz = N > 0 && a.zcoef != 0.0f ? a.dloss[1] * a.zcoef * 2.0f / (float)N : 0.0f;
  float zn[NV], stn = 0.0f;  // logits and stat of the next token, on their way
  uint8_t mn = 1;
  const auto fetch = [&](int64_t t) {
    if (t >= c1) return;
    load_row<VEC, J>(a.logits + t * a.E, a.E, l, G, -INFINITY, zn);
    stn = a.stat[t];
    if (a.mask != nullptr) mn = a.mask[t];
  };
  fetch(c0 + g);
  int s = seg_of_wave(a, c0);
  int64_t s0 = s < a.S ? seg_at(a, s) : a.T, s1 = s < a.S ? seg_at(a, s + 1) : a.T;
  float c[NV], gs = 0.0f;  // counts of segment `have`
  int have = -1;
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = 0.0f;
  for (int64_t t = c0 + g; t < c1; t += groups) {
    float z[NV];
    const float st = stn;
    const bool counted = mn != 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] = zn[i];
    fetch(t + groups);
    if (t >= s1 && s < a.S) {
      s = s + 1 < a.S && t < seg_at(a, s + 2) ? s + 1 : seg_of(a, t);
      s0 = s < a.S ? seg_at(a, s) : a.T;
      s1 = s < a.S ? seg_at(a, s + 1) : a.T;
    }
    const bool on = s < a.S && t >= s0 && counted;
    if (on && have != s) {
      have = s;
      const float n = (float)a.tokens[s];
      gs = n > 0.0f ? a.dloss[0] * a.coef * (float)a.E / ((float)full * (float)a.k * n * n) : 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const int e = (l + j * G) * VEC + v;
          c[j * VEC + v] = e < a.E ? (float)a.counts[(int64_t)s * a.E + e] : 0.0f;
        }
    }
    if (!on) {
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] = 0.0f;
    } else {
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
  w.rows = (int)std::max<int64_t>(std::max(kBalanceRows, kThreadsB / row_shape(E).G), (T + kBalanceChunks - 1) / kBalanceChunks);
  w.chunks = (int)std::max<int64_t>(1, (T + w.rows - 1) / w.rows);
  const size_t pairs = (size_t)w.chunks + S;
  size_t o = 0;
  w.q = o; o = up(o + 4 * pairs * E);
  w.c = o; o = up(o + 4 * pairs * E);
  w.n = o; o = up(o + 4 * pairs);
  w.z = o; o = up(o + 4 * (size_t)w.chunks);
  w.done = o; o = up(o + 4);
  w.loss = o; o = up(o + 8 * (size_t)S * ((E + kSegExperts - 1) / kSegExperts));
  w.bytes = o;
  return w;
}

hipError_t launch_balance_fwd(const BalanceArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.E);
  const bool all = a.T * a.E <= kBalanceSmall && a.S <= (a.chunks == 1 ? kBalanceSmallSegs : 1);
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
  if (!all) {
    // Many partial rows a segment: 64 row lanes, else 4 and fewer workgroups, which are counted on
    // one address (37 segments, E = 384: 888 workgroups 16 us, 222 7 us).
    if (a.chunks >= 64 * a.S)
      hipLaunchKernelGGL((balance_seg_kernel<1024, kSegExperts>), dim3((a.E + kSegExperts - 1) / kSegExperts, a.S),
                         dim3(1024), 0, s, a);
    else
      hipLaunchKernelGGL((balance_seg_kernel<256, 64>), dim3((a.E + 63) / 64, a.S), dim3(256), 0, s, a);
  }
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
