// Softmax statistic of a set of logits kept as (largest logit m, sum of 2^((x - m) c)),
// c = log2(e) / T.
//
// The forward passes of rowpass_fwd.cuh keep the offset m c instead, which saves one packed
// multiply per pair and overflows past |x / T| = 2^30.  The operators here meet logits that a
// mask set to the type's lowest value: the difference x - m is taken first, so every finite
// logit is right, alone in its row or not.  An empty set has m = -FLT_MAX and s = 0 (so that
// x - m is -inf, not NaN, for x = -inf).
#pragma once

#include <cfloat>

#include "rowpass_common.cuh"

namespace grpo {

struct MaxStat {
  float m, s;
};

struct MaxRun {
  float m = -FLT_MAX;
  float2 s = make_float2(0.f, 0.f);
  __device__ __forceinline__ MaxStat stat() const { return MaxStat{m, s.x + s.y}; }
};

__device__ __forceinline__ void maxrun_raise(MaxRun& r, float m, float c) {
  if (m > r.m) {
    const float e = ex2((r.m - m) * c);
    r.s = __fmul2_rn(make_float2(e, e), r.s);
    r.m = m;
  }
}

__device__ __forceinline__ void maxrun_scalar(MaxRun& r, float x, float c) {
  maxrun_raise(r, x, c);
  r.s.x += ex2((x - r.m) * c);
}

template <class E, int N>
__device__ __forceinline__ void maxrun_sum(MaxRun& r, const uint4 (&v)[N], float c) {
  const float2 c2 = make_float2(c, c), nm = make_float2(-r.m, -r.m);
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int i = 0; i < E::kPairs; ++i) {
      const float2 t = __fmul2_rn(__fadd2_rn(E::pair(v[k], i), nm), c2);
      r.s = __fadd2_rn(r.s, make_float2(ex2(t.x), ex2(t.y)));
    }
}

// Largest element of the vectors' even and of their odd places (NaN loses against a number).
template <int N>
__device__ __forceinline__ float2 pair_max(const uint4 (&v)[N], BF16*) {
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v[k]);
    m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
  }
  return make_float2(__low2float(m), __high2float(m));
}
template <int N>
__device__ __forceinline__ float2 pair_max(const uint4 (&v)[N], F32*) {
  float2 m = make_float2(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
#pragma unroll
  for (int k = 0; k < N; ++k) {
    m.x = fmaxf(m.x, fmaxf(__uint_as_float(v[k].x), __uint_as_float(v[k].z)));
    m.y = fmaxf(m.y, fmaxf(__uint_as_float(v[k].y), __uint_as_float(v[k].w)));
  }
  return m;
}

// Fold vectors in; returns pair_max of them.
template <class E, int N>
__device__ __forceinline__ float2 maxrun_vectors(MaxRun& r, const uint4 (&v)[N], float c) {
  const float2 m = pair_max(v, static_cast<E*>(nullptr));
  maxrun_raise(r, fmaxf(m.x, m.y), c);
  maxrun_sum<E, N>(r, v, c);
  return m;
}

__device__ __forceinline__ MaxStat maxstat_warp(MaxStat v, float c) {
  float m = v.s == 0.f ? -FLT_MAX : v.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  v.s *= ex2((v.m - m) * c);
  v.m = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.s += __shfl_xor_sync(0xFFFFFFFFu, v.s, o);
  return v;
}

// The CTA's statistic, in every lane of warp 0.  One barrier; `sh` is read after it.
template <int THREADS>
__device__ __forceinline__ MaxStat maxstat_block(MaxStat v, float c) {
  constexpr int kWarps = THREADS / 32;
  v = maxstat_warp(v, c);
  if (kWarps == 1) return v;
  __shared__ MaxStat sh[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = lane < kWarps ? sh[lane] : MaxStat{-FLT_MAX, 0.f};
    v = maxstat_warp(v, c);
  }
  return v;
}

}  // namespace grpo
