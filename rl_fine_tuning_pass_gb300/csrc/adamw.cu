// AdamW over many tensors in one launch, states in 32 or in 8 bits.
//
//   g' = g coef             coef = max_norm / norm where norm > max_norm, else 1
//   m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   p' = p - (lr wd p + lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps))
//
// Moments in fp32: products and sums rounded one by one, so that a state in 8 bits is a function of
// its inputs and not of how the compiler contracts.  The parameter is updated in fp32 from its master
// copy, if it has one, and rounded once to its type: to nearest, or with `stochastic` and without
// a master copy up or down with the probability that keeps its expectation (a bf16 parameter would
// not move under updates of less than 2^-9 of it).
//
// 8-bit states: blocks of 256 elements share two fp32 scales.  The first moment is a signed code with
// four bits of exponent and three of mantissa; the second moment is held as its root r = sqrt(v),
// which needs half the range, in an unsigned code with four bits of each:
//   m = scale_m (-1)^s (code << 20 as fp32) 2^120,     r = scale_r (code << 19 as fp32) 2^112
// where the scales put a block's largest at the codes' top (448 and 1.9375).  With `stochastic` r
// is rounded by 16 random bits: it changes by 0.05 % a step, which rounding to nearest would lose
// each time.  No r but 0 becomes 0: m / (sqrt(v) + eps) could not stand that.
//
// Floor: 10 bytes a parameter with 8-bit states (bf16 parameters and gradients), 28 with 32-bit ones
// (fp32).  The table of tensors is a kernel parameter; a CTA takes a run of chunks of 2048 elements, eight
// blocks, of one tensor.  Measured: 300M fp32 parameters, norm included, 1.41 ms, and 156M bf16 ones with
// fp32 gradients and master copies 0.68 ms: both the copy rate.  With 8-bit states see update().
#include <algorithm>
#include <cmath>
#include <cuda_fp16.h>

#include "many_tensors.cuh"

namespace grpo {
namespace {

constexpr int kAdamwThreads = 256, kAdamwPer = 8;
constexpr int64_t kAdamwChunk = kAdamwThreads * kAdamwPer;
// Three CTAs an SM (80 registers): 600M bf16 with 8-bit states, norm and moments included, took 2.44 ms then,
// 2.60 with two; four and five leave no registers for the loads ahead (2.29 and 2.24 ms against 2.21).
constexpr int kAdamwCtasPerSm = 3;
constexpr float kTiny = 0x1p-100f;  // a block whose largest is below is stored as zeros

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// What a CTA needs of the scalars, worked out by its first thread.
struct Step {
  float lr, alpha, root, coef;  // lr, lr / (1 - b1^t), 1 / sqrt(1 - b2^t), clipping
  uint32_t key;                 // of the step's random bits
  bool skip;                    // a norm that is not finite: nothing is changed
  int64_t step;                 // the state after it
  double pow1, pow2;
};

__device__ __forceinline__ Step begin_step(const AdamwScalars& s) {
  Step q;
  const AdamwState* st = s.state;
  const int64_t step = *reinterpret_cast<const volatile int64_t*>(&st->step);
  const double p1 = step == 0 ? 1.0 : *reinterpret_cast<const volatile double*>(&st->beta1_pow);
  const double p2 = step == 0 ? 1.0 : *reinterpret_cast<const volatile double*>(&st->beta2_pow);
  const float norm = s.norm ? *s.norm : 0.f;
  q.step = step + 1;
  q.pow1 = p1 * s.beta1;
  q.pow2 = p2 * s.beta2;
  q.lr = s.lr_dev ? *s.lr_dev : static_cast<float>(s.lr);
  q.alpha = q.lr / static_cast<float>(1.0 - q.pow1);
  q.root = 1.f / sqrtf(static_cast<float>(1.0 - q.pow2));
  q.coef = norm > s.max_norm ? __fdiv_rn(s.max_norm, norm) : 1.f;
  q.skip = !(norm <= 3.4028235e38f);
  uint32_t k = mix(s.seed_lo + 0x9E3779B9u);
  k = mix(k ^ s.seed_hi);
  q.key = mix(k ^ static_cast<uint32_t>(q.step));
  return q;
}

// In the call's last launch: every CTA takes a ticket after it has read the state, so the one that
// takes the last ticket may write it; the ticket is then 0 again.
__device__ __forceinline__ void end_step(const AdamwScalars& s, const Step& q) {
  AdamwState* st = s.state;
  __threadfence();
  if (atomicInc(&st->ticket, gridDim.x - 1) == gridDim.x - 1 && !q.skip) {
    st->beta1_pow = q.pow1;
    st->beta2_pow = q.pow2;
    st->step = q.step;
  }
}

// The update works on four consecutive elements a thread, twice a chunk: element 4 lane + k of a
// warp's first and second 128.  Every access of a warp is then contiguous whatever the type, and a
// warp's chunk is one block.  Raw holds a thread's share as it lies in memory.
enum Source : int { kF32 = 0, kBf16 = 1, kMaster = 2 };  // where the parameter is read from
template <int SRC, bool GRAD_BF16, int BITS>
struct Raw {
  static constexpr int kP = SRC == kBf16 ? 2 : 4, kG = GRAD_BF16 ? 2 : 4, kS = BITS == 8 ? 1 : 4;
  uint32_t p[2][kP], g[2][kG], m[2][kS], v[2][kS];
  uint32_t copy[2][2];  // kMaster: the bf16 parameter, written only
  float2 scale;
};

// A quad's W words (4 elements of W bytes) at p, or its first `left` elements, one by one, and zeros after
// them.  Each byte is touched once a step: streaming accesses.
template <int W, bool FULL>
__device__ __forceinline__ void load_quad(uint32_t (&w)[W], const char* p, int64_t left) {
  if constexpr (FULL) {
    if constexpr (W == 4) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (W == 2) {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = x.x; w[1] = x.y;
    } else {
      w[0] = __ldcs(reinterpret_cast<const unsigned int*>(p));
    }
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= left) break;
      if constexpr (W == 4) w[k] = reinterpret_cast<const uint32_t*>(p)[k];
      else if constexpr (W == 2) w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[k]) << 16 * (k % 2);
      else w[0] |= static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(p)[k]) << 8 * k;
    }
  }
}
template <int W, bool FULL>
__device__ __forceinline__ void store_quad(const uint32_t (&w)[W], char* p, int64_t left) {
  if constexpr (FULL) {
    if constexpr (W == 4) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (W == 2) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    else __stcs(reinterpret_cast<unsigned int*>(p), w[0]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= left) break;
      if constexpr (W == 4) reinterpret_cast<uint32_t*>(p)[k] = w[k];
      else if constexpr (W == 2) reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(w[k / 2] >> 16 * (k % 2));
      else reinterpret_cast<uint8_t*>(p)[k] = static_cast<uint8_t>(w[0] >> 8 * k);
    }
  }
}

// A run of chunks of one tensor: its arrays from the run's first element, the same for the whole CTA,
// so that a thread needs 32-bit offsets only.  left: elements from there to the tensor's end.
struct Run {
  const char* grad;
  char *param, *copy, *exp_avg, *exp_avg_sq;
  float* scale;
  int64_t left;
};

// e: the thread's first element in the run.
template <int SRC, bool GB, int BITS, bool FULL>
__device__ __forceinline__ void load_raw(Raw<SRC, GB, BITS>& x, const Run& a, uint32_t e) {
  using R = Raw<SRC, GB, BITS>;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t i = e + 128u * j;
    const int64_t left = a.left - i;
    load_quad<R::kG, FULL>(x.g[j], a.grad + i * R::kG, left);
    load_quad<R::kS, FULL>(x.m[j], a.exp_avg + i * R::kS, left);
    load_quad<R::kS, FULL>(x.v[j], a.exp_avg_sq + i * R::kS, left);
    load_quad<R::kP, FULL>(x.p[j], a.param + i * R::kP, left);
  }
  if (BITS == 8) {
    const uint32_t block = e / kAdamwBlock;
    x.scale = FULL || static_cast<int64_t>(block) * kAdamwBlock < a.left ? reinterpret_cast<const float2*>(a.scale)[block]
                                                                         : make_float2(0.f, 0.f);
  }
}
// scale (8 bits): in lane 0 the first moment's, in lane 1 the second's.
template <int SRC, bool GB, int BITS, bool FULL>
__device__ __forceinline__ void store_raw(const Raw<SRC, GB, BITS>& x, const Run& a, uint32_t e, float scale) {
  using R = Raw<SRC, GB, BITS>;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t i = e + 128u * j;
    const int64_t left = a.left - i;
    store_quad<R::kS, FULL>(x.m[j], a.exp_avg + i * R::kS, left);
    store_quad<R::kS, FULL>(x.v[j], a.exp_avg_sq + i * R::kS, left);
    store_quad<R::kP, FULL>(x.p[j], a.param + i * R::kP, left);
    if (SRC == kMaster) store_quad<2, FULL>(x.copy[j], a.copy + i * 2u, left);
  }
  if (BITS == 8) {
    const uint32_t lane = threadIdx.x & 31u, block = e / kAdamwBlock;
    if (lane < 2 && (FULL || static_cast<int64_t>(block) * kAdamwBlock < a.left)) a.scale[2 * block + lane] = scale;
  }
}

template <int W>
__device__ __forceinline__ float2 pair_of(const uint32_t (&w)[W], int h) {
  if constexpr (W == 4) return make_float2(__uint_as_float(w[2 * h]), __uint_as_float(w[2 * h + 1]));
  else return make_float2(BF16::lo(w[h]), BF16::hi(w[h]));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// The sum of two packed products, each rounded: added one by one, for a packed sum is fused with the
// product before it, however it is written (every fourth sum came out an ulp off).
__device__ __forceinline__ float2 add_rounded(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Two values to bf16, each up or down by sixteen of `bits` (x's the lower ones): they are added below
// the bits that stay.
__device__ __forceinline__ uint32_t stochastic_pair(float2 x, uint32_t bits) {
  uint32_t d;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(d) : "f"(x.y), "f"(x.x), "r"(bits));
  return d;
}
// The signed codes are those of e4m3: values of codes 2h and 2h + 1 of a quad's word, and back.
__device__ __forceinline__ float2 values_m(uint32_t w, int h) {
  const uint16_t two = static_cast<uint16_t>(h == 0 ? w : w >> 16);
  uint32_t half2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&half2));
}
__device__ __forceinline__ uint32_t codes_m(float2 x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(x.y), "f"(x.x));
  return d;
}
// The unsigned code k of a quad's word as the upper bits of an fp32 number: its value times 2^-112.
__device__ __forceinline__ float bits_r(uint32_t w, int k) {
  return __uint_as_float((k < 3 ? w << (19 - 8 * k) : w >> 5) & 0x07F80000u);
}

// The rounded root of v in [2^-100, inf): with y near 1 / sqrt(v) and a = v y, the residual v - a^2 comes
// out of one FMA, and a + (v - a^2) y / 2 rounds to the root (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990; compared with the rounded root over all
// fp32 numbers of [1, 4) and of four more pairs of octaves: no difference).
__device__ __forceinline__ float2 roots(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  const float2 a = __fmul2_rn(v, y), h = __fmul2_rn(y, both(0.5f));
  return __ffma2_rn(__ffma2_rn(__fmul2_rn(a, both(-1.f)), a, v), h, a);
}

// max(|a|, |b|, |c|), NaN if one is; min(a, b, c)
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min_of(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float reciprocal_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One thread's eight elements; pair0: the first one's pair in the tensor (the second four are 128 further).
// Returns the block's scale that lane 0 or 1 stores.  With 8-bit states this is bound by instructions:
// 60 an element of a bf16 parameter, stochastically rounded, take 208 us for 100M of them where
// the memory would take 148 (81 before the roots and conversions above, and 266 us).
template <int SRC, bool GB, int BITS>
__device__ __forceinline__ float update(Raw<SRC, GB, BITS>& x, const AdamwScalars& s, const Step& q, float decay,
                                        uint32_t key, uint32_t pair0) {
  float2 m[4], r[4], v[4];
  // a code's bits times 2^112 and the scale, in one product (exact powers of two apart) where that is
  // an fp32 number
  const bool wide = BITS == 8 && !(x.scale.y < 0x1p15f);
  const float up_r = x.scale.y * (wide ? 0x1p60f : 0x1p112f);  // a root is below 2^64
  const bool dither_p = SRC == kBf16 && s.stochastic != 0, dither_r = BITS == 8 && s.stochastic != 0;
  uint32_t w[4];
  if (dither_p || dither_r)
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = mix(pair0 + (e >> 1) * 64 + (e & 1) + key);
#pragma unroll
  for (int e = 0; e < 4; ++e) {  // pairs
    const int j = e >> 1, h = e & 1;
    const float2 g = __fmul2_rn(pair_of(x.g[j], h), both(q.coef));
    if constexpr (BITS == 8) {
      m[e] = __fmul2_rn(values_m(x.m[j][0], h), both(x.scale.x));
      float2 old = __fmul2_rn(make_float2(bits_r(x.v[j][0], 2 * h), bits_r(x.v[j][0], 2 * h + 1)), both(up_r));
      if (wide) old = __fmul2_rn(old, both(0x1p52f));
      v[e] = __fmul2_rn(old, old);
    } else {
      m[e] = pair_of(x.m[j], h);
      v[e] = pair_of(x.v[j], h);
    }
    m[e] = add_rounded(__fmul2_rn(m[e], both(s.b1)), __fmul2_rn(g, both(s.w1)));
    v[e] = add_rounded(__fmul2_rn(v[e], both(s.b2)), __fmul2_rn(__fmul2_rn(g, g), both(s.w2)));
  }
  float top_m = 0.f, top_r = 0.f;
  bool zeros = false;  // v outside the range of roots(): zero, next to nothing, or not finite
  if constexpr (BITS == 8) {
    float low = 1.f, high = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      low = min_of(low, v[e].x, v[e].y);
      high = max_abs(high, v[e].x, v[e].y);
      top_m = max_abs(top_m, m[e].x, m[e].y);
      r[e] = roots(v[e]);
    }
    zeros = !(low >= 0x1p-100f && high <= 3.4028235e38f);
    if (zeros)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = make_float2(__fsqrt_rn(v[e].x), __fsqrt_rn(v[e].y));
#pragma unroll
    for (int e = 0; e < 4; ++e) top_r = max_abs(top_r, r[e].x, r[e].y);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = e >> 1, h = e & 1;
    if constexpr (BITS == 32) {
      // only the update sees this root: the approximation's 2^-22 is far below its roundings' sum
      asm("sqrt.approx.f32 %0, %1;" : "=f"(r[e].x) : "f"(v[e].x));
      asm("sqrt.approx.f32 %0, %1;" : "=f"(r[e].y) : "f"(v[e].y));
      x.m[j][2 * h] = __float_as_uint(m[e].x);
      x.m[j][2 * h + 1] = __float_as_uint(m[e].y);
      x.v[j][2 * h] = __float_as_uint(v[e].x);
      x.v[j][2 * h + 1] = __float_as_uint(v[e].y);
    }
    const float2 den = __ffma2_rn(r[e], both(q.root), both(s.eps));
    const float2 u = __fmul2_rn(m[e], make_float2(reciprocal_near(den.x), reciprocal_near(den.y)));
    float2 p = pair_of(x.p[j], h);
    const float2 t = __ffma2_rn(both(q.alpha), u, __fmul2_rn(both(decay), p));
    p = __ffma2_rn(t, both(-1.f), p);
    if constexpr (SRC != kBf16) {
      x.p[j][2 * h] = __float_as_uint(p.x);
      x.p[j][2 * h + 1] = __float_as_uint(p.y);
      if constexpr (SRC == kMaster) x.copy[j][h] = BF16::pack2(p.x, p.y);
    } else if (dither_p) {
      const uint32_t t16 = w[e] * 0x9E3779B9u;
      x.p[j][h] = stochastic_pair(p, t16 ^ (t16 >> 16));
    } else {
      x.p[j][h] = BF16::pack2(p.x, p.y);
    }
  }
  float scale = 0.f;
  if constexpr (BITS == 8) {
    // the warp's 256 elements are a block; bits of floats of one sign are ordered as they are, NaN last.
    // Even lanes work out the first moment's scale, odd ones the second's.
    const uint32_t all_m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_m));
    const uint32_t all_r = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_r));
    const bool second = (threadIdx.x & 1) != 0;
    const float top = __uint_as_float(second ? all_r : all_m), most = second ? 1.9375f : 448.f;
    const bool tiny = top < kTiny;  // NaN is not
    const float inverse = tiny ? 0.f : __fdiv_rn(most, top);
    scale = tiny ? 0.f : __fmul_rn(top, second ? 1.f / 1.9375f : 1.f / 448.f);
    const float im = __shfl_sync(0xFFFFFFFFu, inverse, 0), ir = __shfl_sync(0xFFFFFFFFu, inverse, 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t cm[2], cr[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 2 * j + h;
        cm[h] = codes_m(__fmul2_rn(m[e], both(im)));
        float2 y = __fmul2_rn(r[e], both(ir));
        // no root but 0 becomes 0: code 1 stands for 2^-18
        if (zeros) {
          y.x = r[e].x > 0.f && ir > 0.f ? fmaxf(y.x, 0x1p-18f) : y.x;
          y.y = r[e].y > 0.f && ir > 0.f ? fmaxf(y.y, 0x1p-18f) : y.y;
        } else {
          y = make_float2(fmaxf(y.x, 0x1p-18f), fmaxf(y.y, 0x1p-18f));
        }
        y = __fmul2_rn(y, both(0x1p-112f));
        const uint32_t u[2] = {__float_as_uint(y.x), __float_as_uint(y.y)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // rounded by what is added below the code's bits before they are cut off
          const uint32_t up = !dither_r ? 0x3FFFFu + ((u[k] >> 19) & 1u) : __byte_perm(w[e], 0u, k ? 0x4432 : 0x4410) << 3;
          cr[2 * h + k] = (u[k] + up) >> 19;
        }
      }
      x.m[j][0] = __byte_perm(cm[0], cm[1], 0x5410);
      x.v[j][0] = __byte_perm(__byte_perm(cr[0], cr[1], 0x0040), __byte_perm(cr[2], cr[3], 0x0040), 0x5410);
    }
  }
  return scale;
}

// Chunks [c0, c1) of one tensor; the next one's loads are under way while one is worked on.
// The first chunk's are before the step's scalars are there, which thread 0 works out meanwhile.
template <int SRC, bool GB, int BITS>
__device__ __forceinline__ void update_run(const AdamwTensor& t, const AdamwScalars& s, Step& shared_step, bool advance,
                                           uint32_t c0, uint32_t c1) {
  using R = Raw<SRC, GB, BITS>;
  const int64_t begin = static_cast<int64_t>(c0) * kAdamwChunk;
  Run a;
  a.grad = static_cast<const char*>(t.grad) + begin * R::kG;
  a.param = (SRC == kMaster ? reinterpret_cast<char*>(t.master) : static_cast<char*>(t.param)) + begin * R::kP;
  a.copy = SRC == kMaster ? static_cast<char*>(t.param) + begin * 2 : nullptr;
  a.exp_avg = static_cast<char*>(t.exp_avg) + begin * R::kS;
  a.exp_avg_sq = static_cast<char*>(t.exp_avg_sq) + begin * R::kS;
  a.scale = BITS == 8 ? reinterpret_cast<float*>(t.scale) + begin / kAdamwBlock * 2 : nullptr;
  a.left = t.n - begin;
  uint32_t e = (threadIdx.x >> 5) * kAdamwBlock + (threadIdx.x & 31) * 4;
  // the upper half of a pair's index goes into the key, which so changes with every 2^22nd chunk
  constexpr uint32_t kKeyChunks = (1u << 22) - 1;
  static_assert(kAdamwChunk << 22 == int64_t(1) << 33, "pairs of one key");
  uint32_t pair = static_cast<uint32_t>(begin >> 1) + (e >> 1);
  // whole chunks by vectors; an odd end, and tensors that are not aligned, element by element
  const uint32_t whole = t.aligned ? static_cast<uint32_t>(t.n / kAdamwChunk) : 0u;
  const uint32_t fast = whole < c0 ? c0 : (whole < c1 ? whole : c1);
  R next;
  if (c0 < fast) load_raw<SRC, GB, BITS, true>(next, a, e);
  if (threadIdx.x == 0) shared_step = begin_step(s);
  __syncthreads();
  const Step q = shared_step;
  if (threadIdx.x == 0 && advance) end_step(s, q);
  if (q.skip) return;
  const float decay = q.lr * t.weight_decay;
  const uint32_t tensor_key = mix(q.key + t.ordinal);
  uint32_t key = mix(tensor_key ^ (c0 >> 22));
  for (uint32_t c = c0; c < fast; ++c, e += kAdamwChunk, pair += kAdamwChunk / 2) {
    R x = next;
    if ((c & kKeyChunks) == 0) key = mix(tensor_key ^ (c >> 22));
    if (c + 1 < fast) load_raw<SRC, GB, BITS, true>(next, a, e + kAdamwChunk);
    const float scale = update<SRC, GB, BITS>(x, s, q, decay, key, pair);
    store_raw<SRC, GB, BITS, true>(x, a, e, scale);
  }
  for (uint32_t c = fast; c < c1; ++c, e += kAdamwChunk, pair += kAdamwChunk / 2) {
    R x;
    if ((c & kKeyChunks) == 0) key = mix(tensor_key ^ (c >> 22));
    load_raw<SRC, GB, BITS, false>(x, a, e);
    const float scale = update<SRC, GB, BITS>(x, s, q, decay, key, pair);
    store_raw<SRC, GB, BITS, false>(x, a, e, scale);
  }
}

// A CTA's work is `run` chunks of a tensor.
template <int N, int SRC, bool GB, int BITS>
__global__ void __launch_bounds__(kAdamwThreads, kAdamwCtasPerSm)
    adamw_kernel(const __grid_constant__ AdamwTable<N> tab, const __grid_constant__ AdamwScalars s, uint32_t run,
                 bool advance) {
  wait_for_previous_grids();
  __shared__ Step shared_step;
  if (tab.items == 0) {  // nothing to update: a step all the same
    if (threadIdx.x == 0 && advance) end_step(s, begin_step(s));
    return;
  }
  const int t = tensor_of_chunk(tab, blockIdx.x, 0);
  const AdamwTensor& a = tab.t[t];
  const uint32_t chunks = static_cast<uint32_t>((a.n + kAdamwChunk - 1) / kAdamwChunk);
  const uint32_t c0 = (blockIdx.x - tab.first[t]) * run;
  update_run<SRC, GB, BITS>(a, s, shared_step, advance, c0, min(c0 + run, chunks));
}

// The moments that 8-bit states stand for: m, and v = r^2.  Sixteen elements a thread, in four quads that
// are loaded together; a CTA takes 4096.
constexpr int kMomentQuads = 4;
__global__ void __launch_bounds__(kAdamwThreads)
    moments_kernel(const char* exp_avg, const char* exp_avg_sq, const float2* scale, int64_t n, char* m, char* v,
                   bool aligned) {
  wait_for_previous_grids();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kMomentQuads * 4 * kAdamwThreads);
  const bool full = aligned && first + kMomentQuads * 4 * kAdamwThreads <= n;
  uint32_t cm[kMomentQuads][1], cr[kMomentQuads][1];
  float2 sc[kMomentQuads];
#pragma unroll
  for (int q = 0; q < kMomentQuads; ++q) {
    const int64_t i = first + (q * kAdamwThreads + threadIdx.x) * 4;
    if (full) {
      load_quad<1, true>(cm[q], exp_avg + i, 4);
      load_quad<1, true>(cr[q], exp_avg_sq + i, 4);
    } else {
      load_quad<1, false>(cm[q], exp_avg + i, n - i);
      load_quad<1, false>(cr[q], exp_avg_sq + i, n - i);
    }
    sc[q] = full || i < n ? scale[i / kAdamwBlock] : make_float2(0.f, 0.f);
  }
#pragma unroll
  for (int q = 0; q < kMomentQuads; ++q) {
    const int64_t i = first + (q * kAdamwThreads + threadIdx.x) * 4;
    uint32_t om[4], ov[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 mv = __fmul2_rn(values_m(cm[q][0], h), both(sc[q].x));
      const float2 r = __fmul2_rn(__fmul2_rn(make_float2(bits_r(cr[q][0], 2 * h), bits_r(cr[q][0], 2 * h + 1)),
                                             both(0x1p112f)), both(sc[q].y));
      const float2 vv = __fmul2_rn(r, r);
      om[2 * h] = __float_as_uint(mv.x);
      om[2 * h + 1] = __float_as_uint(mv.y);
      ov[2 * h] = __float_as_uint(vv.x);
      ov[2 * h + 1] = __float_as_uint(vv.y);
    }
    if (full) {
      store_quad<4, true>(om, m + i * 4, 4);
      store_quad<4, true>(ov, v + i * 4, 4);
    } else {
      store_quad<4, false>(om, m + i * 4, n - i);
      store_quad<4, false>(ov, v + i * 4, n - i);
    }
  }
}

struct Part {
  const AdamwTensor* tensors;
  int count;
  uint32_t run;  // chunks a CTA
  bool advance;
};
int64_t chunks_of(const AdamwTensor& t) { return (t.n + kAdamwChunk - 1) / kAdamwChunk; }
int kind_of(const AdamwTensor& t) { return (t.master ? kMaster : t.param_bf16 ? kBf16 : kF32) * 2 + t.grad_bf16; }

template <int N, int SRC, bool GB, int BITS>
cudaError_t launch_table(const Part& p, const AdamwScalars& s, cudaStream_t stream) {
  AdamwTable<N> tab;
  uint32_t items = 0;
  for (int i = 0; i < p.count; ++i) {
    tab.t[i] = p.tensors[i];
    tab.first[i] = items;
    items += static_cast<uint32_t>((chunks_of(p.tensors[i]) + p.run - 1) / p.run);
  }
  tab.count = p.count;
  tab.items = items;
  return launch_after_previous(adamw_kernel<N, SRC, GB, BITS>, dim3(items > 0 ? items : 1), dim3(kAdamwThreads), stream, tab,
                               s, p.run, p.advance);
}
template <int SRC, bool GB>
cudaError_t launch_kind(const Part& p, const AdamwScalars& s, int bits, cudaStream_t stream) {
  if (bits == 8)
    return p.count <= kAdamwFew ? launch_table<kAdamwFew, SRC, GB, 8>(p, s, stream)
                                : launch_table<kAdamwMany, SRC, GB, 8>(p, s, stream);
  return p.count <= kAdamwFew ? launch_table<kAdamwFew, SRC, GB, 32>(p, s, stream)
                              : launch_table<kAdamwMany, SRC, GB, 32>(p, s, stream);
}

}  // namespace

// One launch for each combination of types that occurs (a kernel for all of them would need the
// registers of the largest), and for each kAdamwMany tensors of it.  `tensors` is put in that order.
// A call without elements still makes its step.
cudaError_t launch_adamw(AdamwTensor* tensors, int64_t count, const AdamwScalars& s, int bits, int sms,
                         cudaStream_t stream) {
  const auto before = [](const AdamwTensor& a, const AdamwTensor& b) { return kind_of(a) < kind_of(b); };
  count = std::remove_if(tensors, tensors + count, [](const AdamwTensor& t) { return t.n == 0; }) - tensors;
  if (!std::is_sorted(tensors, tensors + count, before)) std::sort(tensors, tensors + count, before);
  for (int64_t at = 0;;) {
    const int kind = count > 0 ? kind_of(tensors[at]) : 0;
    int64_t end = at, chunks = 0;
    while (end < count && end - at < kAdamwMany && kind_of(tensors[end]) == kind) chunks += chunks_of(tensors[end++]);
    // chunks a CTA: few enough for some sixteen CTAs after one another in each place, which evens out that
    // some SMs are farther from the memory, but four where there are enough of them for every place, so
    // that the step's beginning and the first loads are a small part; at most 64 (which 2^32 chunks, the most
    // that a call may have, come to: 2^26 CTAs)
    const int64_t places = static_cast<int64_t>(sms) * kAdamwCtasPerSm;
    int64_t run = std::max<int64_t>(chunks / (16 * places), std::min<int64_t>(4, chunks / places));
    run = std::min<int64_t>(64, std::max<int64_t>(1, run));
    const Part p{tensors + at, static_cast<int>(end - at), static_cast<uint32_t>(run), end == count};
    cudaError_t e = cudaErrorInvalidValue;
    switch (kind) {
      case kF32 * 2: e = launch_kind<kF32, false>(p, s, bits, stream); break;
      case kF32 * 2 + 1: e = launch_kind<kF32, true>(p, s, bits, stream); break;
      case kBf16 * 2: e = launch_kind<kBf16, false>(p, s, bits, stream); break;
      case kBf16 * 2 + 1: e = launch_kind<kBf16, true>(p, s, bits, stream); break;
      case kMaster * 2: e = launch_kind<kMaster, false>(p, s, bits, stream); break;
      case kMaster * 2 + 1: e = launch_kind<kMaster, true>(p, s, bits, stream); break;
    }
    if (e != cudaSuccess || end == count) return e;
    at = end;
  }
}

cudaError_t launch_adamw_moments(const uint8_t* exp_avg, const uint8_t* exp_avg_sq, const float2* scale, int64_t n,
                                 float* m, float* v, cudaStream_t stream) {
  const auto off = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  const bool aligned = (off(exp_avg) | off(exp_avg_sq)) % 4 == 0 && (off(m) | off(v)) % 16 == 0;
  const int64_t ctas = (n + kMomentQuads * 4 * kAdamwThreads - 1) / (kMomentQuads * 4 * kAdamwThreads);
  return launch_after_previous(moments_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAdamwThreads), stream,
                               reinterpret_cast<const char*>(exp_avg), reinterpret_cast<const char*>(exp_avg_sq), scale, n,
                               reinterpret_cast<char*>(m), reinterpret_cast<char*>(v), aligned);
}

}  // namespace grpo
