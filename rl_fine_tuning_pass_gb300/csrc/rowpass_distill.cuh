// Distillation from a teacher's top log-probs, forward and backward.  Buckets: the listed
// columns i_k with teacher probability q_k, and the rest of the vocabulary (q_rest, 0 when the
// teacher is renormalised over its list); p the student's softmax(x / T) mass of each bucket.
//
//   L = beta KL(q | m) + (1 - beta) KL(p | m),  m = beta q + (1 - beta) p
//   (the limits KL(q | p) at beta = 0 and KL(p | q) at beta = 1)
//   G_b = p_b dL/dp_b,  S = sum_b G_b
//   dL/dx_j = (1 / T) (G_k - p_j S) at j = i_k,  (1 / T) p_j (G_rest / p_rest - S) elsewhere
//
// (any constant added to dL/dp changes nothing, since the p_b sum to 1: below G_b is taken with
// the constant that leaves it near 0 where p_b is near q_b).  So the backward is the softmax stream
// of rowgrad_kernel with one factor per row, and K elements written after it.  p_rest is summed
// from the columns outside the list (a bitmap in shared memory leaves the listed ones out of the
// stream), not taken from 1 - sum p_k: it keeps its relative accuracy when the list holds nearly all
// of the mass.  Where no unlisted column has any (they are all -inf, or there are none), there is
// no rest: the row is taken as without the tail, its teacher renormalised over the list.
// A rest of less mass than fp32's normal numbers hold ("faint": the list is 87 T or more above it) is
// kept as its statistic: its log-ratio comes from log s and the maxima, and the unlisted columns'
// gradient at beta = 0, -g q_rest p_j / p_rest, from 2^((x_j - m_rest) c) / s_rest.  The backward, which
// has p_rest alone, sweeps such a row once more for that statistic (rest_stat).
//
// Bound by HBM: 8192 rows of 151936 bf16, a quarter of them masked, take 281 us forward (6.6 TB/s),
// 667 us backward (6.5 TB/s, reads and writes), 835 us fused.
//
// A CTA takes a row.  Its last warp, the list warp, does not stream: it reads the list, marks the
// bitmap, and works out what the teacher says (with 64-bit exponentials, the rest's mass being
// 1 - sum q_k) while the others stream the row; then it finishes the row from their statistic.
// log-probs of the buckets are formed from differences x_k - max in fp32 with a correction term:
// an error that all buckets share cancels in the loss (below) and in the gradient.
#pragma once

#include "logits_ops.h"
#include "logits_load.cuh"
#include "logits_stat.cuh"
#include "rowpass_fused.cuh"

namespace grpo {
namespace {

constexpr int kBitmapBytes = 32768;      // 262144 columns; beyond, positions wrap and are checked
constexpr double kRestMin = 0x1p-20;     // least teacher mass outside the list
constexpr float kLeastMass = 0x1p-149f;  // p_rest of a rest whose mass underflows: 0 says that there is none

// The list of one row in shared memory.  id -1: an unused slot.
struct Slots {
  int* id;
  float* lq;  // teacher log-prob as given; later G_k
  float* x;   // the student's logit; later p_k
};
__device__ __forceinline__ Slots slots_at(void* at, int K) {
  Slots sl;
  sl.id = static_cast<int*>(at);
  sl.lq = reinterpret_cast<float*>(sl.id + K);
  sl.x = sl.lq + K;
  return sl;
}

// Terms of one bucket: its part of the loss and G.  r = log q - log p, which carries the
// precision where p and q are near each other.  The parts of the loss carry (p - q) or (q - p)
// besides (they sum to nothing over the buckets, `row_loss` takes out what is left): an error of
// r then enters times p - q, so one that all buckets share, such as that of log s, does not count.
// F = G / p (at beta = 0 that of q = 0).
struct Term {
  float loss, G, F;
};
__device__ __forceinline__ Term bucket(float q, float p, float r, float beta) {
  Term t;
  if (beta == 0.f) {
    const bool near = fabsf(r) < 0.5f;
    const float e = expm1f(near ? r : 0.f);
    t.G = near ? -p * e : p - q;  // p (1 - q / p)
    t.F = 1.f;
    t.loss = q == 0.f ? p : (near ? q * (expm1f(-r) + r) : q * r - q + p);
  } else if (beta == 1.f) {
    const bool near = fabsf(r) < 0.5f;
    t.F = -r;
    t.G = p == 0.f ? 0.f : -p * r;
    t.loss = p == 0.f ? q : (near ? p * (expm1f(r) - r) : t.G - p + q);
  } else {
    // log(p/m) and log(q/m) from r alone.  With b the weight of the larger of p and q, and s = |r|:
    // m / larger = 1 + (1 - b)(e^-s - 1), m / smaller = 1 + b (e^s - 1).  For a small b the first has lost
    // b's digits (it is b + (1 - b) e^-s then), and the second gives a log(smaller / m) near 0 its own
    const bool up = r > 0.f;  // q is the larger
    const float s = fabsf(r), b = up ? beta : 1.f - beta, nb = up ? 1.f - beta : beta;
    float large, small;
    if (b >= 0.25f) {
      large = -log1pf(nb * expm1f(-s));
      small = large - s;
    } else {
      const float a = b * expm1f(s);
      small = -log1pf(a);
      large = s + small;
      if (!(a < 1.f)) {
        large = -logf(fmaf(nb, expf(-s), b));
        small = large - s;
      }
    }
    const float lpm = up ? small : large, lqm = up ? large : small;
    t.F = (1.f - beta) * lpm;
    t.G = p == 0.f ? 0.f : (1.f - beta) * p * lpm;
    t.loss = (q == 0.f ? 0.f : beta * q * lqm) + t.G;
  }
  return t;
}
// The loss from the sum of its parts; over = sum q - 1.
__device__ __forceinline__ float row_loss(float parts, float over, float beta) {
  return beta == 0.f ? parts + over : (beta == 1.f ? parts - over : parts);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// d / T as a value and what its rounding left.
struct Scaled {
  float hi, lo;
};
__device__ __forceinline__ Scaled over_T(float d, const DistillParams& p) {
  Scaled z;
  z.hi = d * p.invT;
  z.lo = fabsf(z.hi) < 1e30f ? fmaf(d, p.invT, -z.hi) + d * p.invT_lo : 0.f;  // (-inf has no rounding)
  return z;
}
// e^(d / T), d <= 0 or small
__device__ __forceinline__ float exp_over_T(float d, const DistillParams& p) {
  const Scaled z = over_T(d, p);
  const float e = expf(z.hi);
  return fmaf(e, z.lo, e);
}

// What the teacher's list says (one warp): log q_k = (lq_k - base) - shift (one number for both would
// round a far-shifted list's q_k alike, and their sum with them), the mass of the list and outside it,
// sum q - 1, and (tail) the list's mass once more.
struct Teacher {
  float base, shift, list, rest, over;
  double sum;
  __device__ __forceinline__ float log_q(float lq) const { return (lq - base) - shift; }
};
__device__ __forceinline__ Teacher teacher_of(const Slots& sl, int K, int tail) {
  const int lane = threadIdx.x & 31;
  Teacher t{0.f, 0.f, 1.f, 0.f, 0.f, 1.0};
  if (tail) {
    double sum = 0.0;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) sum += exp(static_cast<double>(sl.lq[k]));
    sum = warp_sum(sum);
    const double left = 1.0 - sum, rest = left < kRestMin ? kRestMin : left;  // a NaN stays one
    t.sum = sum;
    t.list = static_cast<float>(sum);
    t.rest = static_cast<float>(rest);
    t.over = static_cast<float>(rest - left);
  } else {
    float m = -INFINITY;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) m = fmaxf(m, sl.lq[k]);
    m = warp_max(m);
    float sum = 0.f;
    int used = 0;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) {
        sum += expf(sl.lq[k] - m);
        used = 1;
      }
    t.base = m;
    t.shift = logf(warp_sum(sum));
    if (!__any_sync(0xFFFFFFFFu, used)) {  // nothing listed
      t.list = 0.f;
      t.over = -1.f;
    }
  }
  return t;
}

// The same renormalised over the list, for a row without a rest.  A mass below fp32's range counts too:
// log(m 2^e) with e log 2 as a product that is exact in fp32 (log 2 to twelve bits) and what that leaves.
__device__ __forceinline__ Teacher renormalised(double sum) {
  constexpr double kLn2D = 0.69314718055994530942;
  constexpr float kHigh = static_cast<float>(static_cast<int>(kLn2D * 4096.0) / 4096.0);
  constexpr float kLow = static_cast<float>(kLn2D - static_cast<double>(kHigh));
  int e;
  const float m = static_cast<float>(frexp(sum, &e)), n = static_cast<float>(e);
  return Teacher{n * kHigh, fmaf(n, kLow, logf(m)), 1.f, 0.f, 0.f, 1.0};
}

// log(q / p) of the rest, d = q - p
__device__ __forceinline__ float rest_ratio(float q, float p, float d) {
  const float e = d / p;
  return fabsf(e) < 0.5f ? log1pf(e) : logf(q / p);
}
// The same of a faint p = s e^a.
__device__ __forceinline__ float faint_ratio(float q, float s, float a) { return logf(q / s) - a; }

// G / p of the rest.  Below fp32's normal numbers G may be less than they hold; a factor past fp32
// belongs to columns without any mass.
__device__ __forceinline__ float rest_factor(const Term& t, float p) {
  if (p >= FLT_MIN) return t.G / p;
  return fabsf(t.F) <= FLT_MAX ? t.F : 0.f;
}

// The unlisted columns' gradient g F p_j as f 2^((x_j - x0) c), from p_j = 2^((x_j - x0) c) scale.
// Where the factor is large (F is of the order of 1 / p_rest where the student leaves the rest next to
// nothing), its power of two moves into x0: neither f nor the exponentials then leave fp32's range
// before their product does.
struct Stream {
  float f, x0;
};
__device__ __forceinline__ Stream stream_of(float g, float F, float scale, float x0, const DistillParams& p) {
  const float lift = ceilf(log2f(fabsf(F)) + log2f(scale) + log2f(fabsf(g)) + 0.01f);  // leaves |f| <= 1
  if (!(lift > 0.f)) return Stream{g * (F * scale), x0};
  const float x1 = x0 - fminf(lift, 240.f) * kLn2 * p.T;
  const Scaled z = over_T(x1 - x0, p);  // 2^-lift, as x1 is rounded
  const float down = expf(0.5f * z.hi);
  return Stream{g * (F * down * scale) * (down * (1.f + z.lo)), x1};
}

// The stream of a faint rest, whose columns have the statistic `rest`: at beta = 0 G_rest is -q (p S is
// nothing beside it), and p_j / p_rest = 2^((x_j - m) c) / s.  Otherwise G / p and p_j are in range.
__device__ __forceinline__ Stream faint_stream(const MaxStat& rest, float lse, float q, float S, float g,
                                               const DistillParams& p) {
  if (p.beta == 0.f && q > 0.f) return stream_of(g, -q, 1.f / rest.s, rest.m, p);
  const Scaled z = over_T(rest.m, p);
  const Term t = bucket(q, 0.f, faint_ratio(q, rest.s, (z.hi - lse) + z.lo), p.beta);
  const float x0 = lse * p.T;
  const Scaled z0 = over_T(x0, p);
  return stream_of(g, rest_factor(t, 0.f) - S, expf((z0.hi - lse) + z0.lo), x0, p);
}

// One row's results (every lane of the list warp); the slots then hold G_k and p_k.
struct RowResult {
  float loss, lse, p_rest;
  float m, inv_s;  // p_j = 2^((x_j - m) c) inv_s
  float S, F;      // sum of G, G_rest / p_rest
  bool faint;
};

// The slots and the rest of a row, from the statistic `st` of the columns outside the list.
__device__ __forceinline__ RowResult finish_row(const Slots& sl, int K, const Teacher& te, const MaxStat& st,
                                                const DistillParams& p) {
  const int lane = threadIdx.x & 31;
  float m = st.s != 0.f ? st.m : -FLT_MAX;
  for (int k = lane; k < K; k += 32)
    if (sl.id[k] >= 0) m = fmaxf(m, sl.x[k]);
  m = warp_max(m);
  const float s_rest = st.s == 0.f ? 0.f : st.s * exp_over_T(st.m - m, p);
  float s_list = 0.f;
  for (int k = lane; k < K; k += 32)
    if (sl.id[k] >= 0) s_list += exp_over_T(sl.x[k] - m, p);
  s_list = warp_sum(s_list);
  const float s = s_rest + s_list, inv_s = 1.f / s, ln_s = logf(s);
  float loss = 0.f, S = 0.f;
  for (int k = lane; k < K; k += 32) {
    if (sl.id[k] < 0) continue;
    const float d = sl.x[k] - m;
    const Scaled z = over_T(d, p);
    const float pk = exp_over_T(d, p) * inv_s, lq = te.log_q(sl.lq[k]);
    const Term t = bucket(expf(lq), pk, ((lq - z.hi) + ln_s) - z.lo, p.beta);
    loss += t.loss;
    S += t.G;
    sl.lq[k] = t.G;
    sl.x[k] = pk;
  }
  const float pr = s_rest * inv_s, pl = s_list * inv_s;
  const float dr = pr > 0.5f && te.over == 0.f ? pl - te.list : te.rest - pr;  // q_rest - p_rest
  RowResult o;
  o.faint = pr < FLT_MIN && st.s != 0.f;
  const Scaled zr = over_T(st.m - m, p);
  const float r = o.faint ? faint_ratio(te.rest, st.s * inv_s, zr.hi + zr.lo) : rest_ratio(te.rest, pr, dr);
  const Term t = bucket(te.rest, pr, r, p.beta);
  const Scaled zm = over_T(m, p);
  o.lse = zm.hi + ln_s;
  // relative to the lse as it is stored: the backward's other p_j are too, and the common factor
  // cancels in its differences
  o.p_rest = s_rest * expf((zm.hi - o.lse) + zm.lo);
  if (o.p_rest == 0.f && st.s != 0.f) o.p_rest = kLeastMass;
  o.loss = row_loss(warp_sum(loss) + t.loss, te.over, p.beta);
  o.m = m;
  o.inv_s = inv_s;
  o.S = warp_sum(S) + t.G;
  o.F = rest_factor(t, pr);
  return o;
}

// The row's list (one warp): ids, teacher log-probs and the student's logits.  Returns whether
// this thread met an id >= V.
template <class E>
__device__ __forceinline__ bool load_slots(const Slots& sl, const DistillParams& p, int64_t r,
                                           const typename E::storage* row) {
  bool bad = false;
  for (int k = threadIdx.x & 31; k < p.K; k += 32) {
    const int64_t id = p.ids[r * p.K + k];
    const bool in = id >= 0 && id < p.x.V;
    bad |= id >= p.x.V;
    sl.id[k] = in ? static_cast<int>(id) : -1;
    sl.lq[k] = p.tlogp[r * p.K + k];
    sl.x[k] = in ? E::load_scalar_coherent(row + static_cast<int>(id)) : 0.f;
  }
  return bad;
}

// The bitmap of listed columns.  Column j of a row whose body starts at `head` has bit
// j - head + kVec (so that body vector i has kVec bits of its own), wrapped to the bitmap.
template <class E>
struct Bitmap {
  uint32_t* w;
  uint32_t mask;  // bits - 1 when positions wrap, else all ones
  int head;
  __device__ __forceinline__ uint32_t pos(int j) const { return static_cast<uint32_t>(j - head + E::kVec) & mask; }
  // sets column j's bit; true if it was set before
  __device__ __forceinline__ bool set(int j) {
    const uint32_t q = pos(j);
    return (atomicOr(&w[q >> 5], 1u << (q & 31u)) >> (q & 31u) & 1u) != 0;
  }
  __device__ __forceinline__ bool get(int j) const {
    const uint32_t q = pos(j);
    return (w[q >> 5] >> (q & 31u) & 1u) != 0;
  }
  // the kVec bits of body vector i
  __device__ __forceinline__ uint32_t vec(int i) const {
    const uint32_t q = (static_cast<uint32_t>(i + 1) * E::kVec) & mask;
    return (w[q >> 5] >> (q & 31u)) & ((1u << E::kVec) - 1u);
  }
  __device__ __forceinline__ bool wraps() const { return mask != 0xFFFFFFFFu; }
};

// -inf in the elements of v whose bit is set.
__device__ __forceinline__ void drop(uint4& v, uint32_t bits, BF16*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (bits >> (2 * q) & 1u) w[q] = (w[q] & 0xFFFF0000u) | 0xFF80u;
    if (bits >> (2 * q + 1) & 1u) w[q] = (w[q] & 0xFFFFu) | 0xFF800000u;
  }
}
__device__ __forceinline__ void drop(uint4& v, uint32_t bits, F32*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (bits >> q & 1u) w[q] = 0xFF800000u;
}

// The listed columns among [j0, j0 + n), by looking through the list.
__device__ __forceinline__ uint32_t listed_bits(const Slots& sl, int K, int j0, int n) {
  uint32_t bits = 0u;
  for (int k = 0; k < K; ++k) {
    const int d = sl.id[k] - j0;
    if (sl.id[k] >= 0 && d >= 0 && d < n) bits |= 1u << d;
  }
  return bits;
}

// Bytes of shared memory: the bitmap, then the list.
template <class E>
__host__ __device__ inline int bitmap_bytes(int V) {
  const int64_t need = (static_cast<int64_t>(V) + 2 * E::kVec + 127) / 128 * 16;
  return need < kBitmapBytes ? static_cast<int>(need) : kBitmapBytes;
}

// out_j = f 2^((x_j - x0) c) over the span (the streaming threads).  With kept_vecs > 0 (the span is
// the row) body vectors [0, kept_vecs) come from `kept` in shared memory, after the others.
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__device__ __forceinline__ void grad_stream(const typename E::storage* in, typename E::storage* out,
                                            const RowSplit& sp, const Span& sn, float x0, float c, float f,
                                            const uint4* kept = nullptr, int kept_vecs = 0) {
  const int tid = threadIdx.x;
  auto scalar = [&](int j) { E::store_scalar(out + j, f * ex2((E::load_scalar_coherent(in + j) - x0) * c)); };
  if (sn.head && tid < sp.head) scalar(tid);
  if (sn.tail && tid < sp.tail) scalar(sp.head + sp.nvec * E::kVec + tid);
  const typename E::storage* ib = in + sp.head;
  uint4* ob = reinterpret_cast<uint4*>(out + sp.head);
  const float2 c2 = make_float2(c, c), n0 = make_float2(-x0, -x0), f2 = make_float2(f, f);
  auto process = [&](const uint4& v, int i) {
    float2 d[E::kPairs];
#pragma unroll
    for (int q = 0; q < E::kPairs; ++q) {
      const float2 t = __fmul2_rn(__fadd2_rn(E::pair(v, q), n0), c2);
      d[q] = __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), f2);
    }
    st_v4_evict_first(ob + i, E::template pack_pairs<false>(d));
  };
  auto sweep = [&](auto load, int i, int n) {
    for (; i + (UNROLL - 1) * THREADS < n; i += UNROLL * THREADS) {
      uint4 v[UNROLL];
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) v[k] = load(i + k * THREADS);
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) process(v[k], i + k * THREADS);
    }
    if (i < n) {  // the last step: its loads go out together too
      uint4 v[UNROLL];
#pragma unroll
      for (int k = 0; k < UNROLL; ++k)
        if (i + k * THREADS < n) v[k] = load(i + k * THREADS);
#pragma unroll
      for (int k = 0; k < UNROLL; ++k)
        if (i + k * THREADS < n) process(v[k], i + k * THREADS);
    }
  };
  if constexpr (SAME_PHASE) {
    sweep([&](int j) { return ld_v4_evict_first(reinterpret_cast<const uint4*>(ib) + j); }, sn.v0 + kept_vecs + tid,
          sn.v1);
  } else {
    for (int i = sn.v0 + tid; i < sn.v1; i += UNROLL * THREADS) {
      uint4 v[UNROLL];
      load_out_of_phase<E, UNROLL, THREADS>(v, ib, i, sn.v1, sp.nvec);
#pragma unroll
      for (int k = 0; k < UNROLL; ++k)
        if (i + k * THREADS < sn.v1) process(v[k], i + k * THREADS);
    }
  }
  if (kept_vecs > 0) sweep([&](int j) { return kept[j]; }, tid, kept_vecs);
}

// Part `part` of `parts` of a row: an equal share of its vectors, the head with the first, the tail
// with the last.
__device__ __forceinline__ Span span_of(const RowSplit& sp, int part, int parts) {
  const int share = (sp.nvec + parts - 1) / parts;
  const int v0 = min(sp.nvec, part * share);
  return Span{v0, min(sp.nvec, v0 + share), part == 0, part == parts - 1};
}
template <class E>
__device__ __forceinline__ bool in_span(const RowSplit& sp, const Span& sn, int j) {
  if (j < sp.head) return sn.head;
  const int i = (j - sp.head) / E::kVec;
  return i >= sp.nvec ? sn.tail : i >= sn.v0 && i < sn.v1;
}

// Forward, or (FUSED) forward and backward in one kernel: the row is swept again for the gradient
// once its factor is known, from L2 or (long rows, 512 threads) from the part kept in shared
// memory, as in fused_kernel.
// The forward of many rows is held to the registers that let five CTAs share an SM (8192 rows of 304
// KB: 280 us, 300 us with four).
// CS > 1 (forward of few rows): a cluster of CTAs takes a row, a part each; the first one gets the
// parts' statistics and finishes the row.
template <class E, int THREADS, int UNROLL, bool FUSED, bool SAME_PHASE, int CS>
__global__ void __launch_bounds__(THREADS + 32, THREADS == 256 && !FUSED ? 5 : 0)
    distill_kernel(const DistillParams p, int bm_bytes, int keep_vecs) {
  using S = typename E::storage;
  constexpr int kWarps = THREADS / 32;
  extern __shared__ uint4 distill_smem[];
  __shared__ MaxStat sh_stat[kWarps], sh_parts[CS];
  __shared__ float sh_factor, sh_m;
  __shared__ __align__(8) uint64_t kept_bar;
  wait_for_previous_grids();
  const int rank = CS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t r = blockIdx.x / CS;
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const int tid = threadIdx.x, V = p.x.V, K = p.K;
  const bool list_warp = tid >= THREADS;
  S* out = FUSED ? static_cast<S*>(p.dx.ptr) + b * p.dx.sb + l * p.dx.sl : nullptr;
  if (p.mask != nullptr && p.mask[r] == 0) {
    if (tid == 0 && rank == 0) {
      p.loss[r] = 0.f;
      p.lse[r] = 0.f;
      p.p_rest[r] = 0.f;
    }
    if (FUSED && !list_warp) {
      const RowSplit osp = split_row<E>(out, V);
      fill_span<E, THREADS>(out, osp, whole_row(osp), 0u);
    }
    return;
  }
  if (CS > 1) cluster_arrive();  // every CTA of the cluster runs before its shared memory is written
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const RowSplit sp = split_row<E>(row, V);
  const Span sn = span_of(sp, rank, CS);
  uint4* kept = distill_smem;
  uint4* bits = kept + (FUSED ? keep_vecs : 0);
  const Slots sl = slots_at(reinterpret_cast<char*>(bits) + bm_bytes, K);
  Bitmap<E> bm;
  bm.w = reinterpret_cast<uint32_t*>(bits);
  bm.mask = V + 2 * E::kVec > bm_bytes * 8 ? static_cast<uint32_t>(bm_bytes) * 8u - 1u : 0xFFFFFFFFu;
  bm.head = sp.head;
  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  const int kv = FUSED && SAME_PHASE ? min(keep_vecs, sp.nvec) : 0;
  const uint32_t bar = smem_addr(&kept_bar);
  if (FUSED && kv > 0 && tid == 0) kept_copy_issue(bar, smem_addr(kept), vb, static_cast<uint32_t>(kv) * 16u);

  bool bad = false;
  if (list_warp) {
    bad = load_slots<E>(sl, p, r, row);
    if (bad && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
  } else {
    for (int i = tid; i < bm_bytes / 16; i += THREADS) bits[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (list_warp) {
    for (int k = tid - THREADS; k < K; k += 32) {
      const int id = sl.id[k];
      if (id < 0 || !bm.set(id)) continue;
      bool twice = !bm.wraps();
      for (int q = 0; !twice && q < K; ++q) twice = q != k && sl.id[q] == id;
      if (twice && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_DUPLICATE_ID_BIT);
      bad |= twice;
    }
  }
  __syncthreads();

  Teacher te{};
  const float c = p.c;
  if (list_warp) {
    te = teacher_of(sl, K, p.tail);
  } else {
    MaxRun rs;
    auto scalar = [&](int j) {
      if (bm.get(j) && (!bm.wraps() || listed_bits(sl, K, j, 1))) return;
      maxrun_scalar(rs, FUSED ? E::load_scalar_coherent(row + j) : E::load_scalar(row + j), c);
    };
    if (sn.head && tid < sp.head) scalar(tid);
    if (sn.tail && tid < sp.tail) scalar(sp.head + sp.nvec * E::kVec + tid);
    auto leave_out = [&](uint4& v, int i) {
      uint32_t w = bm.vec(i);
      if (w != 0u) {
        if (bm.wraps()) w = listed_bits(sl, K, sp.head + i * E::kVec, E::kVec);
        drop(v, w, static_cast<E*>(nullptr));
      }
    };
    auto sweep = [&](auto load, int i, int n) {
      for (; i + (UNROLL - 1) * THREADS < n; i += UNROLL * THREADS) {
        uint4 v[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) v[k] = load(i + k * THREADS);
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) leave_out(v[k], i + k * THREADS);
        maxrun_vectors<E>(rs, v, c);
      }
      if (i < n) {  // the last step: its loads go out together too
        const uint32_t pad = sizeof(S) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
        uint4 v[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          v[k] = make_uint4(pad, pad, pad, pad);
          if (i + k * THREADS < n) v[k] = load(i + k * THREADS);
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
          if (i + k * THREADS < n) leave_out(v[k], i + k * THREADS);
        maxrun_vectors<E>(rs, v, c);
      }
    };
    // FUSED: coherent loads (dlogits may alias the logits), kept in L2 for the second sweep
    sweep([&](int i) { return FUSED ? ld_v4_evict_last(vb + i) : ld_nc_v4(vb + i); }, sn.v0 + kv + tid, sn.v1);
    if (FUSED && kv > 0) {
      if (!kept_copy_wait(bar)) {  // the row's outputs are not valid; wait once more for the copies in flight
        if (tid == 0 && p.dev_err != nullptr) atomicOr(p.dev_err, GRPO_DEVERR_TIMEOUT_BIT);
        kept_copy_wait(bar);
      }
      sweep([&](int i) { return kept[i]; }, tid, kv);
    }
    const MaxStat st = maxstat_warp(rs.stat(), c);
    if ((tid & 31) == 0) sh_stat[tid >> 5] = st;
  }
  __syncthreads();
  if (CS > 1) {
    cluster_wait();
    if (list_warp) {
      const int lane = tid - THREADS;
      const MaxStat st = maxstat_warp(lane < kWarps ? sh_stat[lane] : MaxStat{-FLT_MAX, 0.f}, c);
      if (lane == 0) {
        const uint32_t to = map_to_rank(smem_addr(&sh_parts[rank]), 0);
        st_cluster_f32(to, st.m);
        st_cluster_f32(to + 4u, st.s);
      }
    }
    cluster_sync();
    if (rank != 0) return;
  }
  if (list_warp) {
    const int lane = tid - THREADS;
    constexpr int kStats = CS > 1 ? CS : kWarps;
    const MaxStat* stats = CS > 1 ? sh_parts : sh_stat;
    const MaxStat st = maxstat_warp(lane < kStats ? stats[lane] : MaxStat{-FLT_MAX, 0.f}, c);
    const float g = FUSED ? p.dloss[r] / p.T : 0.f;
    if (p.tail && st.s == 0.f) te = renormalised(te.sum);  // there is no rest
    const RowResult o = finish_row(sl, K, te, st, p);
    const float nan = __int_as_float(0x7FC00000);
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      p.loss[r] = bad ? nan : o.loss;
      p.lse[r] = bad ? nan : o.lse;
      p.p_rest[r] = bad ? nan : o.p_rest;
    }
    if (FUSED) {
      for (int k = lane; k < K; k += 32) sl.lq[k] = bad ? nan : g * (sl.lq[k] - sl.x[k] * o.S);
      if (lane == 0) {
        const Stream t =
            o.faint ? faint_stream(st, o.lse, te.rest, o.S, g, p) : stream_of(g, o.F - o.S, o.inv_s, o.m, p);
        sh_factor = g == 0.f ? 0.f : (bad ? nan : t.f);
        sh_m = t.x0;
        sh_stat[0].s = g;
      }
    }
  }
  if (!FUSED) return;
  __syncthreads();
  const RowSplit osp = split_row<E>(out, V);
  const float f = sh_factor, g = sh_stat[0].s;
  if (!list_warp) {
    if (f == 0.f) {
      fill_span<E, THREADS>(out, osp, whole_row(osp), 0u);
      l2_demote<THREADS>(row, static_cast<int64_t>(V) * sizeof(S));  // not read again after all
    } else {
      grad_stream<E, THREADS, UNROLL, SAME_PHASE>(row, out, osp, whole_row(osp), sh_m, c, f, kept, kv);
    }
  }
  if (g == 0.f) return;  // +0.0 everywhere
  __syncthreads();       // the listed columns' values go over the stream's
  if (list_warp)
    for (int k = tid - THREADS; k < K; k += 32)
      if (sl.id[k] >= 0) E::store_scalar(out + sl.id[k], sl.lq[k]);
}

// The statistic of a row's columns outside the list, whose slots are loaded (the backward of a faint
// rest; all threads call).  Vectors with a listed column are found by a bit per vector, places shared
// modulo kMarks; only those look through the list.  One vector in flight, so that the kernel's registers
// do not grow for it (four in flight: 56 of them where the stream takes 32 to 40): such rows take twice
// the time of others.
constexpr int kMarks = 8192;
template <class E, int THREADS>
__device__ __forceinline__ MaxStat rest_stat(const typename E::storage* row, const Slots sl, int K, int V, float c) {
  constexpr int kWarps = THREADS / 32;
  __shared__ uint32_t marks[kMarks / 32];
  __shared__ MaxStat sh[kWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < kMarks / 32; i += THREADS + 32) marks[i] = 0u;
  __syncthreads();
  const RowSplit sp = split_row<E>(row, V);
  if (tid >= THREADS)
    for (int k = lane; k < K; k += 32) {
      const int j = sl.id[k] - sp.head;
      if (sl.id[k] < 0 || j < 0) continue;  // the head and the tail look through the list anyway
      const unsigned v = static_cast<unsigned>(j / E::kVec) % kMarks;
      atomicOr(&marks[v >> 5], 1u << (v & 31u));
    }
  __syncthreads();
  if (tid < THREADS) {
    MaxRun rs;
    auto scalar = [&](int j) {
      if (listed_bits(sl, K, j, 1) == 0u) maxrun_scalar(rs, E::load_scalar_coherent(row + j), c);
    };
    if (tid < sp.head) scalar(tid);
    if (tid < sp.tail) scalar(sp.head + sp.nvec * E::kVec + tid);
    const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
    for (int i = tid; i < sp.nvec; i += THREADS) {
      uint4 v[1] = {ld_v4(vb + i)};
      const unsigned q = static_cast<unsigned>(i) % kMarks;
      if (marks[q >> 5] >> (q & 31u) & 1u)
        drop(v[0], listed_bits(sl, K, sp.head + i * E::kVec, E::kVec), static_cast<E*>(nullptr));
      maxrun_vectors<E>(rs, v, c);
    }
    const MaxStat st = maxstat_warp(rs.stat(), c);
    if (lane == 0) sh[tid >> 5] = st;
  }
  __syncthreads();
  return maxstat_warp(lane < kWarps ? sh[lane] : MaxStat{-FLT_MAX, 0.f}, c);
}

// CTAs of the backward per SM that its registers are held to: as many as the stream alone allows,
// rest_stat aside (with its registers 8192 rows of 4 KB take 24.3 us, 21.1 us without; 2048 rows of 128 KB
// of fp32 86 us and 78 us).
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
constexpr int kBwdPlaces =
    UNROLL != kUnroll || !SAME_PHASE ? 0 : (THREADS == 64 ? 21 : (sizeof(typename E::storage) == 2 ? 5 : 7));

// The backward: the list warp works out the row's factor and the listed columns' gradients, then
// the others stream the row as rowgrad_kernel does.
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__global__ void __launch_bounds__(THREADS + 32, kBwdPlaces<E, THREADS, UNROLL, SAME_PHASE>)
    distill_bwd_kernel(const DistillParams p, int parts) {
  using S = typename E::storage;
  extern __shared__ uint4 distill_smem[];
  __shared__ float sh_factor, sh_x0, sh_faint, sh_S;
  wait_for_previous_grids();
  const int64_t r = blockIdx.x / static_cast<unsigned>(parts);
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(parts));
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const int tid = threadIdx.x, V = p.x.V, K = p.K;
  const bool list_warp = tid >= THREADS;
  const bool live = p.mask == nullptr || p.mask[r] != 0;
  const float g = live ? p.dloss[r] / p.T : 0.f;
  S* out = static_cast<S*>(p.dx.ptr) + b * p.dx.sb + l * p.dx.sl;
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const RowSplit sp = split_row<E>(out, V);
  const Span sn = span_of(sp, part, parts);
  if (g == 0.f) {
    if (!list_warp) fill_span<E, THREADS>(out, sp, sn, 0u);
    return;
  }
  const Slots sl = slots_at(distill_smem, K);
  // long rows: their start comes to L2 while the list is worked on (999 rows of 200 KB: 64 us against
  // 67 us; rows of 64 KB took longer with it)
  const int64_t span_bytes = static_cast<int64_t>(sn.v1 - sn.v0) * 16;
  if (tid == 0 && span_bytes >= 131072) prefetch_row(row + sp.head + static_cast<int64_t>(sn.v0) * E::kVec, span_bytes);
  if (list_warp) {
    const int lane = tid - THREADS;
    const float lse = p.lse[r], p_rest = p.p_rest[r];
    load_slots<E>(sl, p, r, row);
    __syncwarp();
    const Teacher te = teacher_of(sl, K, p.tail && p_rest != 0.f);
    float S_sum = 0.f;
    for (int k = lane; k < K; k += 32) {
      if (sl.id[k] < 0) continue;
      const Scaled z = over_T(sl.x[k], p);
      const float lp = z.hi - lse, lq = te.log_q(sl.lq[k]);  // lp: near lse, so the difference is exact
      const float pk = expf(lp + z.lo);
      const Term t = bucket(expf(lq), pk, (lq - lp) - z.lo, p.beta);
      S_sum += t.G;
      sl.x[k] = pk;
      sl.lq[k] = t.G;
    }
    // of a faint rest only G_rest, which is -q_rest at beta = 0 and next to nothing else; its stream below
    const bool faint = p.tail && p_rest != 0.f && p_rest < FLT_MIN;
    const Term t = bucket(te.rest, p_rest, rest_ratio(te.rest, p_rest, te.rest - p_rest), p.beta);
    S_sum = warp_sum(S_sum) + (!faint ? t.G : (p.beta == 0.f ? -te.rest : 0.f));
    for (int k = lane; k < K; k += 32) sl.lq[k] = g * (sl.lq[k] - sl.x[k] * S_sum);
    // p_j = 2^((x_j - x0) c) e^(x0 / T - lse): x0 takes up lse, so that no exponent is a small
    // difference of large products
    if (lane == 0) {
      const float x0 = lse * p.T;
      const Scaled z = over_T(x0, p);
      const Stream st = stream_of(g, rest_factor(t, p_rest) - S_sum, expf((z.hi - lse) + z.lo), x0, p);
      sh_factor = st.f;
      sh_x0 = st.x0;
      sh_faint = faint ? te.rest : 0.f;
      sh_S = S_sum;
    }
  }
  __syncthreads();
  Stream st{sh_factor, sh_x0};
  if (sh_faint != 0.f) {
    const MaxStat rest = rest_stat<E, THREADS>(row, sl, K, V, p.c);
    st = faint_stream(rest, p.lse[r], sh_faint, sh_S, g, p);
  }
  if (!list_warp) {
    if (st.f == 0.f) fill_span<E, THREADS>(out, sp, sn, 0u);
    else grad_stream<E, THREADS, UNROLL, SAME_PHASE>(row, out, sp, sn, st.x0, p.c, st.f);
  }
  __syncthreads();  // the listed columns' values go over the stream's
  if (list_warp)
    for (int k = tid - THREADS; k < K; k += 32)
      if (sl.id[k] >= 0 && in_span<E>(sp, sn, sl.id[k])) E::store_scalar(out + sl.id[k], sl.lq[k]);
}

template <class E, int THREADS, int U, bool FUSED, bool SAME_PHASE, int CS = 1>
cudaError_t launch_distill_k(const DistillParams& p, int64_t rows, int keep_bytes, cudaStream_t s) {
  const int bm = bitmap_bytes<E>(p.x.V);
  const size_t smem = static_cast<size_t>(keep_bytes) + bm + 12 * static_cast<size_t>(p.K);
  auto* kernel = distill_kernel<E, THREADS, U, FUSED, SAME_PHASE, CS>;
  if (smem > 46 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kFusedKeepBytes + kBitmapBytes + 12 * kDistillMaxK);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * CS));
  cfg.blockDim = dim3(THREADS + 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, bm, keep_bytes / 16);
}

// CTAs per row: as many (8 at most) as keep `places` CTAs at once, each with a step of its sweep
// (1024 vectors) or more.
template <class E>
int row_parts(const DistillParams& p, int64_t rows, int64_t places) {
  int n = 1;
  while (n < 8 && rows * n * 2 <= places && p.x.V / E::kVec >= 2048 * n) n *= 2;
  return n;
}

// Streaming threads of the forward, and vectors in flight of each: 64 x 4 for short rows; 128 x 8 while
// that leaves most rows resident (6 such CTAs per SM: 2048 rows of 64 KB 26 us, against 30 us with
// 256 x 4 and 34 us with 256 x 8, whose last step is mostly empty), in clusters while rows leave SMs
// idle; else 256 x 4.
template <class E>
cudaError_t launch_distill_fwd_e(const DistillParams& p, int64_t rows, int sms, cudaStream_t s) {
  if (static_cast<int64_t>(p.x.V) * sizeof(typename E::storage) <= 8192)
    return launch_distill_k<E, 64, kUnroll, false, true>(p, rows, 0, s);
  switch (row_parts<E>(p, rows, 7LL * sms)) {
    case 8: return launch_distill_k<E, 128, 8, false, true, 8>(p, rows, 0, s);
    case 4: return launch_distill_k<E, 128, 8, false, true, 4>(p, rows, 0, s);
    case 2: return launch_distill_k<E, 128, 8, false, true, 2>(p, rows, 0, s);
    default: break;
  }
  return rows <= 20LL * sms ? launch_distill_k<E, 128, 8, false, true>(p, rows, 0, s)
                            : launch_distill_k<E, 256, kUnroll, false, true>(p, rows, 0, s);
}

template <class E, int THREADS, int U>
cudaError_t launch_distill_bwd_t(bool same_phase, const DistillParams& p, int64_t rows, int parts, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows * parts)), block(THREADS + 32);
  const size_t smem = 12 * static_cast<size_t>(p.K);
  return same_phase
             ? launch_after_previous_smem(distill_bwd_kernel<E, THREADS, U, true>, grid, block, smem, s, p, parts)
             : launch_after_previous_smem(distill_bwd_kernel<E, THREADS, kUnroll, false>, grid, block, smem, s, p, parts);
}

// Long rows with eight vectors in flight per thread (8192 rows of 304 KB: 662 us against 673 us); few
// rows in parts, a CTA each, unless the gradients go over the logits: every part reads all of the row's
// listed logits, which another part may have overwritten by then.
template <class E>
cudaError_t launch_distill_bwd_e(bool same_phase, const DistillParams& p, int64_t rows, int sms, cudaStream_t s) {
  const int64_t bytes = static_cast<int64_t>(p.x.V) * sizeof(typename E::storage);
  if (pick_threads_bwd(p.x.V, sizeof(typename E::storage), rows, sms) == 64)
    return launch_distill_bwd_t<E, 64, kUnroll>(same_phase, p, rows, 1, s);
  const int parts = p.dx.ptr == p.x.ptr ? 1 : row_parts<E>(p, rows, 5LL * sms);
  return bytes / parts < 131072 ? launch_distill_bwd_t<E, 256, kUnroll>(same_phase, p, rows, parts, s)
                                : launch_distill_bwd_t<E, 256, 8>(same_phase, p, rows, parts, s);
}

template <class E, int THREADS, int U>
cudaError_t launch_distill_fused_t(bool same_phase, const DistillParams& p, int64_t rows, int keep, cudaStream_t s) {
  return same_phase ? launch_distill_k<E, THREADS, U, true, true>(p, rows, keep, s)
                    : launch_distill_k<E, THREADS, kUnroll, true, false>(p, rows, 0, s);
}

// The part of long rows that is kept is that of grpo_loss_fused less the bitmap and the list, so that
// two CTAs still share an SM.  Shorter rows: 128 streaming threads, eight vectors in flight each (2048
// rows of 64 KB, on one machine: 51 us; 58 us with four in flight, 61 us with 256 x 4: more CTAs are in
// different phases of their rows; others take up to 66 us).
template <class E>
cudaError_t launch_distill_fused_e(bool same_phase, const DistillParams& p, int64_t rows, int sms, cudaStream_t s) {
  (void)sms;
  const int64_t bytes = static_cast<int64_t>(p.x.V) * sizeof(typename E::storage);
  if (bytes <= 8192) return launch_distill_fused_t<E, 64, kUnroll>(same_phase, p, rows, 0, s);
  if (bytes < 131072) return launch_distill_fused_t<E, 128, 8>(same_phase, p, rows, 0, s);
  const int keep = (kFusedKeepBytes - bitmap_bytes<E>(p.x.V) - 12 * p.K) / 1024 * 1024;
  return launch_distill_fused_t<E, 512, kUnroll>(same_phase, p, rows, keep, s);
}

}  // namespace
}  // namespace grpo
