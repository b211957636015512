// Preference loss on pairs of sequences (paired log ratios), on the row pass.
//
// With S_b the sum (or mean) of a sequence's log-probs on its unmasked tokens and
//   h_i = beta ((S_i - ref_i) - (S_{P+i} - ref_{P+i})) - gamma,
// a pair's loss is a function of its margin h_i alone, so
//   dlogits_rj = g_r (1[j == idx_r] - p_j),  g_r = coef_b dloss_i / T,
// with one factor coef_b a sequence.  Three kernels: the rows' statistics (masked rows are not
// read), the pairs' terms, and the gradient rows (those with g == 0 are filled, not read).  The first
// and the last are streams over the logits: 2 x 2048 tokens at V = 151936 bf16, three eighths unmasked,
// take 155 and 506 us where the copy rate would take 138 and 505; the forward of rows of 64 KB stays at 75 to
// 92 % of it, for each row's start and end.  The terms are one chain of 5 us.
#pragma once

#include "logits_load.cuh"
#include "rowpass_bwd.cuh"
#include "rowpass_fwd.cuh"
#include "train_ops.h"
#include "two_sum.cuh"

namespace grpo {
namespace {

// ln s for s > 0, to about 1e-9: with s = 2^e m, m within a root of 2 of 1, and z = (m-1)/(m+1),
// ln m = 2 atanh z = 2 (z + z^3/3 + z^5/5 + ...); the quotient in two parts.
__device__ __forceinline__ TwoSum ln_two_parts(float s) {
  if (!(s >= 1.17549435e-38f && s <= 3.4028235e38f)) return TwoSum{logf(s), 0.f};  // 0, inf, NaN
  int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;
  float m = __uint_as_float((__float_as_uint(s) & 0x007FFFFFu) | 0x3F800000u);
  if (m > 1.41421356f) {
    m *= 0.5f;
    ++e;
  }
  const float num = m - 1.f, den = m + 1.f, den_lo = m - (den - 1.f);  // num and den_lo exact
  const float z = num / den;
  const float z_lo = (fmaf(-z, den, num) - z * den_lo) / den;
  const float z2 = z * z;
  const float series = z2 * fmaf(z2, fmaf(z2, fmaf(z2, fmaf(z2, 1.f / 11.f, 1.f / 9.f), 1.f / 7.f), 0.2f), 1.f / 3.f);
  constexpr float kLn2Hi = 0.69314718055994530942f;
  constexpr float kLn2Lo = static_cast<float>(0.69314718055994530942 - static_cast<double>(kLn2Hi));
  return two_add(two_mul(static_cast<float>(e), TwoSum{kLn2Hi, kLn2Lo}), TwoSum{2.f * z, 2.f * fmaf(z, series, z_lo)});
}

// A margin is the difference of two sums of thousands of log-probs, so what errs the same way on
// every token counts (at 2 x 2048 tokens the rewards came out 1.1e-5 off).  Five things did:
// - the rescaling of sums when a maximum moves: the offsets a are whole numbers here (the maximum
//   times c, rounded up, and 1), so every rescaling is by a power of two, and exact;
// - the sums: a bf16 logit that occurs often adds the same number often, and loses the same part of it
//   to the large sum each time (6e-7 for 151936 columns).  So the exponentials of a step are added
//   to one another first, which takes no more additions;
// - the exponential: ex2.approx is 5.1e-8 too small on average below -1, the same in every octave (3e-8 of
//   spread around that), but 2.2e-8 in (-1, 0) for arguments of all 24 bits: hence the 1 in the offsets, without
//   which rows of one large logit err by 2e-8 more than others.  What the log-sum-exps came out too small is added: 5.1e-8
//   for bf16 logits; for fp32 ones 4.58e-8, a little less, for in a row of few logits at whole distances the
//   exponential is exact.  Means over 2048 rows, V = 512 to 151936, T = 0.7 to 1.3, logits of a spread of 1 or 2: within
//   4e-9 for bf16 and 6e-9 for fp32.  (With 4.5e-8 for both and no 1: -8e-9 for bf16 and up to 2.1e-8 for fp32, which is
//   1.5e-6 of a reward of 1 over 700 tokens, where the plain sum of such log-probs is 3e-7 off.  A spread of 4 at T =
//   0.7 and V = 151936 leaves 1e-7: what small terms lose beside a thread's large ones.)
// - the rounding of t = x c - a, which is the same for the same bf16 logit in every row: c has 15 bits
//   for bf16 logits, so that x c is exact (fp32 logits are not alike, and their errors average out);
// - the rounding of c: x_idx / T is formed in two parts, and the log-sum-exp is corrected to first
//   order.  With 1 + d the exact log2(e) / T over c, |d| <= 2^-15 (the second order is below 1e-8),
//   ln sum 2^(x c (1 + d)) = ln2 (1 + d) a + ln s + d ln2 u / s,   u = sum 2^t t.
template <class E>
constexpr float kExpLow = E::kVec == 8 ? 5.1e-8f : 4.58e-8f;

__device__ __forceinline__ void pref_offset(Running& rs, float newm, float c) {
  newm = fmaxf(newm, kNegClamp);  // columns masked by their type's lowest value: newm * c may be -inf
  const float a = ceilf(newm * c) + 1.f;
  if (rs.s.x != 0.f || rs.s.y != 0.f) {
    const float delta = rs.a - a;
    const float2 al = make_float2(ex2(delta), ex2(delta));
    rs.u = __fmul2_rn(al, __ffma2_rn(make_float2(delta, delta), rs.s, rs.u));
    rs.s = __fmul2_rn(al, rs.s);
  }
  rs.m = newm;
  rs.a = a;
}

__device__ __forceinline__ void pref_scalar(Running& rs, float x, float c) {
  if (x > rs.m) pref_offset(rs, x, c);
  if (x < kNegClamp) x = kNegClamp;  // a -inf logit adds 0 to u, not 0 * -inf
  const float t = fmaf(x, c, -rs.a), e = ex2(t);
  rs.s.x += e;
  rs.u.x = fmaf(e, t, rs.u.x);
}

template <class E, int N>
__device__ __forceinline__ void pref_vectors(Running& rs, uint4 (&v)[N], float c) {
  const float cm = E::template chunk_max<N>(v);
  if (cm > rs.m) pref_offset(rs, cm, c);
  const float2 c2 = make_float2(c, c), na2 = make_float2(-rs.a, -rs.a);
  float2 s[N], u[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    E::clamp_low(v[k]);
    float2 e[E::kPairs];
#pragma unroll
    for (int i = 0; i < E::kPairs; ++i) {
      const float2 t = __ffma2_rn(E::pair(v[k], i), c2, na2);
      e[i] = make_float2(ex2(t.x), ex2(t.y));
      u[k] = i == 0 ? __fmul2_rn(e[0], t) : __ffma2_rn(e[i], t, u[k]);
    }
    s[k] = __fadd2_rn(e[0], e[1]);
    if constexpr (E::kPairs == 4) s[k] = __fadd2_rn(s[k], __fadd2_rn(e[2], e[3]));
  }
#pragma unroll
  for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
    for (int k = 0; k < w; ++k) {
      s[k] = __fadd2_rn(s[k], s[k + w]);
      u[k] = __fadd2_rn(u[k], u[k + w]);
    }
  rs.s = __fadd2_rn(rs.s, s[0]);
  rs.u = __fadd2_rn(rs.u, u[0]);
}

// This thread's part of a row's statistic.  KEEP: with L2 priority evict_last, for a backward that reads
// the rows again (see launch_pref_rows_threads).
template <class E, int THREADS, int UNROLL, bool KEEP>
__device__ __forceinline__ Stat pref_row(const typename E::storage* row, int V, float c) {
  const int tid = threadIdx.x;
  const auto load = [](const uint4* q) { return KEEP ? ld_nc_v4_evict_last(q) : ld_nc_v4(q); };
  Running rs{-INFINITY, 0.f, make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const RowSplit sp = split_row<E>(row, V);
  if (tid < sp.head) pref_scalar(rs, E::load_scalar(row + tid), c);
  if (tid < sp.tail) pref_scalar(rs, E::load_scalar(row + sp.head + sp.nvec * E::kVec + tid), c);
  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  int i = tid;
  for (; i + (UNROLL - 1) * THREADS < sp.nvec; i += UNROLL * THREADS) {
    uint4 v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) v[k] = load(vb + i + k * THREADS);
    pref_vectors<E>(rs, v, c);
  }
  for (; i < sp.nvec; i += THREADS) {
    uint4 v[1] = {load(vb + i)};
    pref_vectors<E>(rs, v, c);
  }
  return Stat{rs.a, rs.s.x + rs.s.y, rs.u.x + rs.u.y};
}

// logp and lse of a row from its merged statistic (thread 0).  Rows without mass: nothing but -inf, or so far down
// (a mask's values in every column) that lse has no fraction in fp32 and the backward no digit of any p_j.
constexpr float kNoMass = -0x1p24f;
template <class E>
__device__ __forceinline__ void pref_row_outputs(const PrefParams& p, int64_t r, const Stat& st, float x_idx, bool bad) {
  const bool none = st.a <= kNoMass;
  const float more = none ? 0.f : fmaf(p.c_off, kLn2 * st.u / st.s, kExpLow<E>);
  const TwoSum lse = two_add(two_add(two_mul(st.a, TwoSum{p.ln2_hi, p.ln2_lo}), ln_two_parts(st.s)), TwoSum{more, 0.f});
  const TwoSum logp = two_sub(two_mul(x_idx, TwoSum{p.inv_hi, p.inv_lo}), lse);
  p.lse[r] = none ? -INFINITY : lse.hi + lse.lo;
  const float rounded = bad || none ? __int_as_float(0x7FC00000) : logp.hi + logp.lo;
  p.logp[r] = rounded;
  p.logp[2 * p.pairs * p.x.L + r] = !isfinite(rounded) ? 0.f : logp.lo - (rounded - logp.hi);
  if (bad && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
}

// Row r = (b, l): logp and lse, +0.0 where it is masked.
template <class E, int THREADS, int UNROLL, bool KEEP>
__device__ __forceinline__ void pref_forward_row(const PrefParams& p, int64_t r, int64_t b, int64_t l) {
  using S = typename E::storage;
  const int tid = threadIdx.x;
  const int64_t id = p.idx[r];
  if (p.mask != nullptr && p.mask[r] == 0) {
    if (tid == 0) {
      p.logp[r] = 0.f;
      p.logp[2 * p.pairs * p.x.L + r] = 0.f;
      p.lse[r] = 0.f;
    }
    return;
  }
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const int V = p.x.V;
  const Stat mine = pref_row<E, THREADS, UNROLL, KEEP>(row, V, p.c_fwd);
  const bool bad = id < 0 || id >= V;
  const float x_idx = tid == 0 ? E::load_scalar(row + (bad ? 0 : static_cast<int>(id))) : 0.f;
  const Stat st = stat_block_reduce<THREADS>(mine);
  if (tid == 0) pref_row_outputs<E>(p, r, st, x_idx, bad);
}

template <class E, int THREADS, int UNROLL, bool KEEP>
__global__ void __launch_bounds__(THREADS) pref_rows_kernel(const PrefParams p) {
  wait_for_previous_grids();
  const int64_t r = blockIdx.x;
  const int64_t b = r / p.x.L;
  pref_forward_row<E, THREADS, UNROLL, KEEP>(p, r, b, r - b * p.x.L);
}

template <int THREADS>
struct PairSums {
  TwoSum sum[2][THREADS / 32];
  int live[2][THREADS / 32];
};

// Terms of pair i from its sequences' sums of log-probs and numbers of unmasked tokens.  The margin is a
// small difference of large sums: in two parts up to there, what follows from it in fp32 (the logistic loss from
// both parts: half a step of a margin of 32 to 64 is 2e-6 of a loss of exp(-h)).
__device__ __forceinline__ void pref_pair(const PrefParams& p, int64_t i, const TwoSum& sum_w, int n_w,
                                          const TwoSum& sum_l, int n_l, float ref_w, float ref_l) {
  const int64_t w = i, l = p.pairs + i;
  const auto per = [](int n) {  // 1 / n
    if (n == 0) return TwoSum{0.f, 0.f};
    const float f = static_cast<float>(n), q = 1.f / f;
    return TwoSum{q, fmaf(-f, q, 1.f) * q};
  };
  const TwoSum per_w = per(n_w), per_l = per(n_l), mean_w = two_mul(sum_w, per_w);
  const TwoSum S_w = p.average ? mean_w : sum_w, S_l = p.average ? two_mul(sum_l, per_l) : sum_l;
  const TwoSum r_w = two_mul(p.beta, two_add(S_w, TwoSum{-ref_w, 0.f}));
  const TwoSum r_l = two_mul(p.beta, two_add(S_l, TwoSum{-ref_l, 0.f}));
  const TwoSum margin = two_add(two_sub(r_w, r_l), TwoSum{-p.gamma, 0.f});
  const float h = margin.hi + margin.lo;
  float loss, slope;  // of the margin
  if (p.kind == 1) {  // hinge: comparisons that leave a NaN margin NaN
    const TwoSum left = two_sub(TwoSum{1.f, 0.f}, margin);
    loss = h >= 1.f ? 0.f : left.hi + left.lo;
    slope = h >= 1.f ? 0.f : (h < 1.f ? -1.f : h);
  } else if (p.kind == 2) {  // squared
    const TwoSum off = two_add(margin, TwoSum{-0.5f, 0.f});
    const float u = (off.hi + off.lo) / p.beta;
    loss = u * u;
    slope = 2.f * u / p.beta;
  } else {  // -(1-e) log sig(h) - e log sig(-h), from soft = log(1 + exp(-|h|)), which never overflows
    // of h and what its rounding lost, which exp(-|h|) takes by a factor
    const float e = p.smoothing, rest = isfinite(h) ? (margin.hi - h) + margin.lo : 0.f;
    const float near = expf(-fabsf(h)), ex = fmaf(near, h >= 0.f ? -rest : rest, near);
    const float soft = log1pf(ex), up = 1.f / (1.f + ex);
    const float neg = h < 0.f ? (soft - rest) - h : soft, pos = h > 0.f ? (soft + rest) + h : soft;
    loss = (e < 1.f ? (1.f - e) * neg : 0.f) + (e > 0.f ? e * pos : 0.f);
    slope = e - (h >= 0.f ? ex * up : up);  // e sig(h) - (1-e) sig(-h) = e - sig(-h)
  }
  float c_w = slope * p.beta, c_l = -c_w;
  if (p.average) {
    c_w *= per_w.hi;
    c_l *= per_l.hi;
  }
  if (p.sft != 0.f) {
    loss = fmaf(-p.sft, mean_w.hi + mean_w.lo, loss);
    c_w = fmaf(-p.sft, per_w.hi, c_w);
  }
  p.loss[i] = loss;
  p.reward[w] = r_w.hi + r_w.lo;
  p.reward[l] = r_l.hi + r_l.lo;
  p.seq_logp[w] = S_w.hi + S_w.lo;
  p.seq_logp[l] = S_l.hi + S_l.lo;
  p.coef[w] = c_w;
  p.coef[l] = c_l;
}

// Both sequences' sums and the pair's terms, by one CTA, in an order that depends on L alone.  The
// log-probs, each read once, are in L2: the launch before has written them.
template <int THREADS>
__device__ __forceinline__ void pref_terms(const PrefParams& p, int64_t i, PairSums<THREADS>& sh) {
  constexpr int kAhead = 4;
  const int64_t L = p.x.L;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool ref = p.ref_logp != nullptr;
  const float ref_w = ref ? p.ref_logp[i] : 0.f, ref_l = ref ? p.ref_logp[p.pairs + i] : 0.f;
  TwoSum s[2] = {{0.f, 0.f}, {0.f, 0.f}};
  int live[2] = {0, 0};
  for (int64_t t0 = tid; t0 < L; t0 += kAhead * THREADS) {
    TwoSum v[2][kAhead];
    bool in[2][kAhead];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int64_t t = t0 + q * THREADS, r = (i + k * p.pairs) * L + t;
        in[k][q] = t < L && (p.mask == nullptr || p.mask[r] != 0);
        v[k][q] = t < L ? TwoSum{__ldcg(p.logp + r), __ldcg(p.logp + 2 * p.pairs * L + r)} : TwoSum{0.f, 0.f};
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        s[k] = two_add(s[k], v[k][q]);  // +0.0 where masked
        live[k] += in[k][q];
      }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s[k] = two_add(s[k], two_shfl(s[k], off));
    live[k] = __reduce_add_sync(0xFFFFFFFFu, live[k]);
    if (lane == 0) {
      sh.sum[k][warp] = s[k];
      sh.live[k][warp] = live[k];
    }
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kWarps = THREADS / 32;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      s[k] = lane < kWarps ? sh.sum[k][lane] : TwoSum{0.f, 0.f};
      live[k] = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.live[k][lane] : 0);
#pragma unroll
      for (int off = kWarps / 2; off > 0; off >>= 1) s[k] = two_add(s[k], two_shfl(s[k], off));
    }
    if (lane == 0) pref_pair(p, i, s[0], live[0], s[1], live[1], ref_w, ref_l);
  }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) pref_terms_kernel(const PrefParams p) {
  wait_for_previous_grids();
  __shared__ PairSums<THREADS> sh;
  pref_terms<THREADS>(p, blockIdx.x, sh);
}

// |g| p_j for fp32 logits.  The log-sum-exp is one fp32 number, whose half step (4.8e-7 of a gradient for one of 8 to
// 16) a whole row shares, as with every loss here; little is added to it.  In one exponent (FoldedPower, as for
// bf16 logits, whose gradients are rounded to 2^-9) the sum of lse log2(e) and log2|g| rounds once more for
// the row, the exponents are as large as the logits and not as their distance from lse, and c's rounding
// counts by the logit's size: gradients came out 4.7e-7 off, and 4e-5 for logits around 1000.  Here
//   |g| p_j = 2^t_j K,   t_j = x_j c - A,   K = |g| 2^(A - lse log2(e) + A c_off),
// with A the second whole number above lse log2(e) (the first one's power in K), whose product is formed in two
// parts, and c_off what c's rounding lost, over c (t_j c_off, below 1e-6, is left out): 3.0e-7, for a product a pair
// and no time (the pass waits for memory).
struct SplitPower {
  float c, nA, K;
  __device__ __forceinline__ float one(float x) const { return ex2(fmaf(x, c, nA)) * K; }
  __device__ __forceinline__ float2 two(float2 x) const {
    const float2 t = __ffma2_rn(x, make_float2(c, c), make_float2(nA, nA));
    return __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(K, K));
  }
};
template <class E>
__device__ __forceinline__ auto pref_power(const PrefParams& p, float lse, float g) {
  if constexpr (E::kVec == 8) {
    return FoldedPower{p.c, fmaf(-lse, kLog2e, log2f(fabsf(g)))};
  } else {
    constexpr float kLog2eLo = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
    const float hi = lse * kLog2e, lo = fmaf(lse, kLog2e, -hi) + lse * kLog2eLo, A = ceilf(hi);
    return SplitPower{p.c, -A - 1.f, 2.f * fabsf(g) * exp2f((A - hi) - lo + fmaf(A, p.c_off, kExpLow<E> * kLog2e))};
  }
}

// A row with g != 0 whose logits start at another address mod 16 than its gradient (see stream_span,
// which does the others): -|g| p_j or |g| p_j to every column, and this thread's part of the sum of
// |g| p_j over the columns but idx.
template <class E, int THREADS, int UNROLL, bool NEG, class P>
__device__ __forceinline__ float pref_stream_shifted(const typename E::storage* in, typename E::storage* out,
                                                     const RowSplit& sp, int idx, const P& power, bool& owner) {
  constexpr int VEC = E::kVec;
  const int tid = threadIdx.x;
  float sum = 0.f;
  auto scalar = [&](int j) {
    const float e = power.one(E::load_scalar(in + j));
    if (j == idx) owner = true;
    else sum += e;
    E::store_scalar(out + j, NEG ? -e : e);
  };
  if (tid < sp.head) scalar(tid);
  if (tid < sp.tail) scalar(sp.head + sp.nvec * VEC + tid);
  uint4* ob = reinterpret_cast<uint4*>(out + sp.head);
  const int idx_body = idx - sp.head;
  for (int i = tid; i < sp.nvec; i += UNROLL * THREADS) {
    uint4 v[UNROLL];
    load_out_of_phase<E, UNROLL, THREADS>(v, in + sp.head, i, sp.nvec, sp.nvec);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int j = i + k * THREADS;
      if (j >= sp.nvec) continue;
      float2 e[E::kPairs];
      float2 s = make_float2(0.f, 0.f);
      const int at = idx_body - j * VEC;
#pragma unroll
      for (int q = 0; q < E::kPairs; ++q) {
        e[q] = power.two(E::pair(v[k], q));
        s = __fadd2_rn(s, make_float2(2 * q == at ? 0.f : e[q].x, 2 * q + 1 == at ? 0.f : e[q].y));
      }
      owner |= static_cast<unsigned>(at) < static_cast<unsigned>(VEC);
      sum += s.x + s.y;
      st_v4_evict_first(ob + j, E::template pack_pairs<NEG>(e));
    }
  }
  return sum;
}

// Gradient of row (b, l), g known (see rowgrad_kernel, whose streaming this is).
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__device__ __forceinline__ void pref_grad_row(const PrefParams& p, int64_t b, int64_t l, float g, int64_t id64, float lse) {
  using S = typename E::storage;
  const int V = p.x.V;
  S* out = static_cast<S*>(p.dx.ptr) + b * p.dx.sb + l * p.dx.sl;
  const RowSplit sp = split_row<E>(out, V);
  const Span sn = whole_row(sp);
  const S* in = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const bool bad = g != 0.f && (id64 < 0 || id64 >= V);
  if (g == 0.f || bad) {
    fill_span<E, THREADS>(out, sp, sn, bad ? E::kNaNPair : 0u);
    if (bad && threadIdx.x == 0 && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
    return;
  }
  const int idx = static_cast<int>(id64);
  const auto power = pref_power<E>(p, lse, g);
  bool owner = false;
  float part;
  if constexpr (SAME_PHASE)
    part = g > 0.f ? stream_span<E, THREADS, UNROLL, true, true, true>(in, out, sp, sn, idx, power, owner)
                   : stream_span<E, THREADS, UNROLL, true, false, true>(in, out, sp, sn, idx, power, owner);
  else
    part = g > 0.f ? pref_stream_shifted<E, THREADS, UNROLL, true>(in, out, sp, idx, power, owner)
                   : pref_stream_shifted<E, THREADS, UNROLL, false>(in, out, sp, idx, power, owner);
  const float total = block_sum_all<THREADS>(part);
  if (owner) E::store_scalar(out + idx, g > 0.f ? total : -total);
}

template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__global__ void __launch_bounds__(THREADS) pref_grad_kernel(const PrefParams p) {
  wait_for_previous_grids();
  const int64_t r = blockIdx.x;
  const int64_t b = r / p.x.L;
  const int64_t l = r - b * p.x.L;
  const bool live = p.mask == nullptr || p.mask[r] != 0;
  const int64_t id64 = p.idx[r];
  const float lse = p.lse[r];
  const float g = live ? p.coef[b] * p.dloss[b < p.pairs ? b : b - p.pairs] / p.T : 0.f;
  pref_grad_row<E, THREADS, UNROLL, SAME_PHASE>(p, b, l, g, id64, lse);
}

// Threads of a row's CTA: enough that the rows fill the SMs' 2048 threads (with a mask, half of the
// rows), so few rows go by large CTAs and many by small ones, down to 128 and to four vectors a thread.
// Forward, rows of 64 KB: 225 live ones of 600 by 512 threads 12.2 us, by 128 16.4; 6144 of 16384 by 128 72
// us, by 512 93.  Rows of 8 KB and less by 64.
inline int pref_threads(const PrefParams& p, int esize, int64_t rows, int sms) {
  const int64_t bytes = static_cast<int64_t>(p.x.V) * esize, fill = (p.mask ? 4096LL : 2048LL) * sms;
  if (bytes <= 8192) return 64;
  int t = 1024;
  while (t > 128 && (rows * t > fill || bytes < t * 64LL)) t /= 2;
  return t;
}

// A batch of whose rows L2 holds most until the backward (384 MB with a mask, which leaves a part of the rows, 192
// without) is read with priority to stay: 4 pairs of 512 tokens at V = 32000 bf16, both passes, 84.6 ->
// 81.3 us, 3 of 170 at V = 32003 fp32 50.7 -> 45.9; a larger one without: 16 pairs of 512 295 -> 292 us.  (How much a
// mask leaves is not known here.  Both passes over 260 and 340 MB at V = 32000 bf16: with priority up to 384 MB 82 and 110
// us where it leaves three eighths, 138 and 178 where it leaves all; up to 192 MB 87 and 112, 137 and 175.)
template <class E, int THREADS, int UNROLL>
cudaError_t launch_pref_rows_threads(const PrefParams& p, int64_t rows, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows));
  const int64_t bytes = rows * p.x.V * static_cast<int64_t>(sizeof(typename E::storage));
  return bytes <= (p.mask ? 384LL << 20 : 192LL << 20)
             ? launch_after_previous(pref_rows_kernel<E, THREADS, UNROLL, true>, grid, dim3(THREADS), s, p)
             : launch_after_previous(pref_rows_kernel<E, THREADS, UNROLL, false>, grid, dim3(THREADS), s, p);
}

template <class E>
cudaError_t launch_pref_rows(const PrefParams& p, int64_t rows, int sms, cudaStream_t s) {
  switch (pref_threads(p, sizeof(typename E::storage), rows, sms)) {
    case 1024: return launch_pref_rows_threads<E, 1024, 2>(p, rows, s);
    case 512: return launch_pref_rows_threads<E, 512, 2>(p, rows, s);
    case 256: return launch_pref_rows_threads<E, 256, kUnroll>(p, rows, s);
    case 128: return launch_pref_rows_threads<E, 128, kUnroll>(p, rows, s);
    default: return launch_pref_rows_threads<E, 64, kUnroll>(p, rows, s);
  }
}

template <class E, int THREADS, int UNROLL>
cudaError_t launch_pref_grad_threads(bool same_phase, const PrefParams& p, int64_t rows, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows));
  return same_phase ? launch_after_previous(pref_grad_kernel<E, THREADS, UNROLL, true>, grid, dim3(THREADS), s, p)
                    : launch_after_previous(pref_grad_kernel<E, THREADS, 2, false>, grid, dim3(THREADS), s, p);
}

template <class E>
cudaError_t launch_pref_grad(bool same_phase, const PrefParams& p, int64_t rows, int sms, cudaStream_t s) {
  switch (pref_threads(p, sizeof(typename E::storage), rows, sms)) {
    case 1024: return launch_pref_grad_threads<E, 1024, 2>(same_phase, p, rows, s);
    case 512: return launch_pref_grad_threads<E, 512, 2>(same_phase, p, rows, s);
    case 64: return launch_pref_grad_threads<E, 64, kUnroll>(same_phase, p, rows, s);
    default: return launch_pref_grad_threads<E, 256, kUnroll>(same_phase, p, rows, s);
  }
}

}  // namespace
}  // namespace grpo
