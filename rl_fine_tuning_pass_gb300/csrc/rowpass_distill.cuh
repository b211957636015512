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
// the constant that leaves it near 0 where p_b is near q_b).  So the backward is the softmax stream of rowgrad_kernel with one factor per row, and K
// elements written after it.  p_rest is summed from the columns outside the list (a bitmap in
// shared memory leaves the listed ones out of the stream), not taken from 1 - sum p_k: it keeps
// its relative accuracy when the list holds nearly all of the mass.
#pragma once

#include "logits_ops.h"
#include "logits_stat.cuh"
#include "rowpass_bwd.cuh"

namespace grpo {
namespace {

constexpr int kBitmapBytes = 32768;      // 262144 columns; beyond, positions wrap and are checked
constexpr double kRestMin = 0x1p-20;     // least teacher mass outside the list

// The list of one row in shared memory.  id -1: an unused slot.
struct Slots {
  int* id;
  float* lq;  // teacher log-prob as given; later G_k - p_k S, scaled
  float* x;   // the student's logit
};

// Terms of one bucket: its part of the loss and G.  r = log q - log p, which carries the
// precision where p and q are near each other.
struct Term {
  float loss, G;
};
__device__ __forceinline__ Term bucket(float q, float p, float r, float beta) {
  Term t;
  if (beta == 0.f) {
    t.loss = q == 0.f ? 0.f : q * r;
    t.G = fabsf(r) < 0.5f ? -p * expm1f(r) : p - q;  // p (1 - q / p)
  } else if (beta == 1.f) {
    t.loss = t.G = p == 0.f ? 0.f : -p * r;
  } else {
    // log(p/m) and log(q/m) from r alone: m/p = 1 + beta (e^r - 1), m/q = 1 + (1 - beta)(e^-r - 1)
    float lpm, lqm;
    if (r <= 0.f) {
      lpm = -log1pf(beta * expm1f(r));
      lqm = r + lpm;
    } else {
      lqm = -log1pf((1.f - beta) * expm1f(-r));
      lpm = lqm - r;
    }
    t.G = p == 0.f ? 0.f : (1.f - beta) * p * lpm;
    t.loss = (q == 0.f ? 0.f : beta * q * lqm) + t.G;
  }
  return t;
}

// log(q / p) of the rest, from masses held in 64 bits.
__device__ __forceinline__ float rest_ratio(double q, double p) {
  const float d = static_cast<float>((q - p) / p);
  return fabsf(d) < 0.5f ? log1pf(d) : logf(static_cast<float>(q / p));
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

// What the teacher's list says: log q_k = lq_k - shift, and the mass outside the list.  One
// warp; the sums over the list in 64 bits, since q_rest = 1 - sum q_k cancels.
struct Teacher {
  double shift, q_rest;
};
__device__ __forceinline__ Teacher teacher_of(const Slots& sl, int K, int tail) {
  const int lane = threadIdx.x & 31;
  Teacher t{0.0, 0.0};
  if (tail) {
    double sum = 0.0;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) sum += exp(static_cast<double>(sl.lq[k]));
    sum = 1.0 - warp_sum(sum);
    t.q_rest = sum < kRestMin ? kRestMin : sum;  // a NaN stays one
  } else {
    float m = -INFINITY;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) m = fmaxf(m, sl.lq[k]);
    m = warp_max(m);
    float sum = 0.f;
    for (int k = lane; k < K; k += 32)
      if (sl.id[k] >= 0) sum += expf(sl.lq[k] - m);
    t.shift = static_cast<double>(m) + log(static_cast<double>(warp_sum(sum)));
  }
  return t;
}

// One row's results (every lane of the calling warp).
struct RowResult {
  float loss, lse, p_rest;
  float S, F_rest;  // sum of G, G_rest / p_rest
};

// The slots and the rest of a row, from the statistic `st` of the columns outside the list
// (every lane of one warp).  Log-probs of the buckets are formed in 64 bits: a divergence is
// a small difference of numbers around 10.
__device__ __forceinline__ RowResult finish_row(const Slots& sl, int K, const MaxStat& st, const DistillParams& p) {
  const int lane = threadIdx.x & 31;
  const Teacher te = teacher_of(sl, K, p.tail);
  float xm = -INFINITY;
  for (int k = lane; k < K; k += 32)
    if (sl.id[k] >= 0) xm = fmaxf(xm, sl.x[k]);
  xm = warp_max(xm);
  const bool any_rest = st.s != 0.f;
  const double a = static_cast<double>(st.m) * p.invT;
  double M = static_cast<double>(xm) * p.invT;
  if (any_rest && !(a < M)) M = a;
  const double s_rest = any_rest ? static_cast<double>(st.s) * exp(a - M) : 0.0;
  double s = 0.0;
  for (int k = lane; k < K; k += 32)
    if (sl.id[k] >= 0) s += static_cast<double>(expf(static_cast<float>(static_cast<double>(sl.x[k]) * p.invT - M)));
  s = s_rest + warp_sum(s);
  const double lse = M + log(s), inv_s = 1.0 / s;
  float loss = 0.f, S = 0.f;
  for (int k = lane; k < K; k += 32) {
    if (sl.id[k] < 0) continue;
    const double z = static_cast<double>(sl.x[k]) * p.invT;
    const float pk = static_cast<float>(static_cast<double>(expf(static_cast<float>(z - M))) * inv_s);
    const double lq = static_cast<double>(sl.lq[k]) - te.shift;
    const Term t = bucket(expf(static_cast<float>(lq)), pk, static_cast<float>(lq - (z - lse)), p.beta);
    loss += t.loss;
    S += t.G;
  }
  const double p_rest = s_rest * inv_s;
  const Term t = bucket(static_cast<float>(te.q_rest), static_cast<float>(p_rest), rest_ratio(te.q_rest, p_rest),
                        p.beta);
  RowResult o;
  o.lse = static_cast<float>(lse);
  // relative to the lse as it is stored: the backward's other p_j are too, and a common factor
  // cancels in its differences
  const float d_lse = static_cast<float>(lse - static_cast<double>(o.lse));
  o.p_rest = static_cast<float>(p_rest + p_rest * static_cast<double>(d_lse));
  o.loss = warp_sum(loss) + t.loss;
  o.S = warp_sum(S) + t.G;
  o.F_rest = p_rest == 0.0 ? 0.f : t.G / static_cast<float>(p_rest);
  return o;
}

// Load the row's list: ids (checked), teacher log-probs and the student's logits.  Returns
// whether this thread met an id >= V.
template <class E, int THREADS>
__device__ __forceinline__ bool load_slots(const Slots& sl, const DistillParams& p, int64_t r,
                                           const typename E::storage* row) {
  bool bad = false;
  for (int k = threadIdx.x; k < p.K; k += THREADS) {
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

template <class E, int THREADS, int UNROLL>
__global__ void __launch_bounds__(THREADS) distill_fwd_kernel(const DistillParams p, int bm_bytes) {
  using S = typename E::storage;
  extern __shared__ uint4 distill_smem[];
  __shared__ int sh_bad;
  wait_for_previous_grids();
  const int64_t r = blockIdx.x;
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const int tid = threadIdx.x, V = p.x.V, K = p.K;
  if (p.mask != nullptr && p.mask[r] == 0) {
    if (tid == 0) {
      p.loss[r] = 0.f;
      p.lse[r] = 0.f;
      p.p_rest[r] = 0.f;
    }
    return;
  }
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const RowSplit sp = split_row<E>(row, V);
  Slots sl;
  sl.id = reinterpret_cast<int*>(reinterpret_cast<char*>(distill_smem) + bm_bytes);
  sl.lq = reinterpret_cast<float*>(sl.id + K);
  sl.x = sl.lq + K;
  Bitmap<E> bm;
  bm.w = reinterpret_cast<uint32_t*>(distill_smem);
  bm.mask = V + 2 * E::kVec > bm_bytes * 8 ? static_cast<uint32_t>(bm_bytes) * 8u - 1u : 0xFFFFFFFFu;
  bm.head = sp.head;

  for (int i = tid; i < bm_bytes / 16; i += THREADS) distill_smem[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) sh_bad = 0;
  bool bad = load_slots<E, THREADS>(sl, p, r, row);
  if (bad && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
  __syncthreads();
  for (int k = tid; k < K; k += THREADS) {
    const int id = sl.id[k];
    if (id < 0 || !bm.set(id)) continue;
    bool twice = !bm.wraps();
    for (int q = 0; !twice && q < K; ++q) twice = q != k && sl.id[q] == id;
    if (twice && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_DUPLICATE_ID_BIT);
    bad |= twice;
  }
  if (bad) sh_bad = 1;
  __syncthreads();

  const float c = p.c;
  MaxRun rs;
  auto scalar = [&](int j) {
    if (bm.get(j) && (!bm.wraps() || listed_bits(sl, K, j, 1))) return;
    maxrun_scalar(rs, E::load_scalar(row + j), c);
  };
  if (tid < sp.head) scalar(tid);
  if (tid < sp.tail) scalar(sp.head + sp.nvec * E::kVec + tid);
  auto leave_out = [&](uint4& v, int i) {
    uint32_t bits = bm.vec(i);
    if (bits != 0u) {
      if (bm.wraps()) bits = listed_bits(sl, K, sp.head + i * E::kVec, E::kVec);
      drop(v, bits, static_cast<E*>(nullptr));
    }
  };
  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  int i = tid;
  for (; i + (UNROLL - 1) * THREADS < sp.nvec; i += UNROLL * THREADS) {
    uint4 v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) v[k] = ld_nc_v4(vb + i + k * THREADS);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) leave_out(v[k], i + k * THREADS);
    maxrun_vectors<E>(rs, v, c);
  }
  for (; i < sp.nvec; i += THREADS) {
    uint4 v[1] = {ld_nc_v4(vb + i)};
    leave_out(v[0], i);
    maxrun_vectors<E>(rs, v, c);
  }
  const MaxStat st = maxstat_block<THREADS>(rs.stat(), c);
  if (tid >= 32) return;
  const RowResult o = finish_row(sl, K, st, p);
  if (tid == 0) {
    const float nan = __int_as_float(0x7FC00000);
    p.loss[r] = sh_bad ? nan : o.loss;
    p.lse[r] = sh_bad ? nan : o.lse;
    p.p_rest[r] = sh_bad ? nan : o.p_rest;
  }
}

// out_j = f 2^((x_j - x0) c) over the row.
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__device__ __forceinline__ void grad_stream(const typename E::storage* in, typename E::storage* out,
                                            const RowSplit& sp, float x0, float c, float f) {
  const int tid = threadIdx.x;
  auto scalar = [&](int j) { E::store_scalar(out + j, f * ex2((E::load_scalar_coherent(in + j) - x0) * c)); };
  if (tid < sp.head) scalar(tid);
  if (tid < sp.tail) scalar(sp.head + sp.nvec * E::kVec + tid);
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
  int i = tid;
  for (; i + (UNROLL - 1) * THREADS < sp.nvec; i += UNROLL * THREADS) {
    uint4 v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) v[k] = load_vec<E, SAME_PHASE, true>(ib, i + k * THREADS);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) process(v[k], i + k * THREADS);
  }
  for (; i < sp.nvec; i += THREADS) process(load_vec<E, SAME_PHASE, true>(ib, i), i);
}

// The backward: one warp works out the row's factor and the listed columns' gradients while
// they are few, then the row is streamed as in rowgrad_kernel.
template <class E, int THREADS, int UNROLL, bool SAME_PHASE>
__global__ void __launch_bounds__(THREADS) distill_bwd_kernel(const DistillParams p) {
  using S = typename E::storage;
  extern __shared__ uint4 distill_smem[];
  __shared__ float sh_factor, sh_x0;
  wait_for_previous_grids();
  const int64_t r = blockIdx.x;
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const int tid = threadIdx.x, V = p.x.V, K = p.K;
  const bool live = p.mask == nullptr || p.mask[r] != 0;
  const float g = live ? p.dloss[r] / p.T : 0.f;
  const float lse = p.lse[r], p_rest = p.p_rest[r];
  S* out = static_cast<S*>(p.dx.ptr) + b * p.dx.sb + l * p.dx.sl;
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const RowSplit sp = split_row<E>(out, V);
  const Span sn = whole_row(sp);
  if (g == 0.f) {
    fill_span<E, THREADS>(out, sp, sn, 0u);
    return;
  }
  Slots sl;
  sl.id = reinterpret_cast<int*>(distill_smem);
  sl.lq = reinterpret_cast<float*>(sl.id + K);
  sl.x = sl.lq + K;
  load_slots<E, THREADS>(sl, p, r, row);
  __syncthreads();
  if (tid < 32) {
    const Teacher te = teacher_of(sl, K, p.tail);
    float S_sum = 0.f;
    const double lse_d = static_cast<double>(lse);
    for (int k = tid; k < K; k += 32) {
      if (sl.id[k] < 0) continue;
      const double lp = static_cast<double>(sl.x[k]) * p.invT - lse_d;
      const double lq = static_cast<double>(sl.lq[k]) - te.shift;
      const float pk = expf(static_cast<float>(lp));
      const Term t = bucket(expf(static_cast<float>(lq)), pk, static_cast<float>(lq - lp), p.beta);
      S_sum += t.G;
      sl.x[k] = pk;
      sl.lq[k] = t.G;
    }
    const Term t = bucket(static_cast<float>(te.q_rest), p_rest, rest_ratio(te.q_rest, static_cast<double>(p_rest)),
                          p.beta);
    S_sum = warp_sum(S_sum) + t.G;
    for (int k = tid; k < K; k += 32) sl.lq[k] = g * (sl.lq[k] - sl.x[k] * S_sum);
    // p_j = 2^((x_j - x0) c) e^(x0 / T - lse): x0 takes up lse, so that no exponent is a small
    // difference of large products
    if (tid == 0) {
      const float x0 = static_cast<float>(lse_d * static_cast<double>(p.T));
      const float scale = expf(static_cast<float>(static_cast<double>(x0) * p.invT - lse_d));
      sh_factor = g * ((p_rest == 0.f ? 0.f : t.G / p_rest) - S_sum) * scale;
      sh_x0 = x0;
    }
  }
  __syncthreads();
  const float f = sh_factor;
  if (f == 0.f) fill_span<E, THREADS>(out, sp, sn, 0u);
  else grad_stream<E, THREADS, UNROLL, SAME_PHASE>(row, out, sp, sh_x0, p.c, f);
  __syncthreads();  // the listed columns' values go over the stream's
  for (int k = tid; k < K; k += THREADS)
    if (sl.id[k] >= 0) E::store_scalar(out + sl.id[k], sl.lq[k]);
}

template <class E, int THREADS, int U>
cudaError_t launch_distill_fwd_t(const DistillParams& p, int64_t rows, cudaStream_t s) {
  const int bm = bitmap_bytes<E>(p.x.V);
  return launch_after_previous_smem(distill_fwd_kernel<E, THREADS, U>, dim3(static_cast<unsigned>(rows)),
                                    dim3(THREADS), static_cast<size_t>(bm) + 12 * p.K, s, p, bm);
}

template <class E>
cudaError_t launch_distill_fwd_e(const DistillParams& p, int64_t rows, int sms, cudaStream_t s) {
  switch (pick_threads_fwd(p.x.V, sizeof(typename E::storage), rows, sms)) {
    case 64: return launch_distill_fwd_t<E, 64, kUnroll>(p, rows, s);
    case 128: return launch_distill_fwd_t<E, 128, 2>(p, rows, s);
    default: return launch_distill_fwd_t<E, 256, kUnroll>(p, rows, s);
  }
}

template <class E, int THREADS>
cudaError_t launch_distill_bwd_t(bool same_phase, const DistillParams& p, int64_t rows, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(rows)), block(THREADS);
  const size_t smem = 12 * static_cast<size_t>(p.K);
  return same_phase ? launch_after_previous_smem(distill_bwd_kernel<E, THREADS, kUnroll, true>, grid, block, smem, s, p)
                    : launch_after_previous_smem(distill_bwd_kernel<E, THREADS, kUnroll, false>, grid, block, smem, s,
                                                 p);
}

template <class E>
cudaError_t launch_distill_bwd_e(bool same_phase, const DistillParams& p, int64_t rows, int sms, cudaStream_t s) {
  return pick_threads_bwd(p.x.V, sizeof(typename E::storage), rows, sms) == 64
             ? launch_distill_bwd_t<E, 64>(same_phase, p, rows, s)
             : launch_distill_bwd_t<E, 256>(same_phase, p, rows, s);
}

}  // namespace
}  // namespace grpo
