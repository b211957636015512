// The K largest log-probs of each row, log_softmax(x / T), with their columns: sorted, ties
// to the lowest column.
//
// A row is streamed once for the softmax statistic (logits_stat.cuh); the K largest are
// then found by radix selection on order-preserving keys of the logits: 8 bits of the key per
// sweep (two sweeps for bf16, four for fp32), then one sweep that collects the columns above
// the K-th key and one, in column order, that takes the ties.
#include "logits_ops.h"
#include "logits_stat.cuh"

namespace grpo {
namespace {

constexpr int kTopkThreads = 256;

// Order-preserving key of a float (-0 counts as +0), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// One 64-bit key in the order of the results: larger value first, then the lower column.
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int j) {
  return static_cast<uint64_t>(key) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}

// f(j, x_j) over the row, every thread taking its own columns.
template <class E, class F>
__device__ __forceinline__ void for_row(const typename E::storage* row, int V, F f) {
  const RowSplit sp = split_row<E>(row, V);
  const int tid = threadIdx.x;
  if (tid < sp.head) f(tid, E::load_scalar(row + tid));
  if (tid < sp.tail) {
    const int j = sp.head + sp.nvec * E::kVec + tid;
    f(j, E::load_scalar(row + j));
  }
  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  for (int i = tid; i < sp.nvec; i += kTopkThreads) {
    float v[E::kVec];
    E::unpack(ld_nc_v4(vb + i), v);
#pragma unroll
    for (int k = 0; k < E::kVec; ++k) f(sp.head + i * E::kVec + k, v[k]);
  }
}

// Radix selection of the K largest entries of the row into list[0..K) (any order).
template <class E>
__device__ void radix_select(const typename E::storage* row, int V, int K, uint64_t* list) {
  __shared__ unsigned hist[256];
  __shared__ unsigned sh_digit, sh_above, sh_n;
  __shared__ unsigned wsum[kTopkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPasses = sizeof(typename E::storage);  // the key's low half is fixed for bf16
  uint32_t prefix = 0u;
  unsigned need = static_cast<unsigned>(K);  // still to be taken among the keys with this prefix
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256; i += kTopkThreads) hist[i] = 0u;
    __syncthreads();
    for_row<E>(row, V, [&](int, float x) {
      const uint32_t k = key_of(x);
      if (pass == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[k >> shift & 255u], 1u);
    });
    __syncthreads();
    if (warp == 0) {  // lane t: digits 255 - 8 t .. 248 - 8 t, from the top
      unsigned c[8], sum = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) sum += c[q] = hist[255 - 8 * lane - q];
      unsigned before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (before < need && need <= before + c[q]) {
          sh_digit = 255u - 8u * lane - q;
          sh_above = before;
        }
        before += c[q];
      }
    }
    __syncthreads();
    prefix = prefix << 8 | sh_digit;
    need -= sh_above;
    __syncthreads();
  }
  constexpr int kShift = 32 - 8 * kPasses;
  if (tid == 0) sh_n = 0u;
  __syncthreads();
  for_row<E>(row, V, [&](int j, float x) {
    const uint32_t k = key_of(x);
    if ((k >> kShift) > prefix) list[atomicAdd(&sh_n, 1u)] = entry_of(k, j);
  });
  // the ties, in column order
  unsigned done = 0;
  for (int j0 = 0; j0 < V && done < need; j0 += kTopkThreads) {
    const int j = j0 + tid;
    uint32_t k = 0u;
    bool tie = false;
    if (j < V) {
      k = key_of(E::load_scalar(row + j));
      tie = (k >> kShift) == prefix;
    }
    const unsigned bal = __ballot_sync(0xFFFFFFFFu, tie);
    if (lane == 0) wsum[warp] = __popc(bal);
    __syncthreads();
    unsigned at = done + __popc(bal & ((1u << lane) - 1u));
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < kTopkThreads / 32; ++w) {
      if (w < warp) at += wsum[w];
      total += wsum[w];
    }
    if (tie && at < need) list[K - need + at] = entry_of(k, j);
    done += total;
    __syncthreads();
  }
  __syncthreads();
}

template <class E>
__global__ void __launch_bounds__(kTopkThreads) topk_kernel(const TopkParams p) {
  using S = typename E::storage;
  wait_for_previous_grids();
  __shared__ uint64_t list[kTopkMax];
  __shared__ float sh_m, sh_ln_s, sh_lse;
  const int64_t r = blockIdx.x;
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const int V = p.x.V, K = p.K, tid = threadIdx.x;
  const float c = p.c;

  MaxRun rs;
  const RowSplit sp = split_row<E>(row, V);
  if (tid < sp.head) maxrun_scalar(rs, E::load_scalar(row + tid), c);
  if (tid < sp.tail) maxrun_scalar(rs, E::load_scalar(row + sp.head + sp.nvec * E::kVec + tid), c);
  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  int i = tid;
  for (; i + (kUnroll - 1) * kTopkThreads < sp.nvec; i += kUnroll * kTopkThreads) {
    uint4 v[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) v[k] = ld_nc_v4(vb + i + k * kTopkThreads);
    maxrun_vectors<E>(rs, v, c);
  }
  for (; i < sp.nvec; i += kTopkThreads) {
    const uint4 v[1] = {ld_nc_v4(vb + i)};
    maxrun_vectors<E>(rs, v, c);
  }
  const MaxStat st = maxstat_block<kTopkThreads>(rs.stat(), c);
  if (tid == 0) {
    sh_m = st.m;
    sh_ln_s = logf(st.s);
    sh_lse = fmaf(st.m, p.invT, sh_ln_s);
    if (p.lse) p.lse[r] = sh_lse;
  }
  __syncthreads();
  int64_t* ids = p.ids + r * K;
  float* logp = p.logp + r * K;
  if (!isfinite(sh_lse)) {  // a NaN or +inf logit, or nothing but -inf: no log-prob is defined
    for (int k = tid; k < K; k += kTopkThreads) {
      ids[k] = k;
      logp[k] = __int_as_float(0x7FC00000);
    }
    return;
  }
  radix_select<E>(row, V, K, list);
  for (int k = tid; k < K; k += kTopkThreads) {  // each entry's rank is its place
    const uint64_t e = list[k];
    int rank = 0;
    for (int q = 0; q < K; ++q) rank += list[q] > e;
    ids[rank] = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(e));
    logp[rank] = fmaf(value_of(static_cast<uint32_t>(e >> 32)) - sh_m, p.invT, -sh_ln_s);
  }
}

}  // namespace

cudaError_t launch_topk(int dtype, const TopkParams& p, int64_t rows, int sms, cudaStream_t stream) {
  (void)sms;
  const dim3 grid(static_cast<unsigned>(rows)), block(kTopkThreads);
  return dtype == 1 ? launch_after_previous(topk_kernel<BF16>, grid, block, stream, p)
                    : launch_after_previous(topk_kernel<F32>, grid, block, stream, p);
}

}  // namespace grpo
