// The sampler's rules on logits (penalties for repeated tokens, biases, grammar masks) and
// their gradient.  With s_j / n_j whether column j occurs in the row's history and how often
// it was generated:
//
//   y_j  = s_j ? (x_j > 0 ? x_j / rho : x_j rho) : x_j;   y_j -= f n_j + a [n_j > 0];
//   y_j += bias_j;   y_j = -inf where the mask forbids j
//   dx_j = dy_j (s_j ? (x_j > 0 ? 1 / rho : rho) : 1),  0 where forbidden
//
// A CTA owns one tile of columns of a row: it counts the history into one 32-bit word per
// column in shared memory (logits_ops.h), then streams the tile.  Values are formed in fp32
// from the whole count and rounded once.
#include "logits_ops.h"
#include "rowpass_common.cuh"

namespace grpo {
namespace {

constexpr int kTileCols = 16384;  // 64 KB of words per CTA
constexpr int kRulesThreads = 256;

struct SeqRules {
  float rho, freq, pres;
  bool has_rep;
  const float* bias;
};

__device__ __forceinline__ bool in_history(uint32_t w) { return (w & ((1u << kRuleBiasShift) - 1)) != 0; }

__device__ __forceinline__ float apply_rules(const SeqRules& q, float x, uint32_t w) {
  if (q.has_rep && in_history(w)) x = x > 0.f ? __fdiv_rn(x, q.rho) : x * q.rho;
  const uint32_t n = w & (kRulePrompt - 1);
  if (n != 0) x = fmaf(-q.freq, static_cast<float>(n), x) - q.pres;
  const uint32_t at = w >> kRuleBiasShift;
  if (at != 0) x += q.bias[at - 1];
  return x;
}

// Bits [j, j + n) of the row's mask, n <= 8.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* m, int j, int words) {
  const int w = j >> 5;
  const uint32_t lo = __ldg(m + w);
  const uint32_t hi = w + 1 < words ? __ldg(m + w + 1) : 0u;
  return __funnelshift_r(lo, hi, j & 31);
}

template <class E>
__device__ __forceinline__ uint4 load_any(const typename E::storage* body, int i, bool same_phase) {
  if (same_phase) return ld_v4(reinterpret_cast<const uint4*>(body) + i);
  float f[E::kVec];
#pragma unroll
  for (int q = 0; q < E::kVec; ++q) f[q] = E::load_scalar_coherent(body + static_cast<int64_t>(i) * E::kVec + q);
  return E::pack(f, 0u);
}

template <class E, bool BWD>
__global__ void __launch_bounds__(kRulesThreads) rules_kernel(const RulesParams p, int tiles, int tile_vecs,
                                                              bool same_phase, bool in_place) {
  extern __shared__ uint32_t words[];
  wait_for_previous_grids();
  constexpr int VEC = E::kVec;
  using S = typename E::storage;
  const int tid = threadIdx.x;
  const int tile = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
  const int64_t r = blockIdx.x / static_cast<unsigned>(tiles);
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const int V = p.x.V;
  S* out = static_cast<S*>(p.out.ptr) + b * p.out.sb + l * p.out.sl;
  const S* x = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const S* src = BWD ? static_cast<const S*>(p.dy.ptr) + b * p.dy.sb + l * p.dy.sl : x;
  const RowSplit sp = split_row<E>(out, V);
  const int last = sp.nvec > 0 ? (sp.nvec - 1) / tile_vecs : 0;  // the tile that takes the row's tail
  if (tile > last) return;
  const int v0 = tile * tile_vecs;
  const int v1 = min(sp.nvec, v0 + tile_vecs);
  // columns [c0, c1) of this tile; word of column j: words[j - base]
  const int c0 = tile == 0 ? 0 : sp.head + v0 * VEC;
  const int c1 = tile == last ? V : sp.head + v1 * VEC;
  const int base = sp.head + v0 * VEC - VEC;

  const bool counted = p.tokens != nullptr;
  const bool used = counted || p.M > 0;
  SeqRules q;
  q.has_rep = counted && p.repetition != nullptr;
  q.rho = q.has_rep ? p.repetition[b] : 1.f;
  q.freq = counted && p.frequency ? p.frequency[b] : 0.f;
  q.pres = counted && p.presence ? p.presence[b] : 0.f;
  q.bias = p.bias + b * p.M;

  if (used) {
    for (int i = tid; i < tile_vecs * VEC + 2 * VEC; i += kRulesThreads) words[i] = 0u;
    __syncthreads();
    if (p.M > 0) {
      const int64_t* ids = p.bias_ids + b * p.M;
      for (int m = tid; m < p.M; m += kRulesThreads) {
        const int64_t id = ids[m];
        if (id >= V && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
        // a column listed twice: the last entry counts
        if (id >= c0 && id < c1) atomicMax(&words[id - base], static_cast<uint32_t>(m + 1) << kRuleBiasShift);
      }
      __syncthreads();
    }
    if (counted) {
      const int64_t* tk = p.tokens + b * p.tokens_stride;
      int64_t n = p.hist_len ? p.hist_len[r] : p.N;
      if (n < 0 || n > p.N) {
        if (tid == 0 && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
        n = n < 0 ? 0 : p.N;
      }
      const int64_t np = p.prompt_len ? p.prompt_len[b] : 0;
      for (int64_t i = tid; i < n; i += kRulesThreads) {
        const int64_t id = tk[i];
        if (id >= V && p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
        if (id < c0 || id >= c1) continue;
        if (i < np) atomicOr(&words[id - base], kRulePrompt);
        else atomicAdd(&words[id - base], 1u);
      }
      __syncthreads();
    }
  }

  const uint32_t* m = p.allowed ? p.allowed + b * p.allowed_sb + l * p.allowed_sl : nullptr;
  const int mwords = (V + 31) >> 5;
  auto scalar = [&](int j) {
    const uint32_t w = used ? words[j - base] : 0u;
    const bool ok = m == nullptr || (mask_bits(m, j, mwords) & 1u) != 0;
    float v;
    if (BWD) {
      v = 0.f;
      if (ok) {
        v = E::load_scalar_coherent(src + j);
        if (q.has_rep && in_history(w)) v = E::load_scalar_coherent(x + j) > 0.f ? __fdiv_rn(v, q.rho) : v * q.rho;
      }
    } else {
      v = ok ? apply_rules(q, E::load_scalar_coherent(x + j), w) : -INFINITY;
    }
    E::store_scalar(out + j, v);
  };
  if (tile == 0 && tid < sp.head) scalar(tid);
  if (tile == last && tid < sp.tail) scalar(sp.head + sp.nvec * VEC + tid);

  uint4* ob = reinterpret_cast<uint4*>(out + sp.head);
  const S* sb = src + sp.head;
  constexpr uint32_t kAll = (1u << VEC) - 1u;
  for (int i = v0 + tid; i < v1; i += kRulesThreads) {
    const int j = sp.head + i * VEC;
    uint32_t w[VEC];
    uint32_t any = 0u;
    if (used) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) any |= w[k] = words[j - base + k];
    }
    const uint32_t ok = m ? mask_bits(m, j, mwords) & kAll : kAll;
    if (in_place && any == 0u && ok == kAll) continue;  // the output is the input already
    float f[VEC];
    if (ok != 0u) E::unpack(load_any<E>(sb, i, same_phase), f);
    if (any != 0u) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (BWD) {
          if (q.has_rep && in_history(w[k]))
            f[k] = E::load_scalar_coherent(x + j + k) > 0.f ? __fdiv_rn(f[k], q.rho) : f[k] * q.rho;
        } else {
          f[k] = apply_rules(q, f[k], w[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (!(ok >> k & 1u)) f[k] = BWD ? 0.f : -INFINITY;
    st_v4_evict_first(ob + i, E::pack(f, 0u));
  }
}

template <class E, bool BWD>
cudaError_t launch_e(bool same_phase, bool in_place, const RulesParams& p, int64_t rows, cudaStream_t s) {
  constexpr int VEC = E::kVec;
  const int nvec = (p.x.V + VEC - 1) / VEC;
  const int tile_vecs = kTileCols / VEC;
  const int tiles = (nvec + tile_vecs - 1) / tile_vecs;
  const bool used = p.tokens != nullptr || p.M > 0;
  const size_t smem = used ? (static_cast<size_t>(kTileCols) + 2 * VEC) * 4 : 0;
  const cudaError_t e = cudaFuncSetAttribute(rules_kernel<E, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (kTileCols + 2 * VEC) * 4);
  if (e != cudaSuccess) return e;
  return launch_after_previous_smem(rules_kernel<E, BWD>, dim3(static_cast<unsigned>(rows * tiles)),
                                    dim3(kRulesThreads), smem, s, p, tiles, tile_vecs, same_phase, in_place);
}

}  // namespace

cudaError_t launch_rules(int dtype, bool bwd, bool same_phase, bool in_place, const RulesParams& p, int64_t rows,
                         int sms, cudaStream_t stream) {
  (void)sms;
  if (dtype == 1)
    return bwd ? launch_e<BF16, true>(same_phase, in_place, p, rows, stream)
               : launch_e<BF16, false>(same_phase, in_place, p, rows, stream);
  return bwd ? launch_e<F32, true>(same_phase, in_place, p, rows, stream)
             : launch_e<F32, false>(same_phase, in_place, p, rows, stream);
}

}  // namespace grpo
