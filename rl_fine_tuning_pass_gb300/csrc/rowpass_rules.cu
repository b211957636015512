// The sampler's rules on logits (penalties for repeated tokens, biases, grammar masks) and
// their gradient.  With s_j / n_j whether column j occurs in the row's history and how often
// it was generated:
//
//   y_j  = s_j ? (x_j > 0 ? x_j / rho : x_j rho) : x_j;   y_j -= f n_j + a [n_j > 0];
//   y_j += bias_j;   y_j = -inf where the mask forbids j
//   dx_j = dy_j (s_j ? (x_j > 0 ? 1 / rho : rho) : 1),  0 where forbidden
//
// A CTA takes one tile of columns (1024 vectors) of a run of rows of one sequence.  The history of
// the run's first row is counted into one 32-bit word per column in shared memory (logits_ops.h);
// from row to row only the tokens that have come in are added (a row whose history is shorter
// than the one before starts anew), so the history is read once per run and tile, not once per
// row.  A bitmap tells which columns have a word: a vector without one is copied as it is.  The
// gradient needs only which columns occur, so its bitmap is all that it keeps.
//
// The pass is bound by HBM (read and write every logit once): five CTAs per SM with four vectors in
// flight per thread cover its latency; vectors that the mask forbids whole are not read.  What
// touched columns need stands outside the stream in functions of its own: inlined, it filled the
// instruction cache and the stream waited for instructions.  Values are formed in fp32 from the
// whole count and rounded once.
#include "logits_ops.h"
#include "rowpass_common.cuh"

namespace grpo {
namespace {

constexpr int kRulesThreads = 256;
constexpr int kTileVecs = 1024;  // vectors of a row per CTA, 4 per thread
constexpr int kPer = kTileVecs / kRulesThreads;
constexpr int kMaxRun = 32;      // rows per CTA
constexpr int kWindow = 256;     // tokens past the first row's history that are held ready

struct SeqRules {
  float rho, freq, pres;
  bool has_rep;
  const float* bias;
};

__device__ __forceinline__ bool in_history(uint32_t w) { return (w & ((1u << kRuleBiasShift) - 1)) != 0; }

__device__ __noinline__ float apply_rules(const SeqRules q, float x, uint32_t w) {
  if (q.has_rep && in_history(w)) x = x > 0.f ? __fdiv_rn(x, q.rho) : x * q.rho;
  const uint32_t n = w & (kRulePrompt - 1);
  if (n != 0) x = fmaf(-q.freq, static_cast<float>(n), x) - q.pres;
  const uint32_t at = w >> kRuleBiasShift;
  if (at != 0) x += q.bias[at - 1];
  return x;
}

__device__ __noinline__ float apply_slope(float rho, float dy, float x) { return x > 0.f ? __fdiv_rn(dy, rho) : dy * rho; }

// Element e of a vector, read and replaced, without indexing registers.
__device__ __forceinline__ uint32_t word_of(const uint4& v, int k) {
  return k == 0 ? v.x : (k == 1 ? v.y : (k == 2 ? v.z : v.w));
}
__device__ __forceinline__ void set_word(uint4& v, int k, uint32_t w) {
  v.x = k == 0 ? w : v.x;
  v.y = k == 1 ? w : v.y;
  v.z = k == 2 ? w : v.z;
  v.w = k == 3 ? w : v.w;
}
__device__ __forceinline__ float get_elem(const uint4& v, int e, BF16*) {
  const uint32_t w = word_of(v, e >> 1);
  return e & 1 ? BF16::hi(w) : BF16::lo(w);
}
__device__ __forceinline__ float get_elem(const uint4& v, int e, F32*) { return __uint_as_float(word_of(v, e)); }
__device__ __forceinline__ void set_elem(uint4& v, int e, float f, BF16*) {
  const uint32_t h = BF16::pack2(f, 0.f) & 0xFFFFu, w = word_of(v, e >> 1);
  set_word(v, e >> 1, e & 1 ? (w & 0xFFFFu) | h << 16 : (w & 0xFFFF0000u) | h);
}
__device__ __forceinline__ void set_elem(uint4& v, int e, float f, F32*) { set_word(v, e, __float_as_uint(f)); }

// `fill` (a pair of equal elements, or one fp32) where ok's bit is 0.
__device__ __forceinline__ void forbid(uint4& v, uint32_t ok, uint32_t fill, BF16*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t keep = (ok >> (2 * k) & 1u) * 0xFFFFu | (ok >> (2 * k + 1) & 1u) * 0xFFFF0000u;
    w[k] = (w[k] & keep) | (fill & ~keep);
  }
}
__device__ __forceinline__ void forbid(uint4& v, uint32_t ok, uint32_t fill, F32*) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = ok >> k & 1u ? w[k] : fill;
}

// Bits j, j + 1, ... of a bitmap of `words` words (at least 25 of them, zeros past its end).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* m, int j, int words) {
  const int w = j >> 5;
  const uint32_t hi = w + 1 < words ? m[w + 1] : 0u;
  return __funnelshift_r(m[w], hi, j & 31);
}

template <class E>
__device__ __forceinline__ uint4 load_any(const typename E::storage* body, int i, bool same_phase) {
  if (same_phase) return ld_v4(reinterpret_cast<const uint4*>(body) + i);
  float f[E::kVec];
#pragma unroll
  for (int q = 0; q < E::kVec; ++q) f[q] = E::load_scalar_coherent(body + static_cast<int64_t>(i) * E::kVec + q);
  return E::pack(f, 0u);
}

// Grid: tiles x runs, tiles innermost.  run: rows per CTA, runs: runs per sequence.
// INPLACE: the output is the input, so only vectors that change are read and written.
template <class E, bool BWD, bool INPLACE>
__global__ void __launch_bounds__(kRulesThreads, 5) rules_kernel(const RulesParams p, int tiles, int run, int runs,
                                                                 bool same_phase) {
  constexpr int VEC = E::kVec, W = kTileVecs * VEC, COLS = W + VEC;  // a tile's last vector may reach past it
  constexpr int MAPW = (COLS + 31) / 32 + 1;
  using S = typename E::storage;
  extern __shared__ uint4 rules_smem[];  // words, one per column (forward)
  __shared__ uint32_t touched[MAPW];
  __shared__ int sh_len[kMaxRun];
  __shared__ int window[kWindow];
  uint32_t* words = reinterpret_cast<uint32_t*>(rules_smem);
  wait_for_previous_grids();
  const int tid = threadIdx.x;
  const int tile = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
  const int64_t seq_run = blockIdx.x / static_cast<unsigned>(tiles);
  const int64_t b = seq_run / runs;
  const int64_t l0 = (seq_run - b * runs) * run;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(run), p.x.L - l0));
  const int V = p.x.V, c0 = tile * W;

  const bool counted = p.tokens != nullptr && (!BWD || p.repetition != nullptr);
  const bool biased = !BWD && p.M > 0;
  const bool used = counted || biased;
  SeqRules q;
  q.has_rep = counted && p.repetition != nullptr;
  q.rho = q.has_rep ? p.repetition[b] : 1.f;
  q.freq = counted && p.frequency ? p.frequency[b] : 0.f;
  q.pres = counted && p.presence ? p.presence[b] : 0.f;
  q.bias = p.bias + b * p.M;
  const int64_t* tk = p.tokens + b * p.tokens_stride;
  const int N = static_cast<int>(p.N);
  const int np = !BWD && counted && p.prompt_len ? max(0, p.prompt_len[b]) : 0;
  const int mwords = (V + 31) >> 5;

  auto bad_index = [&]() {
    if (p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
  };
  auto add_token = [&](int col, int i) {  // column col of the tile, place i of the history
    if (!BWD) {
      if (i < np) atomicOr(&words[col], kRulePrompt);
      else atomicAdd(&words[col], 1u);
    }
    atomicOr(&touched[col >> 5], 1u << (col & 31));
  };
  // the tile's column of a token, or -1
  auto col_of = [&](int64_t id) {
    if (id >= V) bad_index();
    const int64_t col = id - c0;
    return id >= 0 && id < V && col >= 0 && col < COLS ? static_cast<int>(col) : -1;
  };
  int held = 0;  // the words hold the history's first `held` tokens; the window what follows `win`
  int win = 0;
  auto rebuild = [&](int n) {  // count the first n tokens
    __syncthreads();
    if (!BWD)
      for (int i = tid; i < (COLS + 3) / 4; i += kRulesThreads) rules_smem[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < MAPW; i += kRulesThreads) touched[i] = 0u;
    __syncthreads();
    if (biased) {
      for (int m = tid; m < p.M; m += kRulesThreads) {
        const int col = col_of(p.bias_ids[b * p.M + m]);
        if (col < 0) continue;
        // a column listed twice: the last entry counts
        atomicMax(&words[col], static_cast<uint32_t>(m + 1) << kRuleBiasShift);
        atomicOr(&touched[col >> 5], 1u << (col & 31));
      }
      __syncthreads();
    }
    if (counted) {
      int i = tid;
      for (; i + 3 * kRulesThreads < n; i += 4 * kRulesThreads) {
        int64_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = tk[i + k * kRulesThreads];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = col_of(id[k]);
          if (col >= 0) add_token(col, i + k * kRulesThreads);
        }
      }
      for (; i < n; i += kRulesThreads) {
        const int col = col_of(tk[i]);
        if (col >= 0) add_token(col, i);
      }
      if (nrows > 1 && tid < kWindow && n + tid < N) {
        const int64_t id = tk[n + tid];
        const int64_t col = id - c0;
        window[tid] = id >= V ? -2 : (id >= 0 && col >= 0 && col < COLS ? static_cast<int>(col) : -1);
      }
    }
    held = win = n;
    __syncthreads();
  };

  if (counted) {
    for (int i = tid; i < nrows; i += kRulesThreads) {
      int n = p.hist_len ? p.hist_len[b * p.x.L + l0 + i] : N;
      if (n < 0 || n > N) {
        bad_index();
        n = n < 0 ? 0 : N;
      }
      sh_len[i] = n;
    }
    __syncthreads();
  }

  // the row's part in this tile: vectors [i0, i1), 1024 at most
  struct Part {
    const S* src;
    const S* x;
    S* out;
    const uint32_t* m;
    RowSplit sp;
    int i0, i1;
  };
  auto part_of = [&](int rr) {
    const int64_t l = l0 + rr;
    Part t;
    t.out = static_cast<S*>(p.out.ptr) + b * p.out.sb + l * p.out.sl;
    t.x = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
    t.src = BWD ? static_cast<const S*>(p.dy.ptr) + b * p.dy.sb + l * p.dy.sl : t.x;
    t.m = p.allowed ? p.allowed + b * p.allowed_sb + l * p.allowed_sl : nullptr;
    t.sp = split_row<E>(t.out, V);
    // a vector belongs to the tile of its first column
    t.i0 = c0 <= t.sp.head ? 0 : (c0 - t.sp.head + VEC - 1) / VEC;
    t.i1 = min(t.sp.nvec, (c0 + W - t.sp.head + VEC - 1) / VEC);
    return t;
  };
  constexpr uint32_t kAll = (1u << VEC) - 1u;
  // the vectors and which of their columns are allowed (a byte each)
  auto load = [&](const Part& t, uint4 (&v)[kPer]) {
    uint32_t allowed = 0xFFFFFFFFu;
    if (t.m != nullptr) {
      allowed = 0u;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = t.i0 + tid + k * kRulesThreads;
        if (i < t.i1) allowed |= (bits_at(t.m, t.sp.head + i * VEC, mwords) & kAll) << (8 * k);
      }
    }
    if (INPLACE) return allowed;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = t.i0 + tid + k * kRulesThreads;
      v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i < t.i1 && (allowed >> (8 * k) & kAll) != 0u) v[k] = load_any<E>(t.src + t.sp.head, i, same_phase);
    }
    return allowed;
  };

  // a vector's touched columns, one after the other
  auto touch = [&](const Part& t, uint4& v, int j, uint32_t any) {
    while (any != 0u) {
      const int e = __ffs(any) - 1;
      any &= any - 1u;
      float f = get_elem(v, e, static_cast<E*>(nullptr));
      f = BWD ? apply_slope(q.rho, f, E::load_scalar_coherent(t.x + j + e)) : apply_rules(q, f, words[j - c0 + e]);
      set_elem(v, e, f, static_cast<E*>(nullptr));
    }
  };

  for (int rr = 0; rr < nrows; ++rr) {
    const Part cur = part_of(rr);
    uint4 v[kPer];
    const uint32_t allowed = load(cur, v);
    if (used) {
      const int n = counted ? sh_len[rr] : 0;
      if (rr == 0 || n < held || n > win + kWindow) {
        rebuild(n);
      } else {
        for (; held < n; ++held) {  // the same in every thread; a token of this tile is seldom
          const int col = window[held - win];
          if (col == -2) bad_index();
          if (col < 0) continue;
          __syncthreads();
          if (tid == 0) add_token(col, held);
          __syncthreads();
        }
      }
    }

    auto scalar = [&](int j) {
      const bool hit = used && (touched[(j - c0) >> 5] >> ((j - c0) & 31) & 1u);
      float f = BWD ? 0.f : -INFINITY;
      if (cur.m == nullptr || (bits_at(cur.m, j, mwords) & 1u) != 0) {
        f = E::load_scalar_coherent(cur.src + j);
        if (hit) f = BWD ? apply_slope(q.rho, f, E::load_scalar_coherent(cur.x + j)) : apply_rules(q, f, words[j - c0]);
      }
      E::store_scalar(cur.out + j, f);
    };
    // the scalar head and tail, at most one element per thread
    int edge = tid < cur.sp.head ? tid : -1;
    if (tid >= kRulesThreads - cur.sp.tail) edge = V - kRulesThreads + tid;
    if (edge >= c0 && edge < c0 + W) scalar(edge);

    uint4* ob = reinterpret_cast<uint4*>(cur.out + cur.sp.head);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = cur.i0 + tid + k * kRulesThreads;
      if (i >= cur.i1) continue;
      const int j = cur.sp.head + i * VEC;
      const uint32_t ok = allowed >> (8 * k) & kAll;
      const uint32_t any = used ? bits_at(touched, j - c0, MAPW) & ok : 0u;
      if (INPLACE) {
        if (any == 0u && ok == kAll) continue;  // the output is the input already
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (ok != 0u) v[k] = load_any<E>(cur.src + cur.sp.head, i, same_phase);
      }
      if (any != 0u) touch(cur, v[k], j, any);
      if (ok != kAll)
        forbid(v[k], ok, BWD ? 0u : (sizeof(S) == 2 ? 0xFF80FF80u : 0xFF800000u), static_cast<E*>(nullptr));
      st_v4_evict_first(ob + i, v[k]);
    }
  }
}

template <class E, bool BWD, bool INPLACE>
cudaError_t launch_e(bool same_phase, const RulesParams& p, int64_t rows, int sms, cudaStream_t s) {
  constexpr int W = kTileVecs * E::kVec, COLS = W + E::kVec;
  const int tiles = (p.x.V + W - 1) / W;
  // rows per CTA: long runs count the history seldom, but leave 6 CTAs or more for each place
  const int64_t places = 5LL * sms;
  int64_t run = rows * tiles / (6 * places);
  run = run < 1 ? 1 : (run > kMaxRun ? kMaxRun : run);
  if (run > p.x.L) run = p.x.L;
  const int64_t runs = (p.x.L + run - 1) / run;
  const bool used = !BWD && (p.tokens != nullptr || p.M > 0);
  const int most = (COLS + 3) / 4 * 16;
  const cudaError_t e = cudaFuncSetAttribute(rules_kernel<E, BWD, INPLACE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  const int64_t grid = rows / p.x.L * runs * tiles;
  return launch_after_previous_smem(rules_kernel<E, BWD, INPLACE>, dim3(static_cast<unsigned>(grid)),
                                    dim3(kRulesThreads), used ? most : 0, s, p, tiles, static_cast<int>(run),
                                    static_cast<int>(runs), same_phase);
}

template <class E>
cudaError_t launch_d(bool bwd, bool same_phase, bool in_place, const RulesParams& p, int64_t rows, int sms,
                     cudaStream_t s) {
  if (bwd) return in_place ? launch_e<E, true, true>(same_phase, p, rows, sms, s)
                           : launch_e<E, true, false>(same_phase, p, rows, sms, s);
  return in_place ? launch_e<E, false, true>(same_phase, p, rows, sms, s)
                  : launch_e<E, false, false>(same_phase, p, rows, sms, s);
}

}  // namespace

cudaError_t launch_rules(int dtype, bool bwd, bool same_phase, bool in_place, const RulesParams& p, int64_t rows,
                         int sms, cudaStream_t stream) {
  return dtype == 1 ? launch_d<BF16>(bwd, same_phase, in_place, p, rows, sms, stream)
                    : launch_d<F32>(bwd, same_phase, in_place, p, rows, sms, stream);
}

}  // namespace grpo
