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
// row.  The gradient needs only which columns occur, and keeps no words.
//
// The pass is bound by HBM (read and write every logit once), so the stream over a row is a copy
// (with -inf or 0 where the mask forbids; vectors that it forbids whole are not read).  The touched
// columns, listed as they are first met, are written over the copy, a thread to each: within the
// stream nearly every warp met one, and its 32 lanes waited for it (1.24 ms against DUAL ms for
// forward and backward at (4, 1024, 151936) bf16).  Values are formed in fp32 from the whole count
// and rounded once.
#include "logits_load.cuh"
#include "logits_ops.h"
#include "rowpass_common.cuh"

namespace grpo {
namespace {

constexpr int kRulesThreads = 256;
constexpr int kTileVecs = 1024;  // vectors of a row per CTA, 4 per thread
constexpr int kPer = kTileVecs / kRulesThreads;
constexpr int kMaxRun = 32;      // rows per CTA
constexpr int kWindow = 256;     // tokens past the first row's history that are held ready
constexpr int kListed = 2048;    // touched columns that are listed; with more, the words are searched

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

__device__ __forceinline__ uint32_t word_of(const uint4& v, int k) {
  return k == 0 ? v.x : (k == 1 ? v.y : (k == 2 ? v.z : v.w));
}

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

// Grid: tiles x runs, tiles innermost.  run: rows per CTA, runs: runs per sequence.
// INPLACE: the output is the input, so only what changes is read and written.
template <class E, bool BWD, bool INPLACE>
__global__ void __launch_bounds__(kRulesThreads, 5) rules_kernel(const RulesParams p, int tiles, int run, int runs,
                                                                 bool same_phase) {
  constexpr int VEC = E::kVec, W = kTileVecs * VEC, COLS = W + VEC;  // a tile's last vector may reach past it
  constexpr int WORDS = BWD ? (COLS + 127) / 128 * 4 : (COLS + 3) / 4 * 4;
  using S = typename E::storage;
  extern __shared__ uint4 rules_smem[];  // forward: a word per column; backward: a bit
  __shared__ uint16_t listed[kListed];
  __shared__ int sh_touched;
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
    if (BWD) atomicOr(&words[col >> 5], 1u << (col & 31));
    else if (i < np) atomicOr(&words[col], kRulePrompt);
    else atomicAdd(&words[col], 1u);
  };
  auto is_touched = [&](int col) { return BWD ? (words[col >> 5] >> (col & 31) & 1u) != 0 : words[col] != 0u; };
  auto list = [&](int col) {
    const int at = atomicAdd(&sh_touched, 1);
    if (at < kListed) listed[at] = static_cast<uint16_t>(col);
  };
  // the tile's column of a token, -1 where it has none, -2 past the vocabulary
  auto col_of = [&](int64_t id) {
    if (static_cast<uint64_t>(id) >= static_cast<uint64_t>(V)) return id < 0 ? -1 : -2;
    const int col = static_cast<int>(id) - c0;
    return static_cast<unsigned>(col) < static_cast<unsigned>(COLS) ? col : -1;
  };
  int held = 0;  // the words hold the history's first `held` tokens; the window what follows `win`
  int win = 0;
  auto rebuild = [&](int n) {  // count the first n tokens
    __syncthreads();
    for (int i = tid; i < WORDS / 4; i += kRulesThreads) rules_smem[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) sh_touched = 0;
    __syncthreads();
    if (biased) {
      for (int m = tid; m < p.M; m += kRulesThreads) {
        const int col = col_of(p.bias_ids[b * p.M + m]);
        if (col == -2) bad_index();
        if (col < 0) continue;
        // a column listed twice: the last entry counts
        atomicMax(&words[col], static_cast<uint32_t>(m + 1) << kRuleBiasShift);
      }
      __syncthreads();
    }
    if (counted) {
      for (int i0 = tid; i0 < n; i0 += 4 * kRulesThreads) {
        int64_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = i0 + k * kRulesThreads < n ? tk[i0 + k * kRulesThreads] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = col_of(id[k]);
          if (col == -2) bad_index();
          if (col >= 0) add_token(col, i0 + k * kRulesThreads);
        }
      }
      if (nrows > 1 && tid < kWindow && n + tid < N) window[tid] = col_of(tk[n + tid]);
    }
    held = win = n;
    __syncthreads();
    for (int i = tid; i < WORDS / 4; i += kRulesThreads) {
      const uint4 v = rules_smem[i];
      if ((v.x | v.y | v.z | v.w) == 0u) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w = word_of(v, k);
        if (!BWD) {
          if (w != 0u) list(4 * i + k);
        } else {
          for (; w != 0u; w &= w - 1u) list(32 * (4 * i + k) + __ffs(w) - 1);
        }
      }
    }
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

  // the output may be the input where they are in phase
  auto load = [&](const S* body, int i, int nvec) {
    return same_phase ? ld_v4(reinterpret_cast<const uint4*>(body) + i) : load_out_of_phase<E>(body, i, nvec);
  };
  constexpr uint32_t kAll = (1u << VEC) - 1u;
  constexpr uint32_t kForbidden = BWD ? 0u : (sizeof(S) == 2 ? 0xFF80FF80u : 0xFF800000u);  // 0 or -inf
  for (int rr = 0; rr < nrows; ++rr) {
    const int64_t l = l0 + rr;
    S* out = static_cast<S*>(p.out.ptr) + b * p.out.sb + l * p.out.sl;
    const S* src = BWD ? static_cast<const S*>(p.dy.ptr) + b * p.dy.sb + l * p.dy.sl
                       : static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
    const uint32_t* m = p.allowed ? p.allowed + b * p.allowed_sb + l * p.allowed_sl : nullptr;
    const RowSplit sp = split_row<E>(out, V);
    // the row's part in this tile: vectors [i0, i1), 1024 at most; a vector belongs to the tile of
    // its first column
    const int i0 = c0 <= sp.head ? 0 : (c0 - sp.head + VEC - 1) / VEC;
    const int i1 = min(sp.nvec, (c0 + W - sp.head + VEC - 1) / VEC);

    // the vectors, and which of their columns are allowed (a byte each)
    uint32_t allowed = 0xFFFFFFFFu;
    if (m != nullptr) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = i0 + tid + k * kRulesThreads;
        if (i < i1) allowed ^= (bits_at(m, sp.head + i * VEC, mwords) & kAll ^ kAll) << (8 * k);
      }
    }
    auto full = [&](int k) { return (allowed >> (8 * k) & kAll) == kAll; };
    auto none = [&](int k) { return (allowed >> (8 * k) & kAll) == 0u; };
    uint4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + tid + k * kRulesThreads;
      if (i < i1 && !none(k) && !(INPLACE && full(k))) v[k] = load(src + sp.head, i, sp.nvec);
    }

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
          if (tid == 0) {
            if (!is_touched(col)) list(col);
            add_token(col, held);
          }
          __syncthreads();
        }
      }
    }

    // the touched column of this thread, loaded ahead of the copy
    const int nt = used ? sh_touched : 0;
    const S* x = BWD ? static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl : src;
    struct Hit {
      int j;  // the column, -1: none of this tile's, or forbidden
      int col;
      float f, x;
    };
    auto look = [&](int t) {
      Hit h{-1, t, 0.f, 0.f};
      if (nt <= kListed) h.col = listed[t];
      else if (!is_touched(t)) return h;
      const int j = c0 + h.col;
      if (j >= V) return h;
      int first = j;  // the column that decides whose it is
      if (j >= sp.head && j < sp.head + sp.nvec * VEC) first = j - (j - sp.head) % VEC;
      if (first < c0 || first >= c0 + W) return h;
      if (m != nullptr && (bits_at(m, j, mwords) & 1u) == 0) return h;
      h.f = E::load_scalar_coherent(src + j);
      if (BWD) h.x = E::load_scalar_coherent(x + j);
      h.j = j;
      return h;
    };
    const int todo = nt <= kListed ? nt : COLS;
    Hit mine{-1, 0, 0.f, 0.f};
    if (nt > 0 && tid < todo) mine = look(tid);

    // the copy: the scalar head and tail (at most one element per thread), then the vectors
    int edge = tid < sp.head ? tid : -1;
    if (tid >= kRulesThreads - sp.tail) edge = V - kRulesThreads + tid;
    if (edge >= c0 && edge < c0 + W) {
      if (m != nullptr && (bits_at(m, edge, mwords) & 1u) == 0) E::store_bits(out + edge, kForbidden);
      else if (!INPLACE) E::store_scalar(out + edge, E::load_scalar_coherent(src + edge));
    }
    uint4* ob = reinterpret_cast<uint4*>(out + sp.head);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + tid + k * kRulesThreads;
      if (i >= i1 || (INPLACE && full(k))) continue;
      if (!full(k)) {
        if (none(k)) v[k] = make_uint4(kForbidden, kForbidden, kForbidden, kForbidden);
        else forbid(v[k], allowed >> (8 * k), kForbidden, static_cast<E*>(nullptr));
      }
      st_v4_evict_first(ob + i, v[k]);
    }

    // the touched columns over the copy
    if (nt == 0) continue;
    __syncthreads();
    auto put = [&](const Hit& h) {
      if (h.j < 0) return;
      const float f = BWD ? (h.x > 0.f ? __fdiv_rn(h.f, q.rho) : h.f * q.rho) : apply_rules(q, h.f, words[h.col]);
      E::store_scalar(out + h.j, f);
    };
    put(mine);
    for (int t = tid + kRulesThreads; t < todo; t += kRulesThreads) put(look(t));
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
  const bool used = (p.tokens != nullptr && (!BWD || p.repetition != nullptr)) || (!BWD && p.M > 0);
  constexpr int most = BWD ? (COLS + 127) / 128 * 16 : (COLS + 3) / 4 * 16;
  static_assert(most < 40 * 1024, "with the static part within the 48 KB that need no leave");
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
