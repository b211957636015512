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
// row (without runs: 2.29 ms for forward and backward at (4, 1024, 151936) bf16, with them 1.66 ms).
// The gradient needs only which columns occur, and keeps no words but bits.
//
// The pass is bound by HBM (read and write every logit once), so the stream over a row is a copy,
// and the touched columns, listed once their run's history is counted, are changed by a thread each:
// within the stream nearly every warp met one, and its 32 lanes waited for it (1.24 ms; 1.07 ms with
// the list).
//   rules_bulk_kernel  input and output in phase: bulk copies (TMA) into a ring of shared memory and
//                      out of it; mask and touched columns are seen to there in between (0.79 ms,
//                      6.3 TB/s of the two passes' 4.98 GB).
//   rules_kernel       in place, out of phase, and where launch_e says so: the copy goes through
//                      registers, with -inf or 0 where the mask forbids (vectors that it forbids whole
//                      are not read), and the touched columns are written over it.
// Values are formed in fp32 from the whole count and rounded once.
#include "logits_load.cuh"
#include "logits_ops.h"
#include "logits_tma.cuh"
#include "rowpass_common.cuh"

namespace grpo {
namespace {

constexpr int kRulesThreads = 256;
constexpr int kTileVecs = 1024;  // vectors of a row per CTA, 4 per thread
constexpr int kPer = kTileVecs / kRulesThreads;
constexpr int kMaxRun = 8;       // rows per CTA
constexpr int kBulkRun = 4;      // rows per CTA from which the forward takes the bulk kernel's ring
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

// An element in shared memory.
template <class E>
__device__ __forceinline__ float load_shared(const typename E::storage* p) {
  if constexpr (sizeof(typename E::storage) == 2) return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  else return *p;
}

// Bits j, j + 1, ... of a bitmap of `words` words (at least 25 of them, zeros past its end).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* m, int j, int words) {
  const int w = j >> 5;
  const uint32_t hi = w + 1 < words ? m[w + 1] : 0u;
  return __funnelshift_r(m[w], hi, j & 31);
}

// The tile's share of a sequence's history and biases: words (forward: one per column; backward:
// a bit per column) and the list of touched columns, for the row that the CTA is at.
template <class E, bool BWD>
struct History {
  static constexpr int VEC = E::kVec, T = kRulesThreads;
  static constexpr int W = kTileVecs * VEC, COLS = W + VEC;  // a tile's last vector may reach past it
  static constexpr int WORDS = BWD ? (COLS + 127) / 128 * 4 : (COLS + 3) / 4 * 4;
  struct Shared {
    uint16_t listed[kListed];
    int touched;
    int len[kMaxRun];
    int window[kWindow];
  };
  const RulesParams& p;
  Shared& sh;
  uint32_t* words;
  int64_t b;
  const int64_t* tk;
  int c0, nrows, N, np;
  bool counted, biased;
  SeqRules q;
  int held = 0, win = 0;  // the words hold the first `held` tokens, the window what follows `win`
  int first_len = 0;
  int64_t pre_token[4], pre_bias;  // of the first count, loaded ahead

  __device__ __forceinline__ History(const RulesParams& p_, Shared& sh_, uint32_t* words_, int64_t b_, int64_t l0,
                                     int nrows_, int c0_)
      : p(p_), sh(sh_), words(words_), b(b_), c0(c0_), nrows(nrows_) {
    const int tid = threadIdx.x;
    counted = p.tokens != nullptr && (!BWD || p.repetition != nullptr);
    biased = !BWD && p.M > 0;
    tk = p.tokens + b * p.tokens_stride;
    N = static_cast<int>(p.N);
    if (counted) {
      const int64_t r = b * p.x.L + l0;
      first_len = length(p.hist_len ? p.hist_len[r] : N);
      for (int i = tid; i < nrows; i += T) sh.len[i] = length(p.hist_len ? p.hist_len[r + i] : N);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) pre_token[k] = counted && tid + k * T < N ? tk[tid + k * T] : -1;
    pre_bias = biased && tid < p.M ? p.bias_ids[b * p.M + tid] : -1;
    np = !BWD && counted && p.prompt_len ? max(0, p.prompt_len[b]) : 0;
    q.has_rep = counted && p.repetition != nullptr;
    q.rho = q.has_rep ? p.repetition[b] : 1.f;
    q.freq = counted && p.frequency ? p.frequency[b] : 0.f;
    q.pres = counted && p.presence ? p.presence[b] : 0.f;
    q.bias = p.bias + b * p.M;
  }
  __device__ __forceinline__ bool used() const { return counted || biased; }
  __device__ __forceinline__ void bad_index() const {
    if (p.dev_err) atomicOr(p.dev_err, GRPO_DEVERR_IDX_OUT_OF_RANGE_BIT);
  }
  __device__ __forceinline__ int length(int n) const {
    if (n >= 0 && n <= N) return n;
    bad_index();
    return n < 0 ? 0 : N;
  }
  // the tile's column of a token, -1 where it has none, -2 past the vocabulary
  __device__ __forceinline__ int col_of(int64_t id) const {
    if (static_cast<uint64_t>(id) >= static_cast<uint64_t>(p.x.V)) return id < 0 ? -1 : -2;
    const int col = static_cast<int>(id) - c0;
    return static_cast<unsigned>(col) < static_cast<unsigned>(COLS) ? col : -1;
  }
  __device__ __forceinline__ bool is_touched(int col) const {
    return BWD ? (words[col >> 5] >> (col & 31) & 1u) != 0 : words[col] != 0u;
  }
  __device__ __forceinline__ void add(int col, int i) const {  // place i of the history
    if (BWD) atomicOr(&words[col >> 5], 1u << (col & 31));
    else if (i < np) atomicOr(&words[col], kRulePrompt);
    else atomicAdd(&words[col], 1u);
  }
  __device__ __forceinline__ void count(int64_t id, int i) const {
    const int col = col_of(id);
    if (col == -2) bad_index();
    if (col >= 0) add(col, i);
  }
  __device__ __forceinline__ void put_bias(int64_t id, int m) const {
    const int col = col_of(id);
    if (col == -2) bad_index();
    // a column listed twice: the last entry counts
    if (col >= 0) atomicMax(&words[col], static_cast<uint32_t>(m + 1) << kRuleBiasShift);
  }

  // Places for this thread's n entries of the list (all threads of the warp call).
  __device__ __forceinline__ int reserve(int n) const {
    const int lane = threadIdx.x & 31;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    int base = 0;
    if (lane == 31 && sum > 0) base = atomicAdd(&sh.touched, sum);
    return __shfl_sync(0xFFFFFFFFu, base, 31) + sum - n;
  }

  // Count the first n tokens; FIRST: the row is the run's first, its loads are under way.
  template <bool FIRST>
  __device__ __forceinline__ void rebuild(int n) {
    const int tid = threadIdx.x;
    if (!FIRST) __syncthreads();
    uint4* quads = reinterpret_cast<uint4*>(words);
    for (int i = tid; i < WORDS / 4; i += T) quads[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) sh.touched = 0;
    __syncthreads();
    if (biased) {
      if (FIRST) put_bias(pre_bias, tid);
      for (int m = FIRST ? tid + T : tid; m < p.M; m += T) put_bias(p.bias_ids[b * p.M + m], m);
      __syncthreads();
    }
    if (counted) {
      int i0 = tid;
      if (FIRST) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (tid + k * T < n) count(pre_token[k], tid + k * T);
        i0 += 4 * T;
      }
      for (; i0 < n; i0 += 4 * T) {
        int64_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = i0 + k * T < n ? tk[i0 + k * T] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) count(id[k], i0 + k * T);
      }
      if (nrows > 1 && tid < kWindow && n + tid < N) sh.window[tid] = col_of(tk[n + tid]);
    }
    held = win = n;
    __syncthreads();
    if (!BWD) {  // a thread's quads of words: which words are not 0
      constexpr int kQuads = (WORDS / 4 + T - 1) / T;
      static_assert(4 * kQuads <= 64, "one mask per thread");
      uint64_t hit = 0u;
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int i = tid + k * T;
        if (i >= WORDS / 4) break;
        const uint4 v = quads[i];
        const uint32_t four = (v.x != 0u) | (v.y != 0u) << 1 | (v.z != 0u) << 2 | (v.w != 0u) << 3;
        hit |= static_cast<uint64_t>(four) << (4 * k);
      }
      int at = reserve(__popcll(hit));
      for (; hit != 0u; hit &= hit - 1u, ++at) {
        const int e = __ffsll(static_cast<long long>(hit)) - 1;
        if (at < kListed) sh.listed[at] = static_cast<uint16_t>(4 * (tid + (e >> 2) * T) + (e & 3));
      }
    } else {
      for (int i0 = 0; i0 < WORDS; i0 += T) {
        uint32_t w = i0 + tid < WORDS ? words[i0 + tid] : 0u;
        int at = reserve(__popc(w));
        for (; w != 0u; w &= w - 1u, ++at)
          if (at < kListed) sh.listed[at] = static_cast<uint16_t>(32 * (i0 + tid) + __ffs(w) - 1);
      }
    }
    __syncthreads();
  }

  // Go to the run's row rr (all threads; they take the same way).
  __device__ __forceinline__ void go_to(int rr) {
    if (!used()) return;
    if (rr == 0) {
      rebuild<true>(first_len);
      return;
    }
    if (!counted) return;
    const int n = sh.len[rr];
    if (n < held || n > win + kWindow) {
      rebuild<false>(n);
      return;
    }
    for (; held < n; ++held) {  // a token of this tile is seldom
      const int col = sh.window[held - win];
      if (col == -2) bad_index();
      if (col < 0) continue;
      __syncthreads();
      if (threadIdx.x == 0) {
        if (!is_touched(col)) {
          const int at = sh.touched++;
          if (at < kListed) sh.listed[at] = static_cast<uint16_t>(col);
        }
        add(col, held);
      }
      __syncthreads();
    }
  }
  // Touched columns: t < todo() and col_at(t) >= 0.
  __device__ __forceinline__ int todo() const {
    const int n = used() ? sh.touched : 0;
    return n <= kListed ? n : COLS;
  }
  __device__ __forceinline__ int col_at(int t) const {
    return sh.touched <= kListed ? sh.listed[t] : (is_touched(t) ? t : -1);
  }
  // The value of touched column col: from the logit, or (backward) from the gradient and the logit.
  __device__ __forceinline__ float value(int col, float f, float x) const {
    if (BWD) return x > 0.f ? __fdiv_rn(f, q.rho) : f * q.rho;
    return apply_rules(q, f, words[col]);
  }
};

// A row's part in a tile: vectors [i0, i1), 1024 at most; a vector belongs to the tile of its first
// column.
struct Part {
  RowSplit sp;
  int i0, i1;
};
template <class E>
__device__ __forceinline__ Part part_of(const void* out, int V, int c0) {
  constexpr int VEC = E::kVec, W = kTileVecs * VEC;
  Part t;
  t.sp = split_row<E>(out, V);
  t.i0 = c0 <= t.sp.head ? 0 : (c0 - t.sp.head + VEC - 1) / VEC;
  t.i1 = min(t.sp.nvec, (c0 + W - t.sp.head + VEC - 1) / VEC);
  return t;
}
// The element of the row's scalar head or tail that this thread has in the tile, or -1.
__device__ __forceinline__ int edge_of(const Part& t, int V, int c0, int W) {
  const int tid = threadIdx.x;
  int edge = tid < t.sp.head ? tid : -1;
  if (tid >= kRulesThreads - t.sp.tail) edge = V - kRulesThreads + tid;
  return edge >= c0 && edge < c0 + W ? edge : -1;
}

// 0 or -inf, in the format of forbid
template <class E, bool BWD>
constexpr uint32_t kForbiddenOf = BWD ? 0u : (sizeof(typename E::storage) == 2 ? 0xFF80FF80u : 0xFF800000u);

// Which columns of this thread's vectors i0 + tid + k kRulesThreads < i1 are allowed, a byte each.
template <class E>
__device__ __forceinline__ uint32_t allowed_of(const uint32_t* m, int head, int i0, int i1, int mwords) {
  constexpr uint32_t kAll = (1u << E::kVec) - 1u;
  uint32_t allowed = 0xFFFFFFFFu;
  if (m != nullptr) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + static_cast<int>(threadIdx.x) + k * kRulesThreads;
      if (i < i1) allowed ^= (bits_at(m, head + i * E::kVec, mwords) & kAll ^ kAll) << (8 * k);
    }
  }
  return allowed;
}

// Grid: tiles x runs, tiles innermost.  run: rows per CTA, runs: runs per sequence.
// HOW: the input and output rows.
enum RulesHow : int {
  kInPlace = 0,     // the same memory: only what changes is read and written
  kInPhase = 1,     // equal addresses mod 16
  kOutOfPhase = 2,  // others
};
template <class E, bool BWD, int HOW>
__global__ void __launch_bounds__(kRulesThreads, BWD ? 4 : 3) rules_kernel(const RulesParams p, int tiles, int run, int runs) {
  constexpr bool INPLACE = HOW == kInPlace;
  using H = History<E, BWD>;
  using S = typename E::storage;
  constexpr int VEC = E::kVec, W = H::W;
  extern __shared__ uint4 rules_smem[];
  __shared__ typename H::Shared sh;
  wait_for_previous_grids();
  const int tid = threadIdx.x;
  const int c0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles)) * W;
  const unsigned seq_run = blockIdx.x / static_cast<unsigned>(tiles);
  const int64_t b = seq_run / static_cast<unsigned>(runs);
  const int64_t l0 = static_cast<int64_t>(seq_run % static_cast<unsigned>(runs)) * run;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(run), p.x.L - l0));
  const int V = p.x.V, mwords = (V + 31) >> 5;
  H h(p, sh, reinterpret_cast<uint32_t*>(rules_smem), b, l0, nrows, c0);

  constexpr uint32_t kAll = (1u << VEC) - 1u;
  constexpr uint32_t kForbidden = kForbiddenOf<E, BWD>;
  for (int rr = 0; rr < nrows; ++rr) {
    const int64_t l = l0 + rr;
    S* out = static_cast<S*>(p.out.ptr) + b * p.out.sb + l * p.out.sl;
    const S* src = BWD ? static_cast<const S*>(p.dy.ptr) + b * p.dy.sb + l * p.dy.sl
                       : static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
    const uint32_t* m = p.allowed ? p.allowed + b * p.allowed_sb + l * p.allowed_sl : nullptr;
    const Part part = part_of<E>(out, V, c0);
    const RowSplit sp = part.sp;
    const int i0 = part.i0, i1 = part.i1;

    // the vectors, and which of their columns are allowed (a byte each)
    uint4 v[kPer];
    if constexpr (HOW == kOutOfPhase)
      load_out_of_phase<E, kPer, kRulesThreads>(v, src + sp.head, i0 + tid, i1, sp.nvec);
    const uint32_t allowed = allowed_of<E>(m, sp.head, i0, i1, mwords);
    auto full = [&](int k) { return (allowed >> (8 * k) & kAll) == kAll; };
    auto none = [&](int k) { return (allowed >> (8 * k) & kAll) == 0u; };
    if constexpr (HOW != kOutOfPhase) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = i0 + tid + k * kRulesThreads;
        if (i < i1 && !none(k) && !(INPLACE && full(k))) v[k] = ld_v4(reinterpret_cast<const uint4*>(src + sp.head) + i);
      }
    }
    h.go_to(rr);

    // the touched column of this thread, loaded ahead of the copy
    const int todo = h.todo();
    const S* x = BWD ? static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl : src;
    struct Hit {
      int j;  // the column, -1: none of this tile's, or forbidden
      int col;
      float f, x;
    };
    auto look = [&](int t) {
      Hit a{-1, h.col_at(t), 0.f, 0.f};
      const int j = c0 + a.col;
      if (a.col < 0 || j >= V) return a;
      int first = j;  // the column that decides whose it is
      if (j >= sp.head && j < sp.head + sp.nvec * VEC) first = j - (j - sp.head) % VEC;
      if (first < c0 || first >= c0 + W) return a;
      if (m != nullptr && (bits_at(m, j, mwords) & 1u) == 0) return a;
      a.f = E::load_scalar_coherent(src + j);
      if (BWD) a.x = E::load_scalar_coherent(x + j);
      a.j = j;
      return a;
    };
    Hit mine{-1, 0, 0.f, 0.f};
    if (tid < todo) mine = look(tid);

    // the copy: the scalar head and tail, then the vectors
    const int edge = edge_of(part, V, c0, W);
    if (edge >= 0) {
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
    if (todo == 0) continue;
    __syncthreads();
    auto put = [&](const Hit& a) {
      if (a.j >= 0) E::store_scalar(out + a.j, h.value(a.col, a.f, a.x));
    };
    put(mine);
    for (int t = tid + kRulesThreads; t < todo; t += kRulesThreads) put(look(t));
  }
}

// Stages of the bulk kernel's ring, a tile's part of a row each.  With the words two CTAs share an SM
// at four stages (374 us for (4, 1024, 151936) bf16, 98% of the copy rate; three stages: 390 us).  The
// backward has no words, and five CTAs at two stages (421 us, with the scattered reads of touched
// columns' logits; three stages: 434 us, four: 462 us).
template <bool BWD>
constexpr int kStagesOf = BWD ? 2 : 4;

// MASK: there is one.  STAGES: of the ring (1: runs of one row).
template <class E, bool BWD, bool MASK, int STAGES>
__global__ void __launch_bounds__(kRulesThreads) rules_bulk_kernel(const RulesParams p, int tiles, int run, int runs) {
  using H = History<E, BWD>;
  using S = typename E::storage;
  constexpr int VEC = E::kVec, W = H::W;
  extern __shared__ uint4 rules_smem[];  // the ring, then the words
  __shared__ typename H::Shared sh;
  __shared__ __align__(8) uint64_t full_bar[STAGES];
  wait_for_previous_grids();
  const int tid = threadIdx.x;
  const int c0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles)) * W;
  const unsigned seq_run = blockIdx.x / static_cast<unsigned>(tiles);
  const int64_t b = seq_run / static_cast<unsigned>(runs);
  const int64_t l0 = static_cast<int64_t>(seq_run % static_cast<unsigned>(runs)) * run;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(run), p.x.L - l0));
  const int V = p.x.V, mwords = (V + 31) >> 5;
  auto out_row = [&](int rr) { return static_cast<S*>(p.out.ptr) + b * p.out.sb + (l0 + rr) * p.out.sl; };
  auto src_row = [&](int rr) {
    return BWD ? static_cast<const S*>(p.dy.ptr) + b * p.dy.sb + (l0 + rr) * p.dy.sl
               : static_cast<const S*>(p.x.ptr) + b * p.x.sb + (l0 + rr) * p.x.sl;
  };
  auto stage = [&](int rr) { return rules_smem + (rr % STAGES) * kTileVecs; };
  auto fill = [&](int rr) {  // thread 0: start the copy of row rr's part into its stage
    const Part t = part_of<E>(out_row(rr), V, c0);
    if (t.i1 <= t.i0) return;
    const uint32_t bar = smem_addr(&full_bar[rr % STAGES]);
    const uint32_t bytes = static_cast<uint32_t>(t.i1 - t.i0) * 16u;
    mbar_expect(bar, bytes);
    bulk_load(smem_addr(stage(rr)), src_row(rr) + t.sp.head + static_cast<int64_t>(t.i0) * VEC, bytes, bar);
  };
  if (tid == 0) {
    for (int k = 0; k < STAGES; ++k) mbar_init(smem_addr(&full_bar[k]), 1u);
    mbar_init_fence();
    for (int k = 0; k < STAGES && k < nrows; ++k) fill(k);
  }
  H h(p, sh, reinterpret_cast<uint32_t*>(rules_smem + STAGES * kTileVecs), b, l0, nrows, c0);
  __syncthreads();  // the barriers are there

  uint32_t phases = 0u;  // bit k: the parity that stage k's next copy completes
  for (int rr = 0; rr < nrows; ++rr) {
    S* out = out_row(rr);
    const S* src = src_row(rr);
    const Part part = part_of<E>(out, V, c0);
    const RowSplit sp = part.sp;
    const uint32_t* m = MASK ? p.allowed + b * p.allowed_sb + (l0 + rr) * p.allowed_sl : nullptr;
    const uint32_t allowed = allowed_of<E>(m, sp.head, part.i0, part.i1, mwords);
    h.go_to(rr);
    const int todo = h.todo();
    const S* x = BWD ? static_cast<const S*>(p.x.ptr) + b * p.x.sb + (l0 + rr) * p.x.sl : nullptr;
    // touched column t, the place of its element among the part's (or -1), and its logit (backward)
    struct Hit {
      int col, at;
      float x;
    };
    auto look = [&](int t) {
      Hit a{h.col_at(t), -1, 0.f};
      const int at = c0 + a.col - sp.head - part.i0 * VEC;
      if (a.col < 0 || at < 0 || at >= (part.i1 - part.i0) * VEC) return a;
      if (MASK && (bits_at(m, c0 + a.col, mwords) & 1u) == 0) return a;
      a.at = at;
      if (BWD) a.x = E::load_scalar_coherent(x + c0 + a.col);
      return a;
    };
    Hit mine{-1, -1, 0.f};
    if (tid < todo) mine = look(tid);

    const int edge = edge_of(part, V, c0, W);
    if (edge >= 0) {
      float f = E::load_scalar_coherent(src + edge);
      if (MASK && (bits_at(m, edge, mwords) & 1u) == 0) f = BWD ? 0.f : -INFINITY;
      else if (todo > 0 && h.is_touched(edge - c0)) f = h.value(edge - c0, f, BWD ? E::load_scalar_coherent(x + edge) : 0.f);
      E::store_scalar(out + edge, f);
    }
    if (part.i1 > part.i0) {
      const int k = rr % STAGES;
      if (!mbar_wait(smem_addr(&full_bar[k]), phases >> k & 1u)) {  // the row is not valid; wait once more for its copy
        if (tid == 0 && p.dev_err != nullptr) atomicOr(p.dev_err, GRPO_DEVERR_TIMEOUT_BIT);
        mbar_wait(smem_addr(&full_bar[k]), phases >> k & 1u);
      }
      phases ^= 1u << k;
      if (MASK) {  // -inf or 0 where the mask forbids; touched columns that it forbids are left
        uint4* vb = stage(rr);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int i = tid + q * kRulesThreads;
          const uint32_t ok = allowed >> (8 * q) & ((1u << VEC) - 1u);
          if (part.i0 + i >= part.i1 || ok == (1u << VEC) - 1u) continue;
          uint4 v = vb[i];
          forbid(v, ok, kForbiddenOf<E, BWD>, static_cast<E*>(nullptr));
          vb[i] = v;
        }
        __syncthreads();
      }
      S* buf = reinterpret_cast<S*>(stage(rr));
      auto put = [&](const Hit& a) {
        if (a.at >= 0) E::store_scalar(buf + a.at, h.value(a.col, load_shared<E>(buf + a.at), a.x));
      };
      put(mine);
      for (int t = tid + kRulesThreads; t < todo; t += kRulesThreads) put(look(t));
      bulk_write_fence();
    }
    __syncthreads();
    if (tid == 0) {
      if (part.i1 > part.i0)
        bulk_store(out + sp.head + static_cast<int64_t>(part.i0) * VEC, smem_addr(stage(rr)),
                   static_cast<uint32_t>(part.i1 - part.i0) * 16u);
      bulk_commit();
      // the row before has left its stage: the next copy into it
      if (rr >= 1 && rr - 1 + STAGES < nrows) {
        bulk_wait_read<1>();
        fill(rr - 1 + STAGES);
      }
    }
  }
  if (tid == 0) bulk_wait_all();
}

// Rows per CTA: long runs count the history seldom, but leave two CTAs or more for each place, and
// runs past 8 rows gain nothing (32 rows: 386 us and 480 us, 8: 374 us and 462 us for the bulk forward
// and backward, four stages both, at (4, 1024, 151936) bf16).
int64_t pick_run(int64_t rows, int64_t L, int tiles, int64_t places) {
  int64_t run = rows * tiles / (2 * places);
  run = run < 1 ? 1 : (run > kMaxRun ? kMaxRun : run);
  return run < L ? run : L;
}

template <class E, bool BWD, bool MASK, int STAGES>
cudaError_t launch_bulk(const RulesParams& p, dim3 grid, int tiles, int64_t run, int64_t runs, int words,
                        cudaStream_t s) {
  constexpr int ring = STAGES * kTileVecs * 16, most = ring + History<E, BWD>::WORDS * 4;
  if (most > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(rules_bulk_kernel<E, BWD, MASK, STAGES>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  return launch_after_previous_smem(rules_bulk_kernel<E, BWD, MASK, STAGES>, grid, dim3(kRulesThreads), ring + words, s,
                                    p, tiles, static_cast<int>(run), static_cast<int>(runs));
}

template <class E, bool BWD, int HOW>
cudaError_t launch_e(const RulesParams& p, int64_t rows, int sms, cudaStream_t s) {
  using H = History<E, BWD>;
  const int tiles = (p.x.V + H::W - 1) / H::W;
  const bool used = (p.tokens != nullptr && (!BWD || p.repetition != nullptr)) || (!BWD && p.M > 0);
  const int words = used ? H::WORDS * 4 : 0;
  static_assert(H::WORDS * 4 < 40 * 1024, "with the static part within the 48 KB that need no leave");
  const int64_t run = pick_run(rows, p.x.L, tiles, 4LL * sms), runs = (p.x.L + run - 1) / run;
  const dim3 grid(static_cast<unsigned>(rows / p.x.L * runs * tiles)), block(kRulesThreads);
  if constexpr (HOW == kInPhase) {
    // One row: its part is all that the ring holds, and more CTAs share an SM (64 decode rows of 151936
    // under masks: 20 us, 24 us through registers).  The forward's longer ring pays from runs of four
    // rows (runs of two, 510 rows of 32003 fp32: 29 us, 24 us through registers), and not with a mask,
    // which lets the registers leave out what it forbids (there 43 us, against 31 us).
    constexpr int many = kStagesOf<BWD>;
    if (run == 1)
      return p.allowed ? launch_bulk<E, BWD, true, 1>(p, grid, tiles, run, runs, words, s)
                       : launch_bulk<E, BWD, false, 1>(p, grid, tiles, run, runs, words, s);
    if (p.allowed == nullptr && (BWD || run >= kBulkRun))
      return launch_bulk<E, BWD, false, many>(p, grid, tiles, run, runs, words, s);
    if constexpr (BWD) return launch_bulk<E, BWD, true, many>(p, grid, tiles, run, runs, words, s);
  }
  if constexpr (!(BWD && HOW == kInPhase))  // which the bulk kernel takes whole
    return launch_after_previous_smem(rules_kernel<E, BWD, HOW>, grid, block, words, s, p, tiles, static_cast<int>(run),
                                      static_cast<int>(runs));
}

template <class E, bool BWD>
cudaError_t launch_d(bool same_phase, bool in_place, const RulesParams& p, int64_t rows, int sms, cudaStream_t s) {
  if (in_place) return launch_e<E, BWD, kInPlace>(p, rows, sms, s);
  return same_phase ? launch_e<E, BWD, kInPhase>(p, rows, sms, s) : launch_e<E, BWD, kOutOfPhase>(p, rows, sms, s);
}

}  // namespace

cudaError_t launch_rules(int dtype, bool bwd, bool same_phase, bool in_place, const RulesParams& p, int64_t rows,
                         int sms, cudaStream_t stream) {
  if (dtype == 1) return bwd ? launch_d<BF16, true>(same_phase, in_place, p, rows, sms, stream)
                             : launch_d<BF16, false>(same_phase, in_place, p, rows, sms, stream);
  return bwd ? launch_d<F32, true>(same_phase, in_place, p, rows, sms, stream)
             : launch_d<F32, false>(same_phase, in_place, p, rows, sms, stream);
}

}  // namespace grpo
