// The K largest log-probs of each row, log_softmax(x / T), with their columns: sorted, ties
// to the lowest column.
//
// One sweep over the row forms the softmax statistic (logits_stat.cuh) and notes the largest element
// of every chunk (the vectors of one thread in one step; in rows past kNotes chunks of several steps).
// Each thread also keeps the largest element it has met in the even and in the odd places of its
// vectors, 512 maxima per CTA (up to K = 64 one of both, 256); the K-th largest of those maxima is a
// lower bound of the K-th largest element (K different elements reach it), so a chunk without an
// element that reaches it cannot hold a result.  The chunks that do (about 70 of a row of N(0, 1)
// elements at K = 64) are listed and read again, and their elements that reach the bound (about 74)
// are ranked (rank_entries).  Noting only the chunks that reach a bound taken again and again within
// the sweep waits at more barriers: 2048 rows of 32000 bf16 at K = 128 took 50 us, against 43 us.
//
// Measured: the top 64 of 8192 rows of 151936 bf16 take 394 us (6.3 TB/s, 93% of the copy rate; radix
// selection alone took 4.2 ms); what is left are the barriers of the bound and of the
// ranking, which five CTAs per SM do not hide whole.  They do not shrink with the row: the top 32 of 8192
// rows of 600 take 60 us, of 4000 63 us.
//
// Rows that collect more than the buffers hold (thousands of ties at the K-th value) are done
// again by radix selection on order-preserving keys.
//
// With few rows, a cluster of CTAs takes a row: each CTA ranks its own part, the first one
// merges the sorted lists and the statistics, which the others write into its shared memory.
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

// The first `need` columns, in column order, whose key >> shift is `key`, into list.
template <class E>
__device__ void fill_ties(const typename E::storage* row, int V, uint32_t key, int shift, unsigned need,
                          uint64_t* list) {
  __shared__ unsigned wsum[kTopkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned done = 0;
  for (int j0 = 0; j0 < V && done < need; j0 += kTopkThreads) {
    const int j = j0 + tid;
    uint32_t k = 0u;
    bool tie = false;
    if (j < V) {
      k = key_of(E::load_scalar(row + j));
      tie = (k >> shift) == key;
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
    if (tie && at < need) list[at] = entry_of(k, j);
    done += total;
    __syncthreads();
  }
  __syncthreads();
}

// Radix selection of the K largest entries of the row into list[0..K) (any order).
template <class E>
__device__ void radix_select(const typename E::storage* row, int V, int K, uint64_t* list) {
  __shared__ unsigned hist[256];
  __shared__ unsigned sh_digit, sh_above, sh_n;
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
  __syncthreads();
  fill_ties<E>(row, V, prefix, kShift, need, list + (K - need));
}

constexpr int kMaxima = 2 * kTopkThreads;   // running maxima per CTA
constexpr int kOneMaximum = 64;             // up to this K one maximum per thread is enough
constexpr int kSurvivors = 1024;            // entries that are ranked
constexpr int kNotes = 8192;                // chunks whose largest element is noted
constexpr uint32_t kKeyNegInf = 0x007Fu;    // high half of the key of -inf

// A lower bound of the K-th largest of the CTA's running maxima (high halves of their keys in sh;
// warp 0 only) that K of them or more reach: that key's high half, or, where just K reach a smaller
// prefix of it, the prefix.
__device__ __forceinline__ uint32_t kth_maximum(const uint16_t* sh, int K) {
  constexpr int kPer = kTopkThreads / 32;
  const int lane = threadIdx.x;
  const bool two = K > kOneMaximum;
  uint32_t k[2 * kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    k[q] = sh[lane + 32 * q];
    k[kPer + q] = two ? sh[kTopkThreads + lane + 32 * q] : 0u;
  }
  uint32_t best = 0u;
#pragma unroll 1
  for (uint32_t bit = 0x8000u; bit != 0u; bit >>= 1) {
    const uint32_t cand = best | bit;
    int n = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) n += k[q] >= cand;
    if (two) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) n += k[kPer + q] >= cand;
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (n >= K) best = cand;
    if (n == K) break;
  }
  return best;
}

__device__ __forceinline__ void st_cluster_u64(uint32_t cluster_addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr), "l"(v) : "memory");
}

// Ranks of m entries whose keys are `least` or more: put(place, entry) for each.  The entries go into
// 256 buckets by their distance from `least` (its exponent and three bits: the top of a row thins
// out with the distance), larger ones first; a place is what the larger buckets hold, and what is
// larger in the entry's own.  Up to 96 entries are counted straight away, which is as fast as the
// buckets' barriers there: the top 64 (about 70 entries) of 2000 rows of 32000 took 39.6 us counted
// and 40.3 us with buckets, the top 128 52.7 us and 49.1 us, the top 256 109 us and 72 us.
template <class E, int T, class F>
__device__ __forceinline__ void rank_entries(const uint64_t* surv, int m, uint32_t least, uint64_t* sorted,
                                             unsigned (&first)[256], F put) {
  static_assert(T == 256, "a thread per bucket");
  const int tid = threadIdx.x;
  if (m <= 96) {
    if (tid < m) {
      const uint64_t e = surv[tid];
      int place = 0;
      for (int q = 0; q < m; ++q) place += surv[q] > e;
      put(place, e);
    }
    return;
  }
  constexpr int kShift = 32 - 8 * static_cast<int>(sizeof(typename E::storage));
  auto bucket = [&](uint64_t e) {  // 0: the largest
    const uint32_t d = ((static_cast<uint32_t>(e >> 32) >> kShift) - (least >> kShift)) + 8u;
    const int top = 31 - __clz(static_cast<int>(d));  // >= 3
    return 255 - ((top - 3) * 8 + static_cast<int>(d >> (top - 3) & 7u));
  };
  first[tid] = 0u;
  __syncthreads();
  for (int i = tid; i < m; i += T) atomicAdd(&first[bucket(surv[i])], 1u);
  __syncthreads();
  // counts to first places
  const int lane = tid & 31, warp = tid >> 5;
  const unsigned mine = first[tid];
  unsigned sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  __shared__ unsigned warps[T / 32];
  if (lane == 31) warps[warp] = sum;
  __syncthreads();
  unsigned base = sum - mine;
  for (int w = 0; w < warp; ++w) base += warps[w];
  first[tid] = base;
  __syncthreads();
  for (int i = tid; i < m; i += T) {
    const uint64_t e = surv[i];
    sorted[atomicAdd(&first[bucket(e)], 1u)] = e;  // leaves each bucket's end
  }
  __syncthreads();
  for (int i = tid; i < m; i += T) {
    const uint64_t e = sorted[i];
    const int k = bucket(e);
    const int lo = k == 0 ? 0 : static_cast<int>(first[k - 1]), hi = static_cast<int>(first[k]);
    int place = lo;
    for (int q = lo; q < hi; ++q) place += sorted[q] > e;
    put(place, e);
  }
}

struct TopkPart {  // what one CTA of a cluster hands to the first
  float m, s;
  int n;           // entries in its list, -1: its buffers overflowed
};

// CS CTAs per row (a cluster when CS > 1).  Dynamic shared memory: cap candidates, then
// kSurvivors, then (CS > 1) the CTAs' lists.
template <class E, int CS>
__global__ void __launch_bounds__(kTopkThreads, 5) topk_kernel(const TopkParams p, int notes, int gs) {
  using S = typename E::storage;
  constexpr int VEC = E::kVec, T = kTopkThreads, U = kUnroll;
  extern __shared__ uint64_t topk_smem[];
  __shared__ uint16_t maxima[kMaxima];
  __shared__ uint64_t list[kTopkMax];
  __shared__ TopkPart parts[CS];
  __shared__ uint32_t sh_least;
  __shared__ unsigned sh_m, sh_c;
  __shared__ unsigned buckets[256];
  // the chunks' largest elements, then room for rank_entries
  float* noted = reinterpret_cast<float*>(topk_smem);
  uint64_t* surv = topk_smem + notes / 2;
  uint64_t* lists = surv + kSurvivors;
  if (CS > 1) cluster_arrive();  // every CTA of the cluster runs before its shared memory is written
  wait_for_previous_grids();
  const uint32_t rank = CS > 1 ? cluster_rank() : 0u;
  const int64_t r = blockIdx.x / CS;
  const int64_t b = r / p.x.L, l = r - b * p.x.L;
  const S* row = static_cast<const S*>(p.x.ptr) + b * p.x.sb + l * p.x.sl;
  const int V = p.x.V, K = p.K, tid = threadIdx.x;
  const float c = p.c;
  const RowSplit sp = split_row<E>(row, V);
  const int part = (sp.nvec + CS - 1) / CS;
  const int v0 = min(sp.nvec, static_cast<int>(rank) * part), v1 = min(sp.nvec, v0 + part);
  if (tid == 0) sh_m = sh_c = 0u;
  __syncthreads();

  MaxRun rs;
  float2 sub = make_float2(-INFINITY, -INFINITY);
  auto take = [&](float x, int j) {
    const unsigned at = atomicAdd(&sh_m, 1u);
    if (at < kSurvivors) surv[at] = entry_of(key_of(x), j);
  };
  // the scalar head and tail: at most one element per thread, kept for the end
  float edge = -INFINITY;
  int edge_j = -1;
  if (rank == 0 && tid < sp.head) edge_j = tid;
  if (rank == CS - 1 && tid >= T - sp.tail) edge_j = V - T + tid;
  if (edge_j >= 0) {
    edge = E::load_scalar(row + edge_j);
    maxrun_scalar(rs, edge, c);
    sub.x = fmaxf(sub.x, edge);
  }

  const uint4* vb = reinterpret_cast<const uint4*>(row + sp.head);
  int step = 0;           // steps done
  float top = -INFINITY;  // of a chunk of several steps
  auto note = [&]() {
    noted[((step - 1) >> gs) * T + tid] = top;
    top = -INFINITY;
  };
  auto fold = [&](const uint4 (&v)[U]) {
    const float2 pm = maxrun_vectors<E>(rs, v, c);
    sub.x = fmaxf(sub.x, pm.x);
    sub.y = fmaxf(sub.y, pm.y);
    const float m = fmaxf(pm.x, pm.y);
    ++step;
    if (gs == 0) {  // chunks of one step (with the general form alone 2048 rows of 32000 fp32 take 48 us, not 42)
      noted[(step - 1) * T + tid] = m;
      return;
    }
    top = fmaxf(top, m);
    if ((step & ((1 << gs) - 1)) == 0) note();
  };
  int i0 = v0;
  for (; i0 + U * T <= v1; i0 += U * T) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = ld_nc_v4(vb + i0 + k * T + tid);
    if (tid == 0) {  // ask L2 for the step after the next (2000 rows of 304 KB: 110 us; the next step: 113 us)
      const int a = i0 == v0 ? i0 + U * T : i0 + 2 * U * T, n = min(v1, i0 + 3 * U * T) - a;
      if (n > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(vb + a), "r"(static_cast<uint32_t>(n) * 16u)
                     : "memory");
    }
    fold(v);
  }
  if (i0 < v1) {
    const uint32_t pad = sizeof(S) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      v[k] = make_uint4(pad, pad, pad, pad);
      if (i0 + k * T + tid < v1) v[k] = ld_nc_v4(vb + i0 + k * T + tid);
    }
    fold(v);
  }
  if ((step & ((1 << gs) - 1)) != 0) note();

  // the bound
  if (K <= kOneMaximum) {
    maxima[tid] = static_cast<uint16_t>(key_of(fmaxf(sub.x, sub.y)) >> 16);
  } else {
    maxima[tid] = static_cast<uint16_t>(key_of(sub.x) >> 16);
    maxima[T + tid] = static_cast<uint16_t>(key_of(sub.y) >> 16);
  }
  __syncthreads();
  if (tid < 32) {
    const uint32_t k = kth_maximum(maxima, K);
    if (tid == 0) sh_least = (k <= kKeyNegInf ? kKeyNegInf + 1u : k) << 16;  // an element above -inf at least
  }
  MaxStat st = maxstat_block<T>(rs.stat(), c);
  __syncthreads();

  // the chunks that reach it, then their elements that do, four threads to a chunk and step
  const uint32_t least = sh_least;
  const float thr = value_of(least);
  const int n = ((step + (1 << gs) - 1) >> gs) * T;
  constexpr unsigned kChunks = 2 * kTopkMax;
  uint32_t* chunks = reinterpret_cast<uint32_t*>(list);
  for (int q = tid; q < n; q += T) {
    if (!(noted[q] >= thr)) continue;
    const unsigned at = atomicAdd(&sh_c, 1u);
    if (at < kChunks) chunks[at] = static_cast<uint32_t>(q);
  }
  __syncthreads();
  const unsigned nc = sh_c;
  if (edge_j >= 0 && edge >= thr) take(edge, edge_j);
  for (unsigned q = tid; q < U * min(nc, kChunks) << gs; q += T) {
    const unsigned at = q / U >> gs, chunk = chunks[at], in = (q / U) - (at << gs);
    const int i = v0 + static_cast<int>(((chunk / T << gs) + in) * U + q % U) * T + static_cast<int>(chunk % T);
    if (i >= v1) continue;
    float f[VEC];
    E::unpack(ld_nc_v4(vb + i), f);
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (f[k] >= thr) take(f[k], sp.head + i * VEC + k);
  }
  __syncthreads();
  int m = static_cast<int>(sh_m);
  const bool over = nc > kChunks || m > kSurvivors;
  uint64_t* mine = list;
  if (CS > 1) {
    cluster_wait();
    // this CTA's sorted list, in the first CTA's shared memory
    const uint32_t at = map_to_rank(smem_addr(lists + rank * static_cast<uint32_t>(K)), 0);
    if (!over)
      rank_entries<E, T>(surv, m, least, topk_smem, buckets, [&](int place, uint64_t e) {
        if (place < K) st_cluster_u64(at + 8u * place, e);
      });
    if (tid == 0) {
      const uint32_t to = map_to_rank(smem_addr(&parts[rank]), 0);
      st_cluster_f32(to, st.m);
      st_cluster_f32(to + 4u, st.s);
      st_cluster_f32(to + 8u, __int_as_float(over ? -1 : min(m, K)));
    }
    cluster_sync();
    if (rank != 0) return;
    if (tid < 32) {
      st = tid < CS ? MaxStat{parts[tid].m, parts[tid].s} : MaxStat{-FLT_MAX, 0.f};
      st = maxstat_warp(st, c);
    }
  }

  __shared__ float sh_max, sh_ln_s, sh_lse;
  if (tid == 0) {
    sh_max = st.m;
    sh_ln_s = logf(st.s);
    sh_lse = fmaf(st.m, p.invT, sh_ln_s);
    if (p.lse) p.lse[r] = sh_lse;
  }
  __syncthreads();
  int64_t* ids = p.ids + r * K;
  float* logp = p.logp + r * K;
  const float ln_s = sh_ln_s, xmax = sh_max;
  if (!(fabsf(ln_s) <= FLT_MAX)) {  // a NaN or +inf logit, or nothing but -inf: no log-prob is defined
    for (int k = tid; k < K; k += T) {
      ids[k] = k;
      logp[k] = __int_as_float(0x7FC00000);
    }
    return;
  }
  auto put = [&](int place, uint64_t e) {
    ids[place] = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(e));
    logp[place] = fmaf(value_of(static_cast<uint32_t>(e >> 32)) - xmax, p.invT, -ln_s);
  };
  int have = m;        // entries that are ranked below or in the lists
  bool again = over;
  if (CS > 1) {
    have = 0;
#pragma unroll
    for (int q = 0; q < CS; ++q) {
      again |= parts[q].n < 0;
      have += parts[q].n;
    }
  }
  if (again) {  // too many candidates: by radix selection
    radix_select<E>(row, V, K, mine);
    for (int k = tid; k < K; k += T) {
      const uint64_t e = mine[k];
      int place = 0;
      for (int q = 0; q < K; ++q) place += mine[q] > e;
      put(place, e);
    }
    return;
  }
  if (have < K) {  // fewer than K columns above -inf: the first of the others follow them
    const uint32_t key = key_of(-INFINITY);
    fill_ties<E>(row, V, key, 0, static_cast<unsigned>(K - have), mine);
    for (int k = tid; k < K - have; k += T) put(have + k, mine[k]);
  }
  if (CS == 1) {
    rank_entries<E, T>(surv, m, least, topk_smem, buckets, [&](int place, uint64_t e) {
      if (place < K) put(place, e);
    });
  } else {
    for (int i = tid; i < CS * K; i += T) {
      const int from = i / K, at = i - from * K;
      if (at >= parts[from].n) continue;
      const uint64_t e = lists[i];
      int place = at;
      int lo[CS] = {};
#pragma unroll 1
      for (int step = kTopkMax / 2; step > 0; step >>= 1) {  // how many of each list are larger, side by side
#pragma unroll
        for (int q = 0; q < CS; ++q)
          if (lo[q] + step <= parts[q].n && lists[q * K + lo[q] + step - 1] > e) lo[q] += step;
      }
#pragma unroll
      for (int q = 0; q < CS; ++q) {
        if (q == from) continue;
        if (lo[q] < parts[q].n && lists[q * K + lo[q]] > e) ++lo[q];  // (all 256 of them)
        place += lo[q];
      }
      if (place < K) put(place, e);
    }
  }
}

// CTAs per row: as many as keep four CTAs or fewer per SM (five fit), each with a step of the sweep
// (1024 vectors) or more.  With parts of half a step the merge costs more than the sweep saves (64 rows
// of 32000 fp32 at K = 64: 8.7 us, 15.2 us with twice the CTAs; one row of 8192 bf16 at K = 20: 4.6 and
// 6.1 us; one of 32000: 6.6 and 6.4 us).
template <class E>
int pick_split(const TopkParams& p, int64_t rows, int sms) {
  int cs = 1;
  while (cs < 8 && rows * cs * 2 <= 4LL * sms && p.x.V / E::kVec >= 2048 * cs) cs *= 2;
  return cs;
}

template <class E, int CS>
cudaError_t launch_topk_cs(const TopkParams& p, int64_t rows, cudaStream_t s) {
  // chunks of 2^gs steps
  const int vecs = p.x.V / E::kVec / CS + 1;
  const int64_t steps = (static_cast<int64_t>(vecs) + kTopkThreads * kUnroll - 1) / (kTopkThreads * kUnroll);
  int gs = 0;
  while (((steps + (1LL << gs) - 1) >> gs) * kTopkThreads > kNotes) ++gs;
  const int least = 2 * kSurvivors;  // rank_entries sorts as many entries there
  const int n = static_cast<int>((steps + (1LL << gs) - 1) >> gs) * kTopkThreads, notes = n < least ? least : n;
  const size_t smem = 4 * static_cast<size_t>(notes) + 8 * (kSurvivors + (CS > 1 ? CS * p.K : 0));
  if (smem > 40 * 1024) {  // with the static part past the 48 KB that need no leave
    const cudaError_t e = cudaFuncSetAttribute(topk_kernel<E, CS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * kNotes + 8 * (kSurvivors + (CS > 1 ? CS * kTopkMax : 0)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * CS));
  cfg.blockDim = dim3(kTopkThreads);
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
  return cudaLaunchKernelEx(&cfg, topk_kernel<E, CS>, p, notes, gs);
}

template <class E>
cudaError_t launch_topk_e(const TopkParams& p, int64_t rows, int sms, cudaStream_t s) {
  switch (pick_split<E>(p, rows, sms)) {
    case 8: return launch_topk_cs<E, 8>(p, rows, s);
    case 4: return launch_topk_cs<E, 4>(p, rows, s);
    case 2: return launch_topk_cs<E, 2>(p, rows, s);
    default: return launch_topk_cs<E, 1>(p, rows, s);
  }
}

}  // namespace

cudaError_t launch_topk(int dtype, const TopkParams& p, int64_t rows, int sms, cudaStream_t stream) {
  return dtype == 1 ? launch_topk_e<BF16>(p, rows, sms, stream) : launch_topk_e<F32>(p, rows, sms, stream);
}

}  // namespace grpo
