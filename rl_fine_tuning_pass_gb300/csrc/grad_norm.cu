// Norm of many gradients: sqrt(sum over all tensors of g^2), one read.
//
// Squares are summed in two fp32 numbers: the sum, and what its roundings lost (a 64-bit addition takes
// a warp some 300 cycles here, and those alone were half of the time).  Without the second number a
// norm of bf16 gradients came out 6e-9 too small: half-way cases are common among sums of 16-bit
// squares, and most are rounded down, for the square of an odd number is 1 modulo 8.  What s = was + g^2 loses is
// g^2 - (s - was), both exact as long as was is not below g^2; so a thread's sums start from a power of two above
// all of its squares, which is taken off at the end.  (From 0, a spike behind small elements left norms 5e-8 off.)
// What is left is the rounding of the losses' sum: up to k 2^-48 of the start at the k-th of a thread's sixteen
// pairs, 2^-40 in all; the start is at most 64 of the largest square, so it is below 7e-11 of a sum.  600M bf16: 187 us, 183 without the start, 195 with sums of two
// numbers that are exact in either order.  An fp32 sum outside [2^-90, 2^80] may have lost what overflowed or fell
// below 2^-149, or bring the total out of range: it is formed again from the elements, read once more and scaled
// by a power of two, and goes into a 64-bit sum beside.  So the norm is right for every finite input.
// Partial sums are per CTA and added in a fixed order.
#include <algorithm>
#include <cmath>

#include "many_tensors.cuh"
#include "two_sum.cuh"

namespace grpo {
namespace {

constexpr int kNormThreads = 256, kNormPer = 32;
constexpr int kNormCtasBf16 = 5, kNormCtasF32 = 4;  // an SM (600M bf16: 202 us with 4, 187 with 5, 189 with 6)
constexpr int64_t kNormChunk = kNormThreads * kNormPer;

// A thread's 32 elements of a chunk, as they lie in memory: four vectors of bf16, eight of fp32.
template <class E>
struct Share {
  static constexpr int kVecs = kNormPer / E::kVec;
  uint4 v[kVecs];
};

// Vector k of thread tid is the chunk's (tid + 256 k)-th.  An odd end, and tensors that are not 16-byte
// aligned, are read element by element, with zeros after the end.  (The vectors by volatile loads: others
// may be put off until what is before them is summed.)
template <class E>
__device__ __forceinline__ void load_share(Share<E>& x, const void* grad, int64_t base, int64_t n) {
  using S = typename E::storage;
  const S* p = static_cast<const S*>(grad) + base;
  const bool aligned = (reinterpret_cast<uintptr_t>(grad) & 15u) == 0;
  const int tid = threadIdx.x % kNormThreads;
  if (aligned && n >= kNormChunk) {
#pragma unroll
    for (int k = 0; k < Share<E>::kVecs; ++k) x.v[k] = ld_v4(reinterpret_cast<const uint4*>(p) + tid + k * kNormThreads);
    return;
  }
  const int left = n < kNormChunk ? static_cast<int>(n) : static_cast<int>(kNormChunk);
  const int whole = aligned ? left / E::kVec : 0;
#pragma unroll
  for (int k = 0; k < Share<E>::kVecs; ++k) {
    x.v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (tid + k * kNormThreads < whole) x.v[k] = ld_v4(reinterpret_cast<const uint4*>(p) + tid + k * kNormThreads);
  }
#pragma unroll
  for (int k = 0; k < Share<E>::kVecs; ++k) {
    const int i = (tid + k * kNormThreads) * E::kVec;
    if (tid + k * kNormThreads < whole || i >= left) continue;
    float f[E::kVec];
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) f[e] = i + e < left ? E::load_scalar(p + i + e) : 0.f;
    x.v[k] = E::pack(f, 0u);  // exact: the values came from this format
  }
}

__device__ __forceinline__ float top_of(const Share<BF16>& x) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x.v[0].x));
#pragma unroll
  for (int k = 0; k < Share<BF16>::kVecs; ++k) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x.v[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(h[i]));
  }
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top_of(const Share<F32>& x) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < Share<F32>::kVecs; ++k)
    m = fmaxf(fmaxf(fmaxf(m, fabsf(__uint_as_float(x.v[k].x))), fabsf(__uint_as_float(x.v[k].y))),
              fmaxf(fabsf(__uint_as_float(x.v[k].z)), fabsf(__uint_as_float(x.v[k].w))));
  return m;
}
// What a thread's sums start from: 2^(2e + 6), above all of their sixteen squares together, for a largest element
// in [2^e, 2^(e + 1)).  (Held to fp32's exponents; the sum is out of [2^-90, 2^80] then.)
template <class E>
__device__ __forceinline__ float start_of(const Share<E>& x) {
  const int e = 2 * static_cast<int>(__float_as_uint(top_of(x)) >> 23) - 121;
  return __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 253)) << 23);
}

// The sum where its squares leave fp32's range: the thread's elements are read once more, and scaled by
// 2^-e, e the largest one's exponent (as two factors, for 2^128 is not an fp32 number).  What
// roundings lose is kept here too, from a start above all 32 squares: in error by 2^-32 at most.
template <class E>
__device__ __noinline__ double sum_scaled(const void* grad, int64_t base, int64_t n) {
  using S = typename E::storage;
  const S* p = static_cast<const S*>(grad) + base;
  const auto element = [&](int k) {
    const int64_t i = static_cast<int64_t>(threadIdx.x % kNormThreads + k / E::kVec * kNormThreads) * E::kVec + k % E::kVec;
    return i < n ? E::load_scalar(p + i) : 0.f;
  };
  float top = 0.f;
  for (int k = 0; k < kNormPer; ++k) {
    const float g = element(k);
    if (g != g) return static_cast<double>(g);
    top = fmaxf(top, fabsf(g));
  }
  if (top == 0.f || top > 3.4028235e38f) return static_cast<double>(top);
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // -127 where top is subnormal
  const int half = e / 2;
  const float by = exp2f(static_cast<float>(-half)), again = exp2f(static_cast<float>(half - e));
  float s = 128.f, lost = 0.f;  // above 32 squares below 4
  for (int k = 0; k < kNormPer; ++k) {
    const float g = element(k) * by * again, was = s;
    s = fmaf(g, g, was);
    lost += fmaf(g, g, was - s);
  }
  return (static_cast<double>(s - 128.f) + static_cast<double>(lost)) * exp2(2.0 * e);
}

struct Total {
  TwoSum near;  // of sums in [2^-90, 2^80]
  double far;   // of the others
};
template <class E>
__device__ __forceinline__ void add_chunk(Total& acc, const NormTensor& t, int64_t base) {
  const int64_t n = t.n - base;
  Share<E> x;
  load_share<E>(x, t.grad, base, n);
  const float2 minus = make_float2(-1.f, -1.f);
  const float start = start_of(x);
  float2 s = make_float2(start, start), lost = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < Share<E>::kVecs; ++k)
#pragma unroll
    for (int i = 0; i < E::kPairs; ++i) {
      const float2 g = E::pair(x.v[k], i), was = s;
      s = __ffma2_rn(g, g, was);
      lost = __fadd2_rn(lost, __ffma2_rn(g, g, __ffma2_rn(s, minus, was)));
    }
  s = __fadd2_rn(s, make_float2(-start, -start));  // exact
  const float sum = s.x + s.y;
  if (sum >= 0x1p-90f && sum <= 0x1p80f) {
    acc.near = two_add(two_add(acc.near, TwoSum{s.x, lost.x}), TwoSum{s.y, lost.y});
    return;
  }
  uint32_t bits = 0;  // rows of an embedding that no token has touched are all zeros
#pragma unroll
  for (int k = 0; k < Share<E>::kVecs; ++k) bits |= x.v[k].x | x.v[k].y | x.v[k].z | x.v[k].w;
  if ((bits & ~E::kSignPair) != 0) acc.far += sum_scaled<E>(t.grad, base, n);
}

// The CTA's sum, in thread 0.  (64-bit additions only where there is something in `far`.)
template <int THREADS>
__device__ __forceinline__ Total cta_sum(Total acc) {
  constexpr int kWarps = THREADS / 32;
  __shared__ TwoSum near[kWarps];
  __shared__ double far[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc.near = two_add(acc.near, two_shfl(acc.near, off));
  if (lane == 0) near[warp] = acc.near;
  const bool any_far = __syncthreads_or(acc.far != 0.0) != 0;  // NaN too
  if (warp == 0) {
    acc.near = lane < kWarps ? near[lane] : TwoSum{0.f, 0.f};
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1) acc.near = two_add(acc.near, two_shfl(acc.near, off));
  }
  if (any_far) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc.far += __shfl_xor_sync(0xFFFFFFFFu, acc.far, off);
    if (lane == 0) far[warp] = acc.far;
    __syncthreads();
    if (threadIdx.x == 0)
#pragma unroll
      for (int i = 1; i < kWarps; ++i) acc.far += far[i];
  }
  return acc;
}

// The root.  In range: that of the first part, and one correction by the residual.
__device__ __forceinline__ float root_of(const Total& t) {
  if (t.far != 0.0) return static_cast<float>(sqrt(static_cast<double>(t.near.hi) + static_cast<double>(t.near.lo) + t.far));
  const float r = sqrtf(t.near.hi);
  return r > 0.f ? fmaf(fmaf(-r, r, t.near.hi) + t.near.lo, 0.5f / r, r) : r;
}

// A CTA sums `run` chunks.  What hides the memory's latency is the number of threads: the chunk's vectors
// are all that a thread holds.
template <int N, class E>
__global__ void __launch_bounds__(kNormThreads, E::kVec == 8 ? kNormCtasBf16 : kNormCtasF32)
    norm_kernel(const __grid_constant__ NormTable<N> tab, uint32_t run, NormPartial* partial) {
  wait_for_previous_grids();
  const uint32_t c0 = blockIdx.x * run, c1 = tab.chunks - c0 < run ? tab.chunks : c0 + run;
  Total acc{{0.f, 0.f}, 0.0};
  int t = tensor_of_chunk(tab, c0, 0);
  for (uint32_t c = c0; c < c1; ++c) {
    t = tensor_of_chunk(tab, c, t);
    add_chunk<E>(acc, tab.t[t], static_cast<int64_t>(c - tab.first[t]) * kNormChunk);
  }
  acc = cta_sum<kNormThreads>(acc);
  if (threadIdx.x == 0) partial[blockIdx.x] = NormPartial{acc.near.hi, acc.near.lo, acc.far};
}

// A few small tensors (an adapter's gradients) by one cluster: 32 groups of 256 threads take a chunk each
// at a time, and the CTAs' sums meet in the first one's shared memory instead of in a second launch.
constexpr int kFewCtas = 8, kFewThreads = 1024, kFewGroups = kFewCtas * kFewThreads / kNormThreads;
template <class E>
__global__ void __launch_bounds__(kFewThreads) norm_cluster_kernel(const __grid_constant__ NormTable<kNormFew> tab,
                                                                   float* norm) {
  wait_for_previous_grids();
  __shared__ __align__(16) NormPartial sums[kFewCtas];
  const uint32_t rank = cluster_rank();
  Total acc{{0.f, 0.f}, 0.0};
  int t = 0;
  for (uint32_t c = threadIdx.x / kNormThreads * kFewCtas + rank; c < tab.chunks; c += kFewGroups) {
    t = tensor_of_chunk(tab, c, t);
    add_chunk<E>(acc, tab.t[t], static_cast<int64_t>(c - tab.first[t]) * kNormChunk);
  }
  acc = cta_sum<kFewThreads>(acc);
  cluster_sync();  // every CTA runs: its shared memory may be written
  if (threadIdx.x == 0) {
    const uint32_t at = map_to_rank(smem_addr(sums + rank), 0);
    st_cluster_f32(at, acc.near.hi);
    st_cluster_f32(at + 4, acc.near.lo);
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at + 8), "d"(acc.far) : "memory");
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    Total all{{0.f, 0.f}, 0.0};
#pragma unroll
    for (int i = 0; i < kFewCtas; ++i) {
      all.near = two_add(all.near, TwoSum{sums[i].hi, sums[i].lo});
      if (sums[i].far != 0.0) all.far += sums[i].far;
    }
    *norm = root_of(all);
  }
}

constexpr int kRootThreads = 1024;
__global__ void __launch_bounds__(kRootThreads) norm_root_kernel(const NormPartial* partial, int n, float* norm) {
  wait_for_previous_grids();
  constexpr int kEach = kNormSlots / kRootThreads;
  NormPartial p[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {  // all loads at once
    const int i = threadIdx.x + k * kRootThreads;
    p[k] = i < n ? partial[i] : NormPartial{0.f, 0.f, 0.0};
  }
  Total acc{{0.f, 0.f}, 0.0};
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    acc.near = two_add(acc.near, TwoSum{p[k].hi, p[k].lo});
    if (p[k].far != 0.0) acc.far += p[k].far;
  }
  acc = cta_sum<kRootThreads>(acc);
  if (threadIdx.x == 0) *norm = root_of(acc);
}

int64_t chunks_of(const NormEntry& e) { return (e.t.n + kNormChunk - 1) / kNormChunk; }

template <int N, class E>
cudaError_t launch_part(const NormEntry* tensors, int count, uint32_t chunks, uint32_t run, int ctas, NormPartial* partial,
                        cudaStream_t stream) {
  NormTable<N> tab;
  uint32_t first = 0;
  for (int i = 0; i < count; ++i) {
    tab.t[i] = tensors[i].t;
    tab.first[i] = first;
    first += static_cast<uint32_t>(chunks_of(tensors[i]));
  }
  tab.count = count;
  tab.chunks = chunks;
  return launch_after_previous(norm_kernel<N, E>, dim3(ctas), dim3(kNormThreads), stream, tab, run, partial);
}

template <class E>
cudaError_t launch_few(const NormEntry* tensors, int count, float* norm, cudaStream_t stream) {
  NormTable<kNormFew> tab;
  uint32_t first = 0;
  for (int i = 0; i < count; ++i) {
    tab.t[i] = tensors[i].t;
    tab.first[i] = first;
    first += static_cast<uint32_t>(chunks_of(tensors[i]));
  }
  tab.count = count;
  tab.chunks = first;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kFewCtas);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kFewCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, norm_cluster_kernel<E>, tab, norm);
}

}  // namespace

// One launch for each type that occurs, and for each kNormMany tensors of it.  `tensors` is put in that
// order, those without elements left out.  A CTA's share is as many chunks
// as leave kNormSlots partial sums at most: shares are fixed, whichever SM takes them and when, so the
// sum is the same each time, but there are some thirteen of them for each place on the SMs, which
// evens out that some are farther from the memory (with one share each, 600M bf16 took 299 us).
cudaError_t launch_grad_norm(NormEntry* tensors, int64_t count, NormPartial* partial, float* norm, cudaStream_t stream) {
  const auto before = [](const NormEntry& a, const NormEntry& b) { return a.bf16 < b.bf16; };
  count = std::remove_if(tensors, tensors + count, [](const NormEntry& e) { return e.t.n == 0; }) - tensors;
  if (!std::is_sorted(tensors, tensors + count, before)) std::stable_sort(tensors, tensors + count, before);
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += chunks_of(tensors[i]);
  if (count > 0 && count <= kNormFew && chunks <= 2 * kFewGroups && tensors[0].bf16 == tensors[count - 1].bf16)
    return tensors[0].bf16 ? launch_few<BF16>(tensors, static_cast<int>(count), norm, stream)
                           : launch_few<F32>(tensors, static_cast<int>(count), norm, stream);
  const int64_t launches = count / kNormMany + 2, run = chunks / (kNormSlots - launches) + 1;
  int slots = 0;
  for (int64_t at = 0; at < count;) {
    const int bf16 = tensors[at].bf16;
    int64_t end = at, here = 0;
    while (end < count && end - at < kNormMany && tensors[end].bf16 == bf16) here += chunks_of(tensors[end++]);
    const NormEntry* part = tensors + at;
    const int k = static_cast<int>(end - at), ctas = static_cast<int>((here + run - 1) / run);
    const uint32_t ch = static_cast<uint32_t>(here), rn = static_cast<uint32_t>(run);
    cudaError_t e;
    if (bf16)
      e = k <= kNormFew ? launch_part<kNormFew, BF16>(part, k, ch, rn, ctas, partial + slots, stream)
                        : launch_part<kNormMany, BF16>(part, k, ch, rn, ctas, partial + slots, stream);
    else
      e = k <= kNormFew ? launch_part<kNormFew, F32>(part, k, ch, rn, ctas, partial + slots, stream)
                        : launch_part<kNormMany, F32>(part, k, ch, rn, ctas, partial + slots, stream);
    if (e != cudaSuccess) return e;
    slots += ctas;
    at = end;
  }
  return launch_after_previous(norm_root_kernel, dim3(1), dim3(kRootThreads), stream,
                               static_cast<const NormPartial*>(partial), slots, norm);
}

}  // namespace grpo
