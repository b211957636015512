// Reading the vectors of a row whose output starts at another address mod 16.
//
// The streams here are laid out by the output row (16-byte stores); an input row at another
// phase (a view like logits[:, :-1] of odd vocabulary, written to a dense tensor) has its 16 bytes
// across two aligned vectors.  Both are loaded (the second is the next lane's first, and comes
// from L1) and shifted together; the row's first and last vectors, whose aligned neighbours may
// lie outside the row, are read element by element.  The loads of all of a thread's vectors stand
// before the first shift: with a branch between them they went out one at a time.
#pragma once

#include "rowpass_common.cuh"

namespace grpo {

// Ask L2 for the start of a row (64 KB at most) that the CTA will stream once it has read other
// things.  One thread.
__device__ __forceinline__ void prefetch_row(const void* row, int64_t bytes) {
  const uintptr_t a = (reinterpret_cast<uintptr_t>(row) + 15u) & ~static_cast<uintptr_t>(15);
  const int64_t left = bytes - 16;
  const uint32_t n = static_cast<uint32_t>(left < 65536 ? left : 65536) & ~15u;
  if (left >= 16) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(n) : "memory");
}

// Bytes [off, off + 16) of a then b; off a multiple of 2.
__device__ __forceinline__ uint4 shift_vectors(const uint4& a, const uint4& b, uint32_t off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8u) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (off & 4u) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  const uint32_t bits = (off & 2u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Vectors i + k STEP < n (k < N) of the row's nvec vectors at `body` (aligned to the element), into
// v; the others are left.  The row is not written meanwhile.
template <class E, int N, int STEP>
__device__ __forceinline__ void load_out_of_phase(uint4 (&v)[N], const typename E::storage* body, int i, int n,
                                                  int nvec) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(body);
  const uint32_t off = static_cast<uint32_t>(at & 15u);
  const uint4* a = reinterpret_cast<const uint4*>(at - off);
  if (off == 0u) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (i + k * STEP < n) v[k] = ld_nc_v4(a + i + k * STEP);
    return;
  }
  uint4 w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {  // the first and last vector: any vector of the row instead
    const int j = i + k * STEP;
    const bool in = j < n && nvec > 2;
    const int q = j < 1 ? 1 : (j > nvec - 2 ? nvec - 2 : j);
    if (in) v[k] = __ldg(a + q);
    if (in) w[k] = __ldg(a + q + 1);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = i + k * STEP;
    if (j >= n) continue;
    if (j > 0 && j < nvec - 1) {
      v[k] = shift_vectors(v[k], w[k], off);
    } else {
      float f[E::kVec];
#pragma unroll
      for (int q = 0; q < E::kVec; ++q) f[q] = E::load_scalar(body + static_cast<int64_t>(j) * E::kVec + q);
      v[k] = E::pack(f, 0u);
    }
  }
}

}  // namespace grpo
