// Reading the vectors of a row whose output starts at another address mod 16.
//
// The streams here are laid out by the output row (16-byte stores); an input row at another
// phase (a view like logits[:, :-1] of odd vocabulary, written to a dense tensor) has its 16 bytes
// across two aligned vectors.  Both are loaded (the second is the next lane's first, and comes
// from L1) and shifted together; the row's first and last vectors, whose aligned neighbours may
// lie outside the row, are read element by element.
#pragma once

#include "rowpass_common.cuh"

namespace grpo {

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

// Vector i of the nvec vectors at `body` (aligned to the element).  The row is not written
// meanwhile.
template <class E>
__device__ __forceinline__ uint4 load_out_of_phase(const typename E::storage* body, int i, int nvec) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(body);
  const uint32_t off = static_cast<uint32_t>(at & 15u);
  const uint4* a = reinterpret_cast<const uint4*>(at - off) + i;
  if (off == 0u) return ld_nc_v4(a);
  if (i > 0 && i < nvec - 1) return shift_vectors(__ldg(a), __ldg(a + 1), off);
  float f[E::kVec];
#pragma unroll
  for (int q = 0; q < E::kVec; ++q) f[q] = E::load_scalar(body + static_cast<int64_t>(i) * E::kVec + q);
  return E::pack(f, 0u);
}

}  // namespace grpo
