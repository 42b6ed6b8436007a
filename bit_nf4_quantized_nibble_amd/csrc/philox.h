// philox.h -- the counter-based generator of the seeded dropout.
//
// Philox 4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit products, the multipliers and the key's
// increments from the paper.  Element (row, column) of a call takes half column % 8 (low halves
// first) of the four words for the counter {column / 8, row, offset} under the key `seed`, so a
// mask depends on nothing but the seed, the offset and the element's place, is formed where it is
// needed in any order, and is never stored.
#pragma once

#include "common.h"

namespace qnf4 {

// A call's generator: seed[0] the key, seed[1] the offset, read on the device (a captured call
// draws another mask at each replay that finds other values there); an element is kept where its
// 16 bits are at least `threshold`.
struct Seeded {
  const uint64_t* seed;
  uint32_t threshold;
};

struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ PhiloxKey philox_key(const Seeded& s) {
  const uint64_t k = s.seed[0], o = s.seed[1];
  return {(uint32_t)k, (uint32_t)(k >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

// The four words of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ u32x4_t philox(const PhiloxKey& key, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}
__device__ __forceinline__ bool keeps(const u32x4_t& w, int e, uint32_t threshold) {
  return ((w[e >> 1] >> (16 * (e & 1))) & 0xffffu) >= threshold;
}

}  // namespace qnf4
