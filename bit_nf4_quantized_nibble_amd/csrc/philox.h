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

// Round i of a counter's words.
constexpr int kPhiloxRounds = 10;
__device__ __forceinline__ void philox_round(const PhiloxKey& key, int i, uint32_t (&c)[4]) {
  const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
  c[0] = (uint32_t)(b >> 32) ^ c[1] ^ (key.k0 + (uint32_t)i * 0x9E3779B9u);
  c[1] = (uint32_t)b;
  c[2] = (uint32_t)(a >> 32) ^ c[3] ^ (key.k1 + (uint32_t)i * 0xBB67AE85u);
  c[3] = (uint32_t)a;
}

// The four words of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ u32x4_t philox(const PhiloxKey& key, uint32_t group, uint32_t row) {
  uint32_t c[4] = {group, row, key.o0, key.o1};
#pragma unroll
  for (int i = 0; i < kPhiloxRounds; ++i) philox_round(key, i, c);
  return u32x4_t{c[0], c[1], c[2], c[3]};
}
__device__ __forceinline__ bool keeps(const u32x4_t& w, int e, uint32_t threshold) {
  return ((w[e >> 1] >> (16 * (e & 1))) & 0xffffu) >= threshold;
}

}  // namespace qnf4
