// dropout_device.h -- the keep decisions of dropout from a counter-based generator.
//
// The generator is Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel Random Numbers: As Easy as
// 1, 2, 3", SC 2011): ten rounds that turn a 128-bit counter and a 64-bit key into four 32-bit
// words.  The key is the seed.  Element i of a call belongs to counter block offset + i / 8 and
// has a 32-bit uniform u: its high half is 16-bit piece i % 8 of the words of counter (block, 0, 0),
// its low half the same piece of counter (block, 1, 0).  It is kept iff u >= round(p * 2^32).  The low half matters
// only where the high half equals the threshold's, one element in 65536, so the second block is
// computed only there: an element costs an eighth of a block, at the full 32-bit resolution.
#pragma once

#include "device_common.h"

namespace moe {

struct Drop {
  uint32_t t_hi, t_lo;   // halves of the threshold round(p * 2^32); t_hi = 65536 drops everything
  float scale;           // 1 / (1 - p); 0 for p = 1
};

Drop make_drop(double p);   // dropout.hip

__device__ __forceinline__ uint4 philox4x32(uint64_t block, uint32_t word2, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = word2, c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0, n2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// bit j: element 8 * (block - offset) + j is kept
__device__ __forceinline__ uint32_t keep_bits(uint64_t block, uint64_t seed, const Drop& d) {
  const uint4 r = philox4x32(block, 0, seed);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t keep = 0, tie = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t hi = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
    keep |= (uint32_t)(hi > d.t_hi) << j;
    tie |= (uint32_t)(hi == d.t_hi) << j;
  }
  if (tie) {
    const uint4 s = philox4x32(block, 1, seed);
    const uint32_t v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t lo = (j & 1) ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu;
      keep |= (uint32_t)(lo >= d.t_lo) << j & tie;
    }
  }
  return keep;
}

}  // namespace moe
