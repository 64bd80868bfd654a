// The counter-based generator behind dropout: Philox4x32-10 (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  Ten
// rounds of two 32x32 -> 64 bit products turn a 128-bit counter and a 64-bit
// key into four independent 32-bit words, so any thread can make the numbers
// of any element on its own and a mask never has to be stored.
#pragma once

#include <stdint.h>

namespace moe {

__host__ __device__ __forceinline__ void philox_round(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
  const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c[0];
  const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
  c[0] = static_cast<uint32_t>(b >> 32) ^ c[1] ^ k0;
  c[1] = static_cast<uint32_t>(b);
  c[2] = static_cast<uint32_t>(a >> 32) ^ c[3] ^ k1;
  c[3] = static_cast<uint32_t>(a);
}

// The keys of the ten rounds, for callers that make many counters' words.
struct PhiloxKeys {
  uint32_t k[20];
};
__host__ __device__ __forceinline__ PhiloxKeys philox_keys(uint64_t seed) {
  PhiloxKeys keys;
  keys.k[0] = static_cast<uint32_t>(seed);
  keys.k[1] = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 1; r < 10; ++r) {
    keys.k[2 * r] = keys.k[2 * r - 2] + 0x9E3779B9u;
    keys.k[2 * r + 1] = keys.k[2 * r - 1] + 0xBB67AE85u;
  }
  return keys;
}

// The four words of counter (n, offset).
__host__ __device__ __forceinline__ void philox4x32_10(uint64_t n, uint64_t offset,
                                                       const PhiloxKeys& keys, uint32_t (&c)[4]) {
  c[0] = static_cast<uint32_t>(n);
  c[1] = static_cast<uint32_t>(n >> 32);
  c[2] = static_cast<uint32_t>(offset);
  c[3] = static_cast<uint32_t>(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) philox_round(c, keys.k[2 * r], keys.k[2 * r + 1]);
}

// Dropout's decision for eight consecutive elements (element group n) from the
// words of counter n: element 8 n + i takes the low (even i) or high half of
// word i / 2 and is dropped below `threshold` (0 .. 65535).  16 random bits an
// element, so one call covers a 16-byte vector of bf16 and the drop
// probability is a multiple of 2^-16.
__host__ __device__ __forceinline__ bool dropout_kept(const uint32_t (&w)[4], int i,
                                                      uint32_t threshold) {
  const uint32_t high = i % 2 ? w[i / 2] : w[i / 2] << 16;  // the low half below plays no part
  return high >= threshold << 16;
}

}  // namespace moe
