// Device helpers shared by the 4-bit operators: random numbers and the lookup
// of a block's matrix in a grouped launch.
#pragma once
#include "muon_mx.h"

namespace muon {
namespace {

__device__ __forceinline__ uint64_t seed_of(const MxSeed& s) { return s.dev ? *s.dev : s.value; }

// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011).
struct Words { uint32_t w[4]; };
__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint64_t seed) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// Matrix of a grouped launch that block b belongs to: the bases are in rising
// order, so it is the number of bases at or below b, counted across a wave.
__device__ __forceinline__ int find_in_list(const uint32_t* base, int n, uint32_t b) {
  if (n == 1) return 0;
  const int lane = threadIdx.x & 63;
  const bool below = lane < n && base[lane < n ? lane : 0] <= b;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(below))) - 1;
}

}  // namespace
}  // namespace muon
