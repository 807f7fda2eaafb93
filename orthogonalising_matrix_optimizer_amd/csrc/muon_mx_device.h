// Device helpers shared by the 4-bit operators: random numbers, block scales and
// codes, and the lookup of a block's matrix in a grouped launch.
#pragma once
#include "muon_mx.h"

namespace muon {
namespace {

#if defined(__HIP_DEVICE_COMPILE__)
#define GAS __attribute__((address_space(1)))
#else
#define GAS
#endif
template <class T>
__device__ __forceinline__ GAS T* glb(T* p) { return (GAS T*)(p); }
template <class T>
__device__ __forceinline__ const GAS T* glb(const T* p) { return (const GAS T*)(p); }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Scale byte of a block from the bits of its largest magnitude (fp32), and the
// power of two itself as fp32 bits (255: the block holds an infinity or NaN).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kMxNan;
  const uint32_t e = (top + 0x3FFFFFu) >> 23;
  return e > 2 ? e - 2 : 0;
}

__device__ __forceinline__ uint64_t seed_of(const MxSeed& s) { return s.dev ? *s.dev : s.value; }

// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011).
struct Words { uint32_t w[4]; };
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);   // one instruction for the two
#else
  return a ^ b ^ c;
#endif
}
__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint64_t seed) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
    c1 = static_cast<uint32_t>(p1);
    c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// Matrix of a grouped launch that block b belongs to: the bases are in rising
// order, so it is the number of bases at or below b, counted across a wave.
template <class L>
__device__ __forceinline__ int find_in_list(const L& l, uint32_t b) {
  if constexpr (L::kCap == 1) return 0;
  const int lane = threadIdx.x & 63;
  const bool below = lane < l.n && l.base[lane < l.n ? lane : 0] <= b;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(below))) - 1;
}

// 16 bytes at any element's address: the hardware needs no more alignment.
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
template <class T>
__device__ __forceinline__ u32x4_t load16b(const T* p) {
  return *reinterpret_cast<const GAS u32x4_any*>(glb(p));
}
template <class T>
__device__ __forceinline__ void store16b(T* p, u32x4_t q) {
  *reinterpret_cast<GAS u32x4_any*>(glb(p)) = q;
}
// Output written past the caches' keeping (operand panels stay in L2).
template <class T>
__device__ __forceinline__ void stream16b(T* p, u32x4_t q) {
  __builtin_nontemporal_store(q, reinterpret_cast<GAS u32x4_any*>(glb(p)));
}

// Eight consecutive elements of a row as fp32, and back.
__device__ __forceinline__ void widen8(u32x4_t q, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(q[i] << 16);
    v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4_t narrow8(const float* v) {
  return u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ u32x4_t bits4(const float* v) {
  return u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) { widen8(load16b(p), v); }
__device__ __forceinline__ void load8(const float* p, float* v) {
  const u32x4_t a = load16b(p), b = load16b(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[4 + i] = __uint_as_float(b[i]);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) { store16b(p, narrow8(v)); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  store16b(p, bits4(v));
  store16b(p + 4, bits4(v + 4));
}
__device__ __forceinline__ float load1(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*glb(p)) << 16);
}
__device__ __forceinline__ float load1(const float* p) { return *glb(p); }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *glb(p) = f2bf(v); }
__device__ __forceinline__ void store1(float* p, float v) { *glb(p) = v; }

// Eight elements of the dropout mask applied: element i of group g of a row.
__device__ __forceinline__ void drop8(float* v, uint32_t g, uint32_t row, uint32_t index,
                                      uint64_t seed, const MxDrop& d) {
  const Words w = philox(g, row, kTagDropout, index, seed);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = ((w.w[i / 2] >> (16 * (i & 1))) & 0xffffu) >= d.threshold ? v[i] * d.scale : 0.f;
}

// Eight codes of a block in a dword, element i in bits 4 i, rounded to nearest
// (ties to the even code): the conversion reads only the scale's exponent.
__device__ __forceinline__ uint32_t encode8_near(const float* v, uint32_t byte) {
  const float sc = __uint_as_float(byte << 23);
  uint32_t out = 0;
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0], v[1], sc, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2], v[3], sc, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4], v[5], sc, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6], v[7], sc, 3);
  return byte == kMxNan ? 0u : out;
}

// The same for eight bf16 elements in four dwords, which need no widening.
__device__ __forceinline__ bf16x2_t bf16_pair(uint32_t q) { return __builtin_bit_cast(bf16x2_t, q); }
__device__ __forceinline__ uint32_t encode8_near(u32x4_t q, uint32_t byte) {
  const float sc = __uint_as_float(byte << 23);
  uint32_t out = 0;
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, bf16_pair(q[0]), sc, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, bf16_pair(q[1]), sc, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, bf16_pair(q[2]), sc, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, bf16_pair(q[3]), sc, 3);
  return byte == kMxNan ? 0u : out;
}

// Bits of the largest magnitude as fp32, of n dwords of two bf16 or one fp32.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
template <int DT, int N>
__device__ __forceinline__ uint32_t top_of(const uint32_t* q) {
  if constexpr (DT == kBF16) {
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, q[i] & 0x7fff7fffu));
    return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = umax(m, q[i] & 0x7fffffffu);
    return m;
  }
}

// Largest of a value over a pair (four) of neighbouring lanes.
__device__ __forceinline__ uint32_t max_pair(uint32_t v) {
  return umax(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
}
__device__ __forceinline__ uint32_t max_quad(uint32_t v) {
  v = max_pair(v);
  return umax(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

}  // namespace
}  // namespace muon
