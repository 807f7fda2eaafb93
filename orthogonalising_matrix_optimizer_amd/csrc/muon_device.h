// Device helpers shared by the MFMA kernels (gfx950): LDS-DMA loads and the
// waits that order them, bf16 packing, XCD-aware block order.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {
namespace {

// Buffer descriptor word 3 for raw (untyped) loads.
constexpr uint32_t kRsrcWord3 = 0x00020000u;

// fp32 -> bf16, round to nearest even: gfx950 converts a pair per
// instruction (v_cvt_pk_bf16_f32); NaN stays NaN.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}
__device__ __forceinline__ uint16_t f2bf(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Raw buffer descriptor over `bytes` bytes at `base` (reads past the end
// return zero).  All fields are block-uniform and live in SGPRs.
__device__ __forceinline__ u32x4_t make_desc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  u32x4_t d;
  d[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  d[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32) & 0xffffu);
  d[2] = __builtin_amdgcn_readfirstlane(bytes);
  d[3] = kRsrcWord3;
  return d;
}

// LDS byte address of a __shared__ location.
__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  // the low half of a flat address in the LDS aperture is the LDS address (an
  // address-space cast here adds a null check that one compiler release
  // fails to select in the single-launch kernel)
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

// One 1 KiB LDS-DMA load: lane L copies 16 bytes from global offset
// voff + soff of the descriptor's buffer to LDS address lds + 16 L.  It is
// issued as inline assembly so that the compiler does not order later LDS
// reads of *other* stage buffers behind it; wait_vm orders it explicitly.
// It has no result register.
// (M0 is reserved for the compiler's own M0 users, which set it right before
// each use; the clobber keeps it from assuming a value survives.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const u32x4_t& d, uint32_t lds, uint32_t voff,
                                      uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(d), "s"(soff)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// Wait until at most n of this wave's vector loads are outstanding (loads
// complete in issue order); LDS and export counters are left alone.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Wait until a stage has landed when min(ahead, MAXA) later stages of PER
// loads each were issued after it.
template <int MAXA, int PER>
__device__ __forceinline__ void wait_ahead(int ahead) {
  if constexpr (MAXA == 0) {
    wait_vm<0>();
  } else {
    if (ahead >= MAXA) wait_vm<MAXA * PER>();
    else wait_ahead<MAXA - 1, PER>(ahead);
  }
}

// Workgroup barrier without a memory fence.  Stage data arrive by LDS DMA
// and are covered by wait_vm before it.  The wave's own LDS reads must have
// returned before it: the compiler is free to sink the MFMAs of the previous
// stage, and the waits for their operands, below a bare s_barrier, and a
// wave past the barrier may then refill (or stage output into) a buffer that
// a slower wave is still reading.  The wait sits in the same statement so
// that nothing can separate the two.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Logical block index: blocks are dealt round-robin to the eight XCDs; this
// gives each XCD a contiguous range of logical tiles, so tiles that share
// operand panels run on the same L2.
__device__ __forceinline__ int xcd_block() {
  const int nb = gridDim.x, b = blockIdx.x;
  const int q = nb >> 3, r = nb & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

}  // namespace
}  // namespace muon
