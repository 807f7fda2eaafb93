// Elementwise kernels of the 4-bit operators on gfx950: quantisation to
// microscaled 4-bit blocks (along rows, along columns, or both from one read),
// reading back, and dropout.  The number format and the random numbers are
// stated in include/muon.h, the storage in muon_mx.h.
//
// Blocks of 32 along the contraction share the scale 2^e, e the smallest
// integer >= -127 with max|x| <= 6 * 2^e.  With u the bits of max|x| as fp32,
// the biased exponent is ((u + 0x3FFFFF) >> 23) - 2: the addend carries into
// the exponent exactly when the significand exceeds 1.5.
#pragma clang fp contract(off)

#include <type_traits>

#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx.h"
#include "muon_mx_device.h"

namespace muon {
namespace {

constexpr int kQuantThreads = 1024;

// Elements of a row as they are in memory: a dword holds two bf16 or one fp32.
template <int DT> struct Elem;
template <> struct Elem<kBF16> {
  using S = uint16_t;
  static constexpr int kPerDword = 2;
};
template <> struct Elem<kF32> {
  using S = float;
  static constexpr int kPerDword = 1;
};

// Sixteen elements of a row from column c on; zeros past the last column.
template <int DT>
__device__ __forceinline__ void load16(const typename Elem<DT>::S* row, int c, int cols, uint32_t* q) {
  constexpr int NV = 4 / Elem<DT>::kPerDword;   // 16-byte loads
  if (c + 16 <= cols) {
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const u32x4_t v = load16b(row + c + h * (16 / NV));
#pragma unroll
      for (int i = 0; i < 4; ++i) q[4 * h + i] = v[i];
    }
  } else {
    // every load is in range, so that all are in flight at once
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) q[i] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = c + i < cols ? c + i : cols - 1;
      if constexpr (DT == kBF16) {
        const uint32_t v = *glb(row + at);
        q[i / 2] |= (c + i < cols ? v : 0u) << (16 * (i & 1));
      } else {
        const uint32_t v = __float_as_uint(*glb(row + at));
        q[i] = c + i < cols ? v : 0u;
      }
    }
  }
}

// Dropout of sixteen elements (columns c .. c + 15, c a multiple of 16), rounded
// to the element type as a stored result would be.
template <int DT>
__device__ __forceinline__ void drop16(uint32_t* q, uint32_t row, uint32_t c, uint32_t index,
                                       uint64_t seed, const MxDrop& d) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
    if constexpr (DT == kBF16) {
      widen8(u32x4_t{q[4 * h], q[4 * h + 1], q[4 * h + 2], q[4 * h + 3]}, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(q[8 * h + i]);
    }
    drop8(v, c / 8 + h, row, index, seed, d);
    if constexpr (DT == kBF16) {
      const u32x4_t n = narrow8(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[4 * h + i] = n[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[8 * h + i] = __float_as_uint(v[i]);
    }
  }
}

// Code of an fp32 x over its scale (magnitude at most 6) rounded
// stochastically: up where 256 times the fraction of the step exceeds r + 1/2.
__device__ __forceinline__ uint32_t code_sr(float x, uint32_t byte, uint32_t r) {
  // 2^(127 - byte), an ordinary number: a finite block's byte is at most 253
  const float t = x * __uint_as_float((254u - byte) << 23), a = fabsf(t);
  const float inv = a >= 4.f ? 0.5f : a >= 2.f ? 1.f : 2.f;
  const uint32_t base = a >= 4.f ? 4u : a >= 2.f ? 2u : 0u;
  const float q = a * inv, low = floorf(q);
  const uint32_t up = (q - low) * 256.f > static_cast<float>(r) + 0.5f;
  return static_cast<uint32_t>(low) + up + base + ((__float_as_uint(t) >> 28) & 8u);
}

// The same for eight bf16 elements in four dwords.  Each is scaled to 2^-126
// times its place on the grid, where the grid's steps are fp32 bit patterns 2^22
// apart (the subnormal grid falls on the fp32 subnormals), so with the pattern
// shifted up by two the code is its top byte, and adding the random byte below
// carries into the code exactly when the element goes up: the threshold
// (2 r + 1) / 512 of a step lies ((255 - r) << 16) + 0x7FFC below the next
// (three more change nothing: the pattern's last two bits are zero).  What
// scaling rounds away of a bf16's eight digits is below every threshold.  The
// signs come from the elements' own top bytes.  Byte selects throughout: the
// instruction count bounds the kernel.
__device__ __forceinline__ uint32_t bytes(uint32_t hi, uint32_t lo, uint32_t select) {
  return __builtin_amdgcn_perm(hi, lo, select);
}
__device__ __forceinline__ uint32_t encode8_sr(const uint32_t* q, uint32_t byte, const uint32_t* r8) {
  const int up = 1 - static_cast<int>(byte);
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = i & 1 ? q[i / 2] & 0xffff0000u : q[i / 2] << 16;
    const uint32_t s = __float_as_uint(__builtin_ldexpf(__uint_as_float(x), up));
    t[i] = (s << 2) + bytes(0x7FFFu, ~r8[i / 4], 0x06000504u | (i & 3) << 16);
  }
  constexpr uint32_t kLow = 0x0c0c0703u, kHigh = 0x07030c0cu;   // the two top bytes, below or above
  const uint32_t even = bytes(t[2], t[0], kLow) | bytes(t[6], t[4], kHigh);
  const uint32_t odd = bytes(t[3], t[1], kLow) | bytes(t[7], t[5], kHigh);
  const uint32_t neg_even = (bytes(q[1], q[0], 0x0c0c0501u) | bytes(q[3], q[2], 0x05010c0cu)) & 0x80808080u;
  const uint32_t neg_odd = (bytes(q[1], q[0], kLow) | bytes(q[3], q[2], kHigh)) & 0x80808080u;
  return even | odd << 4 | neg_even >> 4 | neg_odd;
}

// Eight codes of a block in a dword, element i in bits 4 i; r8: their random
// bytes.  (q: dwords of the eight elements.)
template <int DT, bool SR>
__device__ __forceinline__ uint32_t encode8(const uint32_t* q, uint32_t byte, const uint32_t* r8) {
  if constexpr (SR) {
    uint32_t out = 0;
    if constexpr (DT == kBF16) {
      out = encode8_sr(q, byte, r8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        out |= code_sr(__uint_as_float(q[i]), byte, (r8[i / 4] >> (8 * (i & 3))) & 255u) << (4 * i);
    }
    return byte == kMxNan ? 0u : out;
  } else if constexpr (DT == kBF16) {
    return encode8_near(u32x4_t{q[0], q[1], q[2], q[3]}, byte);
  } else {
    return encode8_near(reinterpret_cast<const float*>(q), byte);
  }
}

// One 128 x 128 tile of the input per block of sixteen waves.  A lane reads 16
// consecutive elements of one row, so a block of 32 is a pair of lanes; for the
// transpose the tile passes through LDS and a pair of lanes takes 32 rows of a
// column.  Short work per lane keeps small matrices quick and costs large ones
// nothing: with four waves of four times the work, both orientations of bf16 on
// MI355X, us (4 | 16 waves): 1 x 2560 3.8 | 3.1; 1024 x 1024 4.1 | 3.4; 8192 x
// 2560 14.8 | 14.5; 16384 x 10240 98.8 | 96.5 (5.3 TB/s, as a copy).  To nearest
// memory is the bound.  Stochastically it is the instruction count: the
// generator's products and the roundings keep the vector units busy 96 % of the
// time at 2.4 GHz, 16384 x 10240 of bf16 both ways 138 us (161 before the
// byte selects of encode8_sr).
template <class Args, int DT, bool ROWS, bool COLS, bool SR>
__global__ __launch_bounds__(kQuantThreads) void k_mx_quantize(Args args) {
  constexpr int T = kMxQuantTile, PD = Elem<DT>::kPerDword, ND = 16 / PD;   // dwords of 16 elements
  using S = typename Elem<DT>::S;
  static_assert(kQuantThreads * 16 == T * T, "a lane takes 16 elements");
  __shared__ __attribute__((aligned(16))) uint32_t tile[COLS ? T * T / PD : 4];
  const int g = find_in_list(args, blockIdx.x);
  const MxQuantMat& m = args.m[g];
  const uint32_t b = blockIdx.x - args.base[g];
  const int kt = (m.cols + T - 1) / T;               // tiles along the columns
  const int tr = b / kt, tc = b % kt;
  const int t = threadIdx.x;
  const int ch = t & 7, lr = t >> 3;                 // 16-column chunk and row of the tile
  const int c0 = tc * T + ch * 16, r = tr * T + lr;
  uint32_t q[ND];
  load16<DT>(static_cast<const S*>(m.in) + static_cast<int64_t>(r < m.rows ? r : m.rows - 1) * m.ld,
             c0, m.cols, q);
  const uint64_t seed = SR ? seed_of(args.c.seed) : 0;
  if (r >= m.rows)
#pragma unroll
    for (int j = 0; j < ND; ++j) q[j] = 0;
  if (args.c.drop.threshold) drop16<DT>(q, r, c0, m.index, seed_of(args.c.drop.seed), args.c.drop);
  // a tile row's quarters swap in pairs every sixteen rows, so that lanes that
  // read rows sixteen apart find them in different banks
  constexpr int kSwap = T / PD / 4;
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < ND; j += 4)
      *reinterpret_cast<u32x4_t*>(tile + lr * (T / PD) + ((ch * ND + j) ^ ((lr >> 4 & 1) * kSwap))) =
          u32x4_t{q[j], q[j + 1], q[j + 2], q[j + 3]};
  }
  if constexpr (ROWS) {
    const uint32_t byte = scale_byte(max_pair(top_of<DT, ND>(q)));
    Words w = {{0, 0, 0, 0}};
    if constexpr (SR) w = philox(c0 / 16, r, kTagRound, m.index, seed);
    uint2 code;
    code.x = encode8<DT, SR>(q, byte, w.w);
    code.y = encode8<DT, SR>(q + ND / 2, byte, w.w + 2);
    const int rt = r >> 4, slot = (ch >> 1) * 16 + (r & 15);
    if (rt * 16 < m.rows) {
      const int64_t o = (static_cast<int64_t>(tc) * ((m.rows + 15) / 16) + rt) * kMxTileBytes;
      *glb(reinterpret_cast<uint2*>(m.codes + o + slot * 16 + (ch & 1) * 8)) = code;
      if ((ch & 1) == 0)
        *glb(m.scales + (static_cast<int64_t>(tc) * ((m.rows + 63) / 64) + (r >> 6)) * kMxScaleBytes +
             slot * 4 + (rt & 3)) = static_cast<uint8_t>(byte);
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int half = t & 1, lc = (t >> 1) & 127, rb = t >> 8;   // half of a block of 32 rows, column
    const int row0 = rb * 32 + half * 16;
    uint32_t v[ND];                                      // 16 rows of the column
    if constexpr (DT == kBF16) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(tile) + row0 * T + (lc ^ (half * 2 * kSwap));
#pragma unroll
      for (int j = 0; j < 16; j += 2) v[j / 2] = h[j * T] | static_cast<uint32_t>(h[(j + 1) * T]) << 16;
    } else {
      const uint32_t* h = tile + row0 * T + (lc ^ (half * kSwap));
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = h[j * T];
    }
    const int c = tc * T + lc;                           // row of the transpose
    const uint32_t byte = scale_byte(max_pair(top_of<DT, ND>(v)));
    Words w = {{0, 0, 0, 0}};
    if constexpr (SR) w = philox((tr * T + row0) / 16, c, kTagRoundT, m.index, seed);
    uint2 code;
    code.x = encode8<DT, SR>(v, byte, w.w);
    code.y = encode8<DT, SR>(v + ND / 2, byte, w.w + 2);
    const int rt = c >> 4, slot = rb * 16 + (c & 15);
    if (rt * 16 < m.cols) {
      *glb(reinterpret_cast<uint2*>(m.codes_t + (static_cast<int64_t>(tr) * ((m.cols + 15) / 16) + rt) * kMxTileBytes +
                                    slot * 16 + half * 8)) = code;
      if (half == 0)
        *glb(m.scales_t + (static_cast<int64_t>(tr) * ((m.cols + 63) / 64) + (c >> 6)) * kMxScaleBytes +
             slot * 4 + (rt & 3)) = static_cast<uint8_t>(byte);
    }
  }
}

// A lane turns four bytes (eight codes) into eight consecutive elements of a
// row, so 16 lanes write 128 consecutive elements.
template <class Args, int DT>
__global__ __launch_bounds__(256) void k_mx_dequantize(Args args) {
  constexpr int T = kMxQuantTile;
  using S = typename Elem<DT>::S;
  const int g = find_in_list(args, blockIdx.x);
  const MxDequantMat& m = args.m[g];
  const uint32_t b = blockIdx.x - args.base[g];
  const int kt = (m.cols + T - 1) / T;
  const int tr = b / kt, tc = b % kt;
  const int t = threadIdx.x;
  const int ch = t & 15, r16 = t >> 4;
  const int c = tc * T + ch * 8;
  if (c >= m.cols) return;
  const int slot = (ch >> 2) * 16 + r16;
  const int rts = (m.rows + 15) / 16, sgs = (m.rows + 63) / 64;
  uint32_t codes[T / 16], scales[T / 64];
#pragma unroll
  for (int i = 0; i < T / 16; ++i) {
    const int rt = tr * (T / 16) + i < rts ? tr * (T / 16) + i : rts - 1;
    codes[i] = *glb(reinterpret_cast<const uint32_t*>(
        m.codes + (static_cast<int64_t>(tc) * rts + rt) * kMxTileBytes + slot * 16 + (ch & 3) * 4));
  }
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    const int sg = tr * (T / 64) + i < sgs ? tr * (T / 64) + i : sgs - 1;
    scales[i] = *glb(reinterpret_cast<const uint32_t*>(
        m.scales + (static_cast<int64_t>(tc) * sgs + sg) * kMxScaleBytes + slot * 4));
  }
#pragma unroll
  for (int i = 0; i < T / 16; ++i) {
    const int r = tr * T + i * 16 + r16;
    if (r >= m.rows) return;
    const uint32_t byte = (scales[i / 4] >> (8 * (i & 3))) & 255u;
    // 2^(byte - 127) in fp32 (2^-127 is subnormal); 255 is NaN
    const float sc = byte == kMxNan ? __uint_as_float(0x7fc00000u)
                                    : byte ? __uint_as_float(byte << 23) : 0x1p-127f;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t q = codes[i] >> (4 * j);
      // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 doubled are the digits of this word
      const uint32_t d = (0xC8643210u >> (4 * (q & 7u))) & 15u;
      v[j] = static_cast<float>(d) * 0.5f * sc;
      v[j] = __uint_as_float(__float_as_uint(v[j]) ^ ((q & 8u) << 28));
    }
    S* o = static_cast<S*>(m.out) + static_cast<int64_t>(r) * m.ld + c;
    if (c + 8 <= m.cols) {
      store8(o, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < m.cols) store1(o + j, v[j]);
    }
  }
}

// Groups of eight consecutive elements of a row, one counter and one lane each.
template <int DT>
__global__ __launch_bounds__(kDropItems) void k_dropout(MxDropArgs a) {
  using S = typename Elem<DT>::S;
  const uint32_t groups = (a.cols + 7) / 8;
  const uint64_t seed = seed_of(a.drop.seed);
  // the block's first group (a scalar division), then this lane's
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kDropItems;
  uint32_t r = static_cast<uint32_t>(first / groups);
  uint32_t g = static_cast<uint32_t>(first - static_cast<uint64_t>(r) * groups) + threadIdx.x;
  if (groups >= kDropItems) {
    if (g >= groups) {
      g -= groups;
      ++r;
    }
  } else {
    const uint32_t over = g / groups;
    g -= over * groups;
    r += over;
  }
  if (r >= static_cast<uint32_t>(a.rows)) return;
  const int c = g * 8;
  const S* in = static_cast<const S*>(a.in) + r * a.ldi + c;
  S* out = static_cast<S*>(a.out) + r * a.ldo + c;
  const bool whole = c + 8 <= a.cols;
  float v[8];
  if (whole) {
    load8(in, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load1(c + i < a.cols ? in + i : in);
  }
  drop8(v, g, r, 0, seed, a.drop);
  if (whole) {
    store8(out, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) store1(out + i, v[i]);
  }
}

template <class Args, int DT, bool SR>
void quantize_rc(const Args& a, bool rows, bool cols, dim3 grid, hipStream_t s) {
  const dim3 block(kQuantThreads);
  if (rows && cols) hipLaunchKernelGGL((k_mx_quantize<Args, DT, true, true, SR>), grid, block, 0, s, a);
  else if (rows) hipLaunchKernelGGL((k_mx_quantize<Args, DT, true, false, SR>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_mx_quantize<Args, DT, false, true, SR>), grid, block, 0, s, a);
}

template <class Args>
void quantize_dt(const Args& a, int dt, bool rows, bool cols, bool stochastic, dim3 grid, hipStream_t s) {
  if (dt == kBF16) {
    if (stochastic) quantize_rc<Args, kBF16, true>(a, rows, cols, grid, s);
    else quantize_rc<Args, kBF16, false>(a, rows, cols, grid, s);
  } else {
    if (stochastic) quantize_rc<Args, kF32, true>(a, rows, cols, grid, s);
    else quantize_rc<Args, kF32, false>(a, rows, cols, grid, s);
  }
}

template <class Args>
void dequantize_dt(const Args& a, int dt, dim3 grid, hipStream_t s) {
  if (dt == kBF16) hipLaunchKernelGGL((k_mx_dequantize<Args, kBF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mx_dequantize<Args, kF32>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, int dt, bool rows, bool cols, bool stochastic,
                              int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (a.n == 1) quantize_dt(list_of_one(a), dt, rows, cols, stochastic, grid, s);
  else quantize_dt(a, dt, rows, cols, stochastic, grid, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxDequantArgs& a, int dt, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (a.n == 1) dequantize_dt(list_of_one(a), dt, grid, s);
  else dequantize_dt(a, dt, grid, s);
  return hipGetLastError();
}

hipError_t launch_dropout(const MxDropArgs& a, int dt, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (dt == kBF16) hipLaunchKernelGGL((k_dropout<kBF16>), grid, dim3(kDropItems), 0, s, a);
  else hipLaunchKernelGGL((k_dropout<kF32>), grid, dim3(kDropItems), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
