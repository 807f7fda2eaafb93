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

#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx.h"
#include "muon_mx_device.h"

namespace muon {
namespace {

// Code of |t| <= 6 (t already divided by the scale) rounded stochastically:
// up where 256 times the fraction of the step exceeds r + 1/2.
__device__ __forceinline__ uint32_t code_sr(float t, uint32_t r) {
  const float a = fabsf(t);
  const float inv = a >= 4.f ? 0.5f : a >= 2.f ? 1.f : 2.f;
  const uint32_t base = a >= 4.f ? 4u : a >= 2.f ? 2u : 0u;
  const float q = a * inv, low = floorf(q);
  const uint32_t up = (q - low) * 256.f > static_cast<float>(r) + 0.5f;
  return static_cast<uint32_t>(low) + up + base + ((__float_as_uint(t) >> 28) & 8u);
}

// 16 loaded elements of a row as fp32 (exact for both types).
template <int DT>
__device__ __forceinline__ void load16(const void* row, int c0, int cols, bool vec, float* v) {
  if constexpr (DT == kBF16) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + c0;
    if (vec && c0 + 16 <= cols) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_t q = *glb(reinterpret_cast<const u32x4_t*>(p) + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * h + 2 * i] = __uint_as_float(q[i] << 16);
          v[8 * h + 2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = c0 + i < cols ? __uint_as_float(static_cast<uint32_t>(*glb(p + i)) << 16) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(row) + c0;
    if (vec && c0 + 16 <= cols) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const u32x4_t q = *glb(reinterpret_cast<const u32x4_t*>(p) + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(q[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = c0 + i < cols ? *glb(p + i) : 0.f;
    }
  }
}

template <int DT>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (DT == kBF16) return __uint_as_float(static_cast<uint32_t>(f2bf(v)) << 16);
  else return v;
}

// Dropout of 16 consecutive elements of a row (c0 a multiple of 16): eight
// 16-bit numbers a counter.
template <int DT>
__device__ __forceinline__ void drop16(float* v, uint32_t row, uint32_t c0, uint32_t index,
                                       uint64_t seed, uint32_t thr, float scale) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const Words w = philox(c0 / 8 + h, row, kTagDropout, index, seed);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = (w.w[i / 2] >> (16 * (i & 1))) & 0xffffu;
      v[8 * h + i] = r >= thr ? rounded<DT>(v[8 * h + i] * scale) : 0.f;
    }
  }
}

// Eight codes of a block in a dword, element i in bits 4 i.
template <bool SR>
__device__ __forceinline__ uint32_t encode8(const float* v, uint32_t byte, const uint32_t* r8) {
  if constexpr (SR) {
    uint32_t out = 0;
    // 2^(127 - byte), an ordinary number: a finite block's byte is at most 253
    const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out |= code_sr(v[i] * inv, (r8[i / 4] >> (8 * (i & 3))) & 255u) << (4 * i);
    return byte == kMxNan ? 0u : out;
  } else {
    return encode8_near(v, byte);
  }
}

// One 128 x 128 tile of the input per block of four waves.  A lane reads 16
// consecutive elements of a row, so a block of 32 is a pair of lanes; waves 0
// and 1 take the tile's first 64 rows, waves 2 and 3 the others, each wave
// eight rows of every 16-row tile, so a lane ends up with the scale dword of
// its four row tiles.  For the transpose the tile passes through LDS, and a
// lane takes two columns of 32 rows.
template <int DT, bool ROWS, bool COLS, bool SR>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantArgs args) {
  constexpr int T = kMxQuantTile;
  using S = typename std::conditional<DT == kBF16, uint16_t, float>::type;
  __shared__ __attribute__((aligned(16))) S tile[COLS ? T * T : 16];
  const int g = find_in_list(args.base, args.n, blockIdx.x);
  const MxQuantMat& m = args.m[g];
  const uint32_t b = blockIdx.x - args.base[g];
  const int kt = (m.cols + T - 1) / T;               // tiles along the columns
  const int tr = b / kt, tc = b % kt;
  const int t = threadIdx.x;
  const int ch = t & 7;                              // 16-column chunk of the tile
  const int c0 = tc * T + ch * 16;
  const int r16 = (t >> 3) & 15;                     // row inside a 16-row tile
  const uint64_t seed = SR ? seed_of(args.seed) : 0;
  const uint64_t dseed = args.drop ? seed_of(args.drop_seed) : 0;
  uint32_t sdw = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = (t >> 7) * 64 + i * 16 + r16;
    const int r = tr * T + lr;
    float v[16];
    if (r < m.rows) {
      const char* row = static_cast<const char*>(m.in) + static_cast<int64_t>(r) * m.ld * sizeof(S);
      load16<DT>(row, c0, m.cols, m.vec, v);
      if (args.drop) drop16<DT>(v, r, c0, m.index, dseed, args.drop, args.drop_scale);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
    if constexpr (COLS) {
      if constexpr (DT == kBF16) {
        u32x4_t q[2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          q[j / 4][j & 3] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xffff0000u);
        *reinterpret_cast<u32x4_t*>(tile + lr * T + ch * 16) = q[0];
        *reinterpret_cast<u32x4_t*>(tile + lr * T + ch * 16 + 8) = q[1];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(tile + lr * T + ch * 16 + 4 * j) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    if constexpr (ROWS) {
      const uint32_t byte = scale_byte(max_pair(top_of<kF32, 16>(reinterpret_cast<const uint32_t*>(v))));
      Words w = {{0, 0, 0, 0}};
      if constexpr (SR) w = philox(c0 / 16, r, kTagRound, m.index, seed);
      uint2 code;
      code.x = encode8<SR>(v, byte, w.w);
      code.y = encode8<SR>(v + 8, byte, w.w + 2);
      const int rt = tr * (T / 16) + (t >> 7) * 4 + i;   // 16-row tile
      if (rt * 16 < m.rows) {
        const int64_t o = (static_cast<int64_t>(tc) * ((m.rows + 15) / 16) + rt) * kMxTileBytes +
                          ((ch >> 1) * 16 + r16) * 16 + (ch & 1) * 8;
        *glb(reinterpret_cast<uint2*>(m.codes + o)) = code;
      }
      sdw |= byte << (8 * i);
    }
  }
  if constexpr (ROWS) {
    const int sg = tr * 2 + (t >> 7);                    // 64-row scale tile
    if ((ch & 1) == 0 && sg * 64 < m.rows)
      *glb(reinterpret_cast<uint32_t*>(m.scales + (static_cast<int64_t>(tc) * ((m.rows + 63) / 64) + sg) * kMxScaleBytes +
                                       ((ch >> 1) * 16 + r16) * 4)) = sdw;
  }
  if constexpr (COLS) {
    __syncthreads();
    const int cp = t & 63, rb = t >> 6;                  // column pair, block of 32 rows
    float v[2][32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if constexpr (DT == kBF16) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(tile + (rb * 32 + j) * T + 2 * cp);
        v[0][j] = __uint_as_float(q << 16);
        v[1][j] = __uint_as_float(q & 0xffff0000u);
      } else {
        const float2 q = *reinterpret_cast<const float2*>(tile + (rb * 32 + j) * T + 2 * cp);
        v[0][j] = q.x;
        v[1][j] = q.y;
      }
    }
    const int rtt = (m.cols + 15) / 16, sgt = (m.cols + 63) / 64;   // the transpose's row and scale tiles
    uint32_t sb = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = tc * T + 2 * cp + e;                 // row of the transpose
      const uint32_t byte = scale_byte(top_of<kF32, 32>(reinterpret_cast<const uint32_t*>(v[e])));
      sb |= byte << (8 * e);
      u32x4_t code;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Words w = {{0, 0, 0, 0}};
        if constexpr (SR) w = philox((tr * T + rb * 32) / 16 + h, c, kTagRoundT, m.index, seed);
        code[2 * h] = encode8<SR>(v[e] + 16 * h, byte, w.w);
        code[2 * h + 1] = encode8<SR>(v[e] + 16 * h + 8, byte, w.w + 2);
      }
      const int rt = c >> 4;
      if (rt * 16 < m.cols)
        *glb(reinterpret_cast<u32x4_t*>(m.codes_t + (static_cast<int64_t>(tr) * rtt + rt) * kMxTileBytes +
                                        (rb * 16 + (c & 15)) * 16)) = code;
    }
    // the four columns c, c + 16, c + 32, c + 48 of a scale dword are eight lanes apart
    const uint32_t s1 = __shfl_down(sb, 8, 64), s2 = __shfl_down(sb, 16, 64), s3 = __shfl_down(sb, 24, 64);
    const int c = tc * T + 2 * cp;
    if ((cp & 24) == 0 && (c & ~63) < m.cols) {
      uint2 d;
      d.x = (sb & 255) | (s1 & 255) << 8 | (s2 & 255) << 16 | (s3 & 255) << 24;
      d.y = (sb >> 8) | (s1 >> 8) << 8 | (s2 >> 8) << 16 | (s3 >> 8) << 24;
      *glb(reinterpret_cast<uint2*>(m.scales_t + (static_cast<int64_t>(tr) * sgt + (c >> 6)) * kMxScaleBytes +
                                    (rb * 16 + (c & 15)) * 4)) = d;
    }
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  uint4 q;
  q.x = pack_bf16(v[0], v[1]);
  q.y = pack_bf16(v[2], v[3]);
  q.z = pack_bf16(v[4], v[5]);
  q.w = pack_bf16(v[6], v[7]);
  *glb(reinterpret_cast<u32x4_t*>(p)) = u32x4_t{q.x, q.y, q.z, q.w};
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *glb(reinterpret_cast<float4*>(p)) = make_float4(v[0], v[1], v[2], v[3]);
  *glb(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *glb(p) = f2bf(v); }
__device__ __forceinline__ void store1(float* p, float v) { *glb(p) = v; }

// A lane turns four bytes (eight codes) into eight consecutive elements of a
// row, so 16 lanes write 128 consecutive elements.
template <int DT>
__global__ __launch_bounds__(256) void k_mx_dequantize(MxDequantArgs args) {
  constexpr int T = kMxQuantTile;
  using S = typename std::conditional<DT == kBF16, uint16_t, float>::type;
  const int g = find_in_list(args.base, args.n, blockIdx.x);
  const MxDequantMat& m = args.m[g];
  const uint32_t b = blockIdx.x - args.base[g];
  const int kt = (m.cols + T - 1) / T;
  const int tr = b / kt, tc = b % kt;
  const int t = threadIdx.x;
  const int ch = t & 15, r16 = t >> 4;
  const int c = tc * T + ch * 8;
  if (c >= m.cols) return;
#pragma unroll
  for (int i = 0; i < T / 16; ++i) {
    const int rt = tr * (T / 16) + i, r = rt * 16 + r16;
    if (r >= m.rows) return;
    const int slot = (ch >> 2) * 16 + r16;
    const uint32_t code = *glb(reinterpret_cast<const uint32_t*>(
        m.codes + (static_cast<int64_t>(tc) * ((m.rows + 15) / 16) + rt) * kMxTileBytes + slot * 16 + (ch & 3) * 4));
    const uint32_t byte = *glb(m.scales + (static_cast<int64_t>(tc) * ((m.rows + 63) / 64) + (rt >> 2)) * kMxScaleBytes +
                               slot * 4 + (rt & 3));
    // 2^(byte - 127) in fp32 (2^-127 is subnormal); 255 is NaN
    const float sc = byte == kMxNan ? __uint_as_float(0x7fc00000u)
                                    : byte ? __uint_as_float(byte << 23) : 0x1p-127f;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t q = code >> (4 * j);
      // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 doubled are the digits of this word
      const uint32_t d = (0xC8643210u >> (4 * (q & 7u))) & 15u;
      v[j] = static_cast<float>(d) * 0.5f * sc;
      v[j] = __uint_as_float(__float_as_uint(v[j]) ^ ((q & 8u) << 28));
    }
    S* row = static_cast<S*>(m.out) + static_cast<int64_t>(r) * m.ld;
    if (m.vec && c + 8 <= m.cols) {
      store8(row + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < m.cols) store1(row + c + j, v[j]);
    }
  }
}

// Groups of eight consecutive elements of a row, one counter each.
template <int DT>
__global__ __launch_bounds__(256) void k_dropout(MxDropArgs a) {
  using S = typename std::conditional<DT == kBF16, uint16_t, float>::type;
  const int groups = (a.cols + 7) / 8;
  const int64_t total = static_cast<int64_t>(a.rows) * groups;
  const uint64_t seed = seed_of(a.seed);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kDropItems;
#pragma unroll
  for (int u = 0; u < kDropItems / 256; ++u) {
    const int64_t it = first + u * 256 + threadIdx.x;
    if (it >= total) return;
    const int r = static_cast<int>(it / groups), c = static_cast<int>(it - static_cast<int64_t>(r) * groups) * 8;
    const S* in = static_cast<const S*>(a.in) + r * a.ldi + c;
    S* out = static_cast<S*>(a.out) + r * a.ldo + c;
    const bool whole = a.vec && c + 8 <= a.cols;
    float v[8];
    if (whole) {
      if constexpr (DT == kBF16) {
        const u32x4_t q = *glb(reinterpret_cast<const u32x4_t*>(in));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(q[i] << 16);
          v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t q = *glb(reinterpret_cast<const u32x4_t*>(in) + h);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(q[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (DT == kBF16) v[i] = c + i < a.cols ? __uint_as_float(static_cast<uint32_t>(*glb(in + i)) << 16) : 0.f;
        else v[i] = c + i < a.cols ? *glb(in + i) : 0.f;
      }
    }
    const Words w = philox(c / 8, r, kTagDropout, 0, seed);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t q = (w.w[i / 2] >> (16 * (i & 1))) & 0xffffu;
      v[i] = q >= a.drop ? v[i] * a.scale : 0.f;
    }
    if (whole) {
      store8(out, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.cols) store1(out + i, v[i]);
    }
  }
}

template <int DT, bool SR>
void quantize_rc(const MxQuantArgs& a, bool rows, bool cols, dim3 grid, hipStream_t s) {
  if (rows && cols) hipLaunchKernelGGL((k_mx_quantize<DT, true, true, SR>), grid, dim3(256), 0, s, a);
  else if (rows) hipLaunchKernelGGL((k_mx_quantize<DT, true, false, SR>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mx_quantize<DT, false, true, SR>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, int dt, bool rows, bool cols, bool stochastic,
                              int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (dt == kBF16) {
    if (stochastic) quantize_rc<kBF16, true>(a, rows, cols, grid, s);
    else quantize_rc<kBF16, false>(a, rows, cols, grid, s);
  } else {
    if (stochastic) quantize_rc<kF32, true>(a, rows, cols, grid, s);
    else quantize_rc<kF32, false>(a, rows, cols, grid, s);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxDequantArgs& a, int dt, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (dt == kBF16) hipLaunchKernelGGL((k_mx_dequantize<kBF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mx_dequantize<kF32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dropout(const MxDropArgs& a, int dt, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (dt == kBF16) hipLaunchKernelGGL((k_dropout<kBF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_dropout<kF32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
