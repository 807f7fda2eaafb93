// Products of 4-bit matrices on gfx950: out (M x N) = a (M x K) b (N x K)^T
// with fp32 accumulation, through v_mfma_scale_f32_16x16x128_f8f6f4, which
// multiplies blocks of 32 codes under their two scales.
//
// A wave's 16 x 128 operand is one 1 KiB code tile (muon_mx.h), so tiles go
// from global memory to LDS as they are (LDS-DMA, 1 KiB an instruction) and
// from LDS to registers by conflict-free 16-byte reads; the scale dword of a
// lane holds the bytes of four row tiles, picked by the instruction's byte
// select.  b is the instruction's first operand, so a lane's four results are
// consecutive columns of out.
#include <utility>

#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx.h"
#include "muon_mx_device.h"

namespace muon {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// 4-bit operands use the first four registers of the eight.
template <int SA, int SB>
__device__ __forceinline__ f32x4_t mfma4(i32x4_t a, i32x4_t b, f32x4_t c, int sa, int sb) {
  const i32x8_t a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8_t b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, SA, sa, SB, sb);
}

template <int... I, class F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// One operand of a block: the code tiles of its rows and their scales.  Row
// tiles past the matrix's last are read as the last one again: their products
// are never stored.
template <int ROWS, int NW>
struct Operand {
  static constexpr int kTiles = ROWS / kMxTileR;          // code tiles per stage
  static constexpr int kPer = kTiles / NW;                // ... per wave
  static constexpr int kScaleLanes = ROWS * 4 / 16 / NW;  // lanes of a wave's scale load
  static constexpr int kBytes = ROWS * (kMxTileK / 2);    // codes per stage
  static constexpr int kScales = ROWS * 4;                // scales per stage
  static_assert(kTiles % NW == 0 && kScaleLanes >= 1, "load split");
  u32x4_t codes, scales;
  uint32_t vcode[kPer];    // byte offset of the wave's tiles in the first stage
  uint32_t vscale;

  __device__ __forceinline__ void plan(const uint8_t* c, const uint8_t* s, int row0, int rows,
                                       int kt, int wave, int lane) {
    const int t0 = row0 / kMxTileR, s0 = row0 / kMxScaleRows;
    const int nt = (rows + kMxTileR - 1) / kMxTileR - t0;     // row tiles from here on
    const int ns = (rows + kMxScaleRows - 1) / kMxScaleRows - s0;
    codes = make_desc(c + static_cast<int64_t>(t0) * kt * kMxTileBytes, 0xffffffffu);
    scales = make_desc(s + static_cast<int64_t>(s0) * kt * kMxScaleBytes, 0xffffffffu);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int j = wave + NW * u;
      vcode[u] = static_cast<uint32_t>(j < nt ? j : nt - 1) * kt * kMxTileBytes;
    }
    const int b = (wave * kScaleLanes + lane) * 16;          // byte of the stage's scales
    const int g = b / kMxScaleBytes;
    vscale = static_cast<uint32_t>(g < ns ? g : ns - 1) * kt * kMxScaleBytes + b % kMxScaleBytes;
  }
  __device__ __forceinline__ void load(int k, int wave, int lane, uint8_t* dst, uint8_t* sdst) const {
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      dma16(codes, lds_addr(dst) + (wave + NW * u) * kMxTileBytes, lane * 16,
            vcode[u] + k * kMxTileBytes);
    if (lane < kScaleLanes)
      dma16(scales, lds_addr(sdst) + wave * kScaleLanes * 16, vscale, k * kMxScaleBytes);
  }
};

__device__ __forceinline__ float load_out(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ float load_out(const float* p) { return *p; }
__device__ __forceinline__ void store_out(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }

// TM x TN output tile by WM x WN waves; NST stages of 128 columns in LDS.
template <int ODT, int TM, int TN, int WM, int WN, int NST>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_mx_gemm(MxGemmArgs args) {
  using T = typename std::conditional<ODT == kBF16, uint16_t, float>::type;
  constexpr int NW = WM * WN;
  using OpN = Operand<TN, NW>;
  using OpM = Operand<TM, NW>;
  constexpr int kStage = OpN::kBytes + OpM::kBytes + OpN::kScales + OpM::kScales;
  constexpr int PER = OpN::kPer + OpM::kPer + 2;      // loads per wave per stage
  constexpr int FN = TN / WN / 16, FM = TM / WM / 16; // 16-row operands of a wave
  static_assert(FN % 4 == 0 && FM % 4 == 0, "a wave takes whole scale dwords");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const uint32_t blk = xcd_block();
  const int g = find_in_list(args.base, args.n, blk);
  const MxProduct& p = args.p[g];
  const uint32_t b = blk - args.base[g];
  // groups of GM row tiles, column by column, so that neighbouring blocks of
  // an XCD share both operands
  constexpr int GM = 8;
  const int tm_n = (p.M + TM - 1) / TM, tn_n = (p.N + TN - 1) / TN;
  const int per_group = GM * tn_n;
  const int grp = b / per_group, in = b % per_group;
  const int gm = tm_n - grp * GM < GM ? tm_n - grp * GM : GM;
  const int tm = grp * GM + in % gm, tn = in / gm;

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int kt = p.kt;
  OpN on;
  OpM om;
  on.plan(p.bc, p.bs, tn * TN, p.N, kt, wave, lane);
  om.plan(p.ac, p.as, tm * TM, p.M, kt, wave, lane);

  auto issue = [&](int k) {
    uint8_t* st = smem + (k % NST) * kStage;
    on.load(k, wave, lane, st, st + OpN::kBytes + OpM::kBytes);
    om.load(k, wave, lane, st + OpN::kBytes, st + OpN::kBytes + OpM::kBytes + OpN::kScales);
  };
  f32x4_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int k = 0; k < NST - 1 && k < kt; ++k) issue(k);
  for (int k = 0; k < kt; ++k) {
    wait_ahead<NST - 2, PER>(kt - 1 - k);
    lds_barrier();
    if (k + NST - 1 < kt) issue(k + NST - 1);
    const uint8_t* st = smem + (k % NST) * kStage;
    const uint8_t* sn = st + OpN::kBytes + OpM::kBytes;
    const uint8_t* sm = sn + OpN::kScales;
    i32x4_t fn[FN], fm[FM];
    int dn[FN / 4], dm[FM / 4];
#pragma unroll
    for (int i = 0; i < FN / 4; ++i)
      dn[i] = *reinterpret_cast<const int*>(sn + (wn * (FN / 4) + i) * kMxScaleBytes + lane * 4);
#pragma unroll
    for (int i = 0; i < FM / 4; ++i)
      dm[i] = *reinterpret_cast<const int*>(sm + (wm * (FM / 4) + i) * kMxScaleBytes + lane * 4);
#pragma unroll
    for (int i = 0; i < FN; ++i)
      fn[i] = *reinterpret_cast<const i32x4_t*>(st + (wn * FN + i) * kMxTileBytes + lane * 16);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fm[i] = *reinterpret_cast<const i32x4_t*>(st + OpN::kBytes + (wm * FM + i) * kMxTileBytes + lane * 16);
    unrolled(std::make_integer_sequence<int, FN>{}, [&](auto I) {
      unrolled(std::make_integer_sequence<int, FM>{}, [&](auto J) {
        constexpr int i = decltype(I)::value, j = decltype(J)::value;
        acc[i][j] = mfma4<i & 3, j & 3>(fn[i], fm[j], acc[i][j], dn[i / 4], dm[j / 4]);
      });
    });
  }

  const uint64_t seed = args.drop ? seed_of(args.drop_seed) : 0;
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int r = tm * TM + (wm * FM + j) * 16 + (lane & 15);
    if (r >= p.M) continue;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int c = tn * TN + (wn * FN + i) * 16 + 4 * (lane >> 4);
      if (c >= p.N) continue;
      T* o = out + r * p.ld + c;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if (args.drop) {
        const Words w = philox(c / 8, r, kTagDropout, p.index, seed);
        const uint32_t lo = c & 4 ? w.w[2] : w.w[0], hi = c & 4 ? w.w[3] : w.w[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t q = ((e < 2 ? lo : hi) >> (16 * (e & 1))) & 0xffffu;
          v[e] = q >= args.drop ? v[e] * args.drop_scale : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < p.N) store_out(o + e, args.accumulate ? load_out(o + e) + v[e] : v[e]);
    }
  }
}

template <int ODT, int TM, int TN, int WM, int WN, int NST>
hipError_t launch_tile(const MxGemmArgs& a, int64_t blocks, hipStream_t s) {
  constexpr int NW = WM * WN;
  constexpr int lds = NST * (Operand<TN, NW>::kBytes + Operand<TM, NW>::kBytes +
                             Operand<TN, NW>::kScales + Operand<TM, NW>::kScales);
  const void* f = reinterpret_cast<const void*>(&k_mx_gemm<ODT, TM, TN, WM, WN, NST>);
  static_assert(lds <= 160 * 1024, "LDS");
  const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_mx_gemm<ODT, TM, TN, WM, WN, NST>), dim3(static_cast<uint32_t>(blocks)),
                     dim3(64 * NW), lds, s, a);
  return hipGetLastError();
}

template <int ODT>
hipError_t launch_odt(const MxGemmArgs& a, int tile, int64_t blocks, hipStream_t s) {
  return launch_tile<ODT, 128, 128, 2, 2, 4>(a, blocks, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, int odt, int tile, int64_t blocks, hipStream_t s) {
  return odt == kBF16 ? launch_odt<kBF16>(a, tile, blocks, s) : launch_odt<kF32>(a, tile, blocks, s);
}

}  // namespace muon
