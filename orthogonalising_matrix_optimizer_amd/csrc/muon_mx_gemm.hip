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
#include <algorithm>
#include <atomic>
#include <type_traits>
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

// One operand of a work item: the code tiles of its rows and their scales, one
// step of 128 columns a stage.  Row tiles past the matrix's last are read as
// the last one again: their products are never stored.  The stage's scales are
// one load, by wave SW (a load costs as much with few lanes as with all).
template <int ROWS, int NW, int SW>
struct Operand {
  static constexpr int kPer = ROWS / kMxTileR / NW;       // row tiles of a wave
  static constexpr int kBytes = ROWS * (kMxTileK / 2);    // codes per stage
  static constexpr int kScales = ROWS * 4;                // scales per stage
  static constexpr int kScaleLanes = kScales / 16;
  static_assert(ROWS / kMxTileR % NW == 0 && kScaleLanes <= 64 && SW < NW, "load split");
  uint64_t codes, scales;  // the next stage's row panel
  uint64_t kcode, kscale;  // bytes from one stage to the next
  uint32_t vcode[kPer];    // byte offsets of the lane's pieces in a panel
  uint32_t vscale;

  __device__ __forceinline__ void plan(const uint8_t* c, const uint8_t* s, int row0, int rows,
                                       int k0, int wave, int lane) {
    const int t0 = row0 / kMxTileR, s0 = row0 / kMxScaleRows;
    const int rt = (rows + kMxTileR - 1) / kMxTileR, st = (rows + kMxScaleRows - 1) / kMxScaleRows;
    kcode = static_cast<uint64_t>(rt) * kMxTileBytes;
    kscale = static_cast<uint64_t>(st) * kMxScaleBytes;
    codes = reinterpret_cast<uint64_t>(c) + k0 * kcode + static_cast<uint64_t>(t0) * kMxTileBytes;
    scales = reinterpret_cast<uint64_t>(s) + k0 * kscale + static_cast<uint64_t>(s0) * kMxScaleBytes;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int j = wave + NW * u;
      vcode[u] = (j < rt - t0 ? j : rt - t0 - 1) * kMxTileBytes + lane * 16;
    }
    const int g = lane * 16 / kMxScaleBytes;
    vscale = (g < st - s0 ? g : st - s0 - 1) * kMxScaleBytes + lane * 16 % kMxScaleBytes;
  }
  // Loads the stage and moves on; dst, sdst: LDS addresses of its codes and scales.
  __device__ __forceinline__ void load(int wave, int lane, uint32_t dst, uint32_t sdst) {
    const u32x4_t dc = make_desc(reinterpret_cast<const void*>(codes), kBytes);
#pragma unroll
    for (int u = 0; u < kPer; ++u) dma16(dc, dst + (wave + NW * u) * kMxTileBytes, vcode[u], 0);
    if (wave == SW) {
      const u32x4_t ds = make_desc(reinterpret_cast<const void*>(scales), kScales);
      if (lane < kScaleLanes) dma16(ds, sdst, vscale, 0);
    }
    codes += kcode;
    scales += kscale;
  }
};

// Work item b of a launch: product, tile origin and contraction range.
struct Item {
  const MxProduct* p;
  int m0, n0, k0, k1, split;
};
template <int TM, int TN, class Args>
__device__ __forceinline__ Item item_of(const Args& args, uint32_t b) {
  const int g = find_in_list(args, b);
  const MxProduct& p = args.m[g];
  const int in_product = static_cast<int>(b - args.base[g]);
  Item it;
  it.p = &p;
  it.split = in_product / p.tiles;
  const int t = in_product % p.tiles;
  // groups of GM row tiles, column by column, so that neighbouring blocks of
  // an XCD share both operands
  constexpr int GM = 8;
  const int tm_n = (p.M + TM - 1) / TM, tn_n = (p.N + TN - 1) / TN;
  const int per_group = GM * tn_n;
  const int grp = t / per_group, in = t % per_group;
  const int gm = tm_n - grp * GM < GM ? tm_n - grp * GM : GM;
  it.m0 = (grp * GM + in % gm) * TM;
  it.n0 = in / gm * TN;
  it.k0 = it.split * p.chunk;
  it.k1 = it.k0 + p.chunk < p.kt ? it.k0 + p.chunk : p.kt;
  return it;
}

// Register operands of one stage for a wave: FN row tiles of b, FM of a.
//
// The 16 results of an instruction that a lane group holds are four
// consecutive rows of the first operand.  So that a lane ends up with eight
// consecutive columns of out (16-byte stores), two operands of b share 32
// rows: row r of the even one is row 8 (r / 4) + 4 (r / 8) + r % 4 of the 32,
// row r of the odd one the same with the other half of the eight.  (The halves
// swap at r = 8 so that 16 lanes still read 16 different 16-byte slots.)
template <int FN, int FM>
struct Frags {
  i32x4_t n[FN], m[FM];
  uint32_t dn[FN / 2];
  int dm[FM / 4];
};

// Wait until a stage has landed when `ahead` (at most MAXA) later stages of PER
// loads each, and EXTRA stores if `extra`, were issued after it.
template <int MAXA, int PER, int EXTRA>
__device__ __forceinline__ void wait_stage(int ahead, bool extra) {
  if constexpr (MAXA == 0) {
    if (extra) wait_vm<(EXTRA < 63 ? EXTRA : 63)>();
    else wait_vm<0>();
  } else {
    if (ahead >= MAXA) {
      if (extra) wait_vm<(MAXA * PER + EXTRA < 63 ? MAXA * PER + EXTRA : 63)>();
      else wait_vm<MAXA * PER>();
    } else {
      wait_stage<MAXA - 1, PER, EXTRA>(ahead, extra);
    }
  }
}

// TM x TN output tiles by WM x WN waves; a ring of NST stages of 128 columns
// in LDS, loaded NST - 1 stages ahead.  A block takes work items in turn (all
// blocks of an XCD neighbouring ones) and the stages of its items form one
// sequence, so an item's stores run beside the next item's loads.  PER_CU
// blocks share a CU, and one multiplies while another waits at its barrier.
// KEEP: the output goes into the caches, else past them.
//
// Measured on MI355X (random codes, 16384 x 2560 outputs, K = 10240): 256 x 128
// tiles of four waves, two blocks a CU, 3.9-4.3 PF; 128 x 128, three blocks,
// 3.5-3.8; 256 x 256 of eight waves 3.6-3.9 (with the two waves of a SIMD
// alternating between reads and products 2.9).  What bounds it: loads into LDS
// and products hardly overlap.  The instruction alone sustains 9.5 PF on zeros and
// 7.1 on random codes, so 16384 x 4096 x 10240 would take 145 and 194 us; the
// loads alone take 194, and 156 from L2 (28 TB/s); together they take 304 us on
// zeros and 424 on random codes, with every stage in L2 278 and 360.  In the
// products of a 2560 x 10240 layer the matrix units are busy 34-43 % of the time at
// 2.1-2.2 GHz, LDS reads 15-19 %, and waves wait for LDS 5-7 % of theirs.
template <class Args, int ODT, int TM, int TN, int WM, int WN, int NST, int PER_CU, bool DROP, bool KEEP>
__global__ __launch_bounds__(64 * WM * WN, PER_CU * WM * WN / 4) void k_mx_gemm(Args args) {
  using T = typename std::conditional<ODT == kBF16, uint16_t, float>::type;
  constexpr int NW = WM * WN;
  using OpN = Operand<TN, NW, 0>;
  using OpM = Operand<TM, NW, 1>;
  constexpr int kStage = OpN::kBytes + OpM::kBytes + OpN::kScales + OpM::kScales;
  constexpr int PER = OpN::kPer + OpM::kPer;          // loads per wave per stage; waves 0 and 1
                                                      // load scales too
  constexpr int FN = TN / WN / 16, FM = TM / WM / 16; // 16-row operands of a wave
  static_assert(FN % 4 == 0 && FM % 4 == 0, "a wave takes whole scale dwords");
  static_assert(NST >= 2, "ring");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lds = lds_addr(smem);

  // items of this block: XCD x (blocks b = x mod 8) owns a contiguous range
  const uint32_t grid = gridDim.x, x = blockIdx.x & 7, loc = blockIdx.x >> 3;
  const uint32_t first = args.c.xcd[x], last = args.c.xcd[x + 1];
  const uint32_t step = (grid + 7 - x) >> 3;

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // ---- loads: run NST stages ahead of the products
  uint32_t ld_item = first + loc;
  int ld_k = 0, ld_k1 = 0, ld_slot = 0;
  int issued = 0;                       // stages issued so far
  OpN on;
  OpM om;
  auto ld_open = [&]() {                // plan ld_item, skipping items without stages
    while (ld_item < last) {
      const Item it = item_of<TM, TN>(args, ld_item);
      ld_k = it.k0;
      ld_k1 = it.k1;
      if (ld_k < ld_k1) {
        on.plan(it.p->bc, it.p->bs, it.n0, it.p->N, it.k0, wave, lane);
        om.plan(it.p->ac, it.p->as, it.m0, it.p->M, it.k0, wave, lane);
        return;
      }
      ld_item += step;
    }
  };
  auto issue = [&]() {                  // the next stage of the sequence, if there is one
    if (ld_item >= last) return;
    const uint32_t st = lds + ld_slot * kStage;
    on.load(wave, lane, st, st + OpN::kBytes + OpM::kBytes);
    om.load(wave, lane, st + OpN::kBytes, st + OpN::kBytes + OpM::kBytes + OpN::kScales);
    ld_slot = ld_slot + 1 == NST ? 0 : ld_slot + 1;
    ++issued;
    if (++ld_k == ld_k1) {
      ld_item += step;
      ld_open();
    }
  };

  // ---- register operands
  const int r = lane & 15, kb = lane >> 4, half = r >> 3;
  const int even = 8 * (r >> 2) + 4 * half + (r & 3), odd = 8 * (r >> 2) + 4 * (1 - half) + (r & 3);
  const int off_e = (even >> 4) * kMxTileBytes + kb * 256 + (even & 15) * 16;
  const int off_o = (odd >> 4) * kMxTileBytes + kb * 256 + (odd & 15) * 16;
  const int soff_e = (kb * 16 + (even & 15)) * 4, soff_o = (kb * 16 + (odd & 15)) * 4;
  int rd_slot = 0;
  auto read = [&](Frags<FN, FM>& f) {   // the stage in rd_slot
    const uint8_t* st = smem + rd_slot * kStage;
    const uint8_t* sn = st + OpN::kBytes + OpM::kBytes;
    const uint8_t* sm = st + OpN::kBytes + OpM::kBytes + OpN::kScales;
    const uint8_t* pn = st + wn * FN * kMxTileBytes;
    const uint8_t* pm = st + OpN::kBytes + wm * FM * kMxTileBytes + lane * 16;
#pragma unroll
    for (int i = 0; i < FN / 4; ++i) {
      const uint8_t* s = sn + (wn * (FN / 4) + i) * kMxScaleBytes;
      f.dn[2 * i] = *reinterpret_cast<const uint32_t*>(s + soff_e);
      f.dn[2 * i + 1] = *reinterpret_cast<const uint32_t*>(s + soff_o);
    }
#pragma unroll
    for (int i = 0; i < FM / 4; ++i)
      f.dm[i] = *reinterpret_cast<const int*>(sm + (wm * (FM / 4) + i) * kMxScaleBytes + lane * 4);
    f.n[0] = *reinterpret_cast<const i32x4_t*>(pn + off_e);
#pragma unroll
    for (int i = 0; i < FM; ++i) f.m[i] = *reinterpret_cast<const i32x4_t*>(pm + i * kMxTileBytes);
#pragma unroll
    for (int i = 1; i < FN; ++i)
      f.n[i] = *reinterpret_cast<const i32x4_t*>(pn + (i & ~1) * kMxTileBytes + (i & 1 ? off_o : off_e));
    rd_slot = rd_slot + 1 == NST ? 0 : rd_slot + 1;
  };

  f32x4_t acc[FN][FM];
  auto multiply = [&](Frags<FN, FM>& f) {
    // lanes of the upper rows use the next row tile's scale byte
#pragma unroll
    for (int i = 0; i < FN / 2; ++i) f.dn[i] >>= 8 * half;
    unrolled(std::make_integer_sequence<int, FN>{}, [&](auto I) {
      unrolled(std::make_integer_sequence<int, FM>{}, [&](auto J) {
        constexpr int i = decltype(I)::value, j = decltype(J)::value;
        acc[i][j] = mfma4<(i & 2), (j & 3)>(f.n[i], f.m[j], acc[i][j], static_cast<int>(f.dn[(i / 4) * 2 + (i & 1)]), f.dm[j / 4]);
      });
    });
  };

  ld_open();
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue();
  int done = 0;                         // stages whose operands were read from LDS
  // stores of a whole tile, and the stages whose loads were issued before them
  constexpr int NSTORE = FM * FN / 2 * (ODT == kBF16 ? 1 : 2);
  int covered = 0;
  // this wave's loads of stage `done` have landed
  const bool scales_too = wave < 2;
  auto wait_next = [&]() {
    if (scales_too) wait_stage<NST - 2, PER + 1, NSTORE>(issued - done - 1, done < covered);
    else wait_stage<NST - 2, PER, NSTORE>(issued - done - 1, done < covered);
  };
  Frags<FN, FM> f;

  for (uint32_t item = first + loc; item < last; item += step) {
    const Item it = item_of<TM, TN>(args, item);
    const MxProduct& p = *it.p;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k = it.k0; k < it.k1; ++k) {
      wait_next();
      lds_barrier();
      read(f);
      ++done;
      // reads first, then the loads, then the products at raised priority
      __builtin_amdgcn_sched_barrier(0);
      issue();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      multiply(f);
      __builtin_amdgcn_s_setprio(0);
    }

    const uint64_t seed = DROP ? seed_of(args.c.drop.seed) : 0;
    T* out = static_cast<T*>(p.out) + it.split * p.stride;
    const bool whole = !args.c.accumulate && it.m0 + TM <= p.M && it.n0 + TN <= p.N;
    covered = whole ? issued : 0;
    // eight columns of a row, from column c = column(i)
    auto column = [&](int i) { return it.n0 + (wn * FN + i) * 16 + 8 * (lane >> 4); };
    auto result = [&](int i, int j, int row, float* v) {
      const bool swap = lane >= 32;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = swap ? acc[i + 1][j][e] : acc[i][j][e];
        v[4 + e] = swap ? acc[i][j][e] : acc[i + 1][j][e];
      }
      if constexpr (DROP) drop8(v, column(i) / 8, row, p.index, seed, args.c.drop);
    };
    // A lane has 16-byte pieces a and b of its row's 128 bytes; lanes r and r + 8
    // swap one, so that a store writes eight whole lines.  (Sixteen half lines past
    // the caches took 1.4 times the bytes to memory: 8192 x 10240, K = 2560, 132
    // against 125 us, 16384 x 10240 283 against 257.)
    const bool up = lane & 8;
    auto put = [&](T* o, u32x4_t a, u32x4_t b, int apart) {
      u32x4_t got;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        got[e] = __builtin_amdgcn_update_dpp(0, up ? a[e] : b[e], 0x128 /* row_ror:8 */, 0xf, 0xf, false);
      o += up ? apart : 0;
      if constexpr (KEEP) {
        store16b(o, up ? got : a);
        store16b(o + 8 * p.ld, up ? b : got);
      } else {
        stream16b(o, up ? got : a);
        stream16b(o + 8 * p.ld, up ? b : got);
      }
    };
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int row = it.m0 + (wm * FM + j) * 16 + r;
      if (whole) {
        T* o = out + (row - (up ? 8 : 0)) * p.ld;
#pragma unroll
        for (int i = 0; i < FN; i += ODT == kBF16 ? 4 : 2) {
          float v[8];
          result(i, j, row, v);
          if constexpr (ODT == kBF16) {
            float w[8];
            result(i + 2, j, row, w);
            put(o + column(i), narrow8(v), narrow8(w), 32);
          } else {
            put(o + column(i), bits4(v), bits4(v + 4), 4);
          }
        }
        continue;
      }
      if (row >= p.M) continue;
#pragma unroll
      for (int i = 0; i < FN; i += 2) {
        const int c = column(i);
        if (c >= p.N) continue;
        float v[8];
        result(i, j, row, v);
        T* o = out + row * p.ld + c;
        if (c + 8 <= p.N) {
          if (args.c.accumulate) {
            float w[8];
            load8(o, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = w[e] + v[e];
          }
          store8(o, v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < p.N) store1(o + e, args.c.accumulate ? load1(o + e) + v[e] : v[e]);
        }
      }
    }
  }
}

constexpr int kCUs = 256;

template <class Args, int ODT, int TM, int TN, int NST, int PER_CU, bool DROP, bool KEEP>
hipError_t launch_tile(const Args& a, hipStream_t s) {
  constexpr int WM = 2, WN = 2, NW = WM * WN;
  using OpN = Operand<TN, NW, 0>;
  using OpM = Operand<TM, NW, 1>;
  constexpr int lds = NST * (OpN::kBytes + OpM::kBytes + OpN::kScales + OpM::kScales);
  static_assert(lds * PER_CU <= 160 * 1024, "LDS");
  auto* k = &k_mx_gemm<Args, ODT, TM, TN, WM, WN, NST, PER_CU, DROP, KEEP>;
  // the LDS limit is raised once per device
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  // as many blocks on every XCD as the longest range has items, if they fit
  int most = 0;
  for (int x = 0; x < 8; ++x) most = std::max(most, a.c.xcd[x + 1] - a.c.xcd[x]);
  const int blocks = std::min(8 * most, kCUs * PER_CU);
  hipLaunchKernelGGL(k, dim3(blocks), dim3(64 * NW), lds, s, a);
  return hipGetLastError();
}

template <class Args, int ODT, bool DROP>
hipError_t launch_keep(const Args& a, int tile_m, bool keep, hipStream_t s) {
  if (tile_m == 256)
    return keep ? launch_tile<Args, ODT, 256, 128, 3, 2, DROP, true>(a, s)
                : launch_tile<Args, ODT, 256, 128, 3, 2, DROP, false>(a, s);
  return keep ? launch_tile<Args, ODT, 128, 128, 3, 3, DROP, true>(a, s)
              : launch_tile<Args, ODT, 128, 128, 3, 3, DROP, false>(a, s);
}

template <class Args>
hipError_t launch_gemm_of(const Args& a, int odt, int tile_m, bool keep, hipStream_t s) {
  const bool drop = a.c.drop.threshold != 0;
  if (odt == kBF16)
    return drop ? launch_keep<Args, kBF16, true>(a, tile_m, keep, s)
                : launch_keep<Args, kBF16, false>(a, tile_m, keep, s);
  return drop ? launch_keep<Args, kF32, true>(a, tile_m, keep, s)
              : launch_keep<Args, kF32, false>(a, tile_m, keep, s);
}

// Sum of the partial products of a split contraction, in the order of the
// splits; eight columns a thread.
template <class Args, int ODT>
__global__ __launch_bounds__(256) void k_mx_reduce(Args args) {
  using T = typename std::conditional<ODT == kBF16, uint16_t, float>::type;
  const int g = find_in_list(args, blockIdx.x);
  const MxReduce& p = args.m[g];
  const uint32_t t = (blockIdx.x - args.base[g]) * 256 + threadIdx.x;
  const uint32_t per_row = p.ldp / 8;
  const uint32_t row = t / per_row, c = (t % per_row) * 8, N = p.N;
  if (row >= static_cast<uint32_t>(p.M)) return;
  const float* in = p.in + static_cast<int64_t>(row) * p.ldp + c;
  float v[8];
  load8(in, v);
  for (int s = 1; s < p.splits; ++s) {
    float w[8];
    load8(in + s * p.stride, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  if (args.c.drop.threshold) drop8(v, c / 8, row, p.index, seed_of(args.c.drop.seed), args.c.drop);
  T* o = static_cast<T*>(p.out) + row * p.ld + c;
  if (c + 8 <= N) {
    if (args.c.accumulate) {
      float w[8];
      load8(o, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = w[e] + v[e];
    }
    store8(o, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < N) store1(o + e, args.c.accumulate ? load1(o + e) + v[e] : v[e]);
  }
}

// At most 16 rows of x, quantised on the way, times b: the waves of a block
// take the steps of 128 columns in turn for R row tiles of b and join their
// sums in LDS in wave order.  Of a step a lane loads eight consecutive
// elements of x (16 lanes a row, so that the loads are whole lines), four lanes
// share a block of 32, and the codes pass through LDS to the lane that feeds
// them to the matrix instruction.  H: groups of four rows of x (1 or 4).
template <int XDT, int ODT, int NW, int R, int U, int H>
__global__ __launch_bounds__(64 * NW) void k_mx_rows(MxRowsArgs a) {
  using X = typename std::conditional<XDT == kBF16, uint16_t, float>::type;
  using T = typename std::conditional<ODT == kBF16, uint16_t, float>::type;
  __shared__ __attribute__((aligned(16))) uint32_t xcodes[NW][256], xscales[NW][64];
  __shared__ f32x4_t part[NW][R][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt0 = blockIdx.x * R, rt = (a.N + 15) / 16, st = (a.N + 63) / 64;
  const int kt = (a.K + kMxTileK - 1) / kMxTileK;
  f32x4_t acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int NQ = XDT == kBF16 ? 1 : 2;   // 16-byte loads of eight elements
  const int row = lane >> 4, ch = lane & 15;
  // rows past x's last are read as the last one again: their sums are not stored
  const X* const xrow = static_cast<const X*>(a.x);
  int64_t xoff[H];
#pragma unroll
  for (int h = 0; h < H; ++h) xoff[h] = (4 * h + row < a.M ? 4 * h + row : a.M - 1) * a.ldx + ch * 8;
  struct Step {
    i32x4_t w[R];
    uint32_t ws;
    u32x4_t x[H][NQ];
  };
  auto load = [&](Step& s, int k) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = rt0 + i < rt ? rt0 + i : rt - 1;
      s.w[i] = *glb(reinterpret_cast<const i32x4_t*>(a.bc + (static_cast<int64_t>(k) * rt + t) * kMxTileBytes) + lane);
    }
    s.ws = *glb(reinterpret_cast<const uint32_t*>(a.bs + (static_cast<int64_t>(k) * st + (rt0 >> 2)) * kMxScaleBytes) + lane);
    const X* p = xrow + k * kMxTileK;
    if ((k + 1) * kMxTileK <= a.K) {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int q = 0; q < NQ; ++q) s.x[h][q] = load16b(p + xoff[h] + q * (8 / NQ));
      return;
    }
    const int c = k * kMxTileK + ch * 8;
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) s.x[h][q] = u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < a.K) {
          if constexpr (XDT == kBF16) s.x[h][0][e / 2] |= static_cast<uint32_t>(*glb(p + xoff[h] + e)) << (16 * (e & 1));
          else s.x[h][e / 4][e & 3] = __float_as_uint(*glb(p + xoff[h] + e));
        }
    }
  };
  auto multiply = [&](const Step& s) {
    uint32_t byte[H], code[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      byte[h] = scale_byte(max_quad(top_of<XDT, NQ * 4>(reinterpret_cast<const uint32_t*>(s.x[h]))));
      if constexpr (XDT == kBF16) code[h] = encode8_near(s.x[h][0], byte[h]);
      else code[h] = encode8_near(reinterpret_cast<const float*>(s.x[h]), byte[h]);
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int slot = (ch >> 2) * 16 + 4 * h + row;
      xcodes[wave][slot * 4 + (ch & 3)] = code[h];
      if ((ch & 3) == 0) xscales[wave][slot] = byte[h];
    }
    // only this wave's own part of LDS, which it reads in order
    __builtin_amdgcn_wave_barrier();
    const i32x4_t xq = *reinterpret_cast<const i32x4_t*>(&xcodes[wave][lane * 4]);
    const int xs = static_cast<int>(xscales[wave][lane]);
    __builtin_amdgcn_wave_barrier();
    const int sw = static_cast<int>(s.ws >> (8 * (rt0 & 3)));
    unrolled(std::make_integer_sequence<int, R>{}, [&](auto I) {
      constexpr int i = decltype(I)::value;
      acc[i] = mfma4<i, 0>(s.w[i], xq, acc[i], sw, xs);
    });
  };
  if constexpr (U == 1) {
    // written as loops over the one step, or the compiler computes the rows'
    // offsets in the loop (16 x 2560 x 2560: 4.6 against 5.0 us)
    for (int k0 = wave; k0 < kt; k0 += NW * U) {
      Step s[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u * NW < kt) load(s[u], k0 + u * NW);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u * NW < kt) multiply(s[u]);
    }
  } else {
    // U steps in flight: against U loaded, then U multiplied, 13 x 10240 x 2560
    // 9.9 and 10.4 us, 1 x 10240 x 2560 5.4 and 5.6
    Step s[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (wave + u * NW < kt) load(s[u], wave + u * NW);
    for (int k0 = wave; k0 < kt; k0 += NW * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * NW;
        if (k >= kt) break;
        multiply(s[u]);
        if (k + NW * U < kt) load(s[u], k + NW * U);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // result (row m, column 4 g + e of tile i) is element e of lane 16 g + m
  for (int t = threadIdx.x; t < R * 256; t += 64 * NW) {
    const int i = t >> 8, m = (t >> 4) & 15, col = t & 15;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += part[w][i][(col >> 2) * 16 + m][col & 3];
    const int n = (rt0 + i) * 16 + col;
    if (m < a.M && n < a.N) store1(static_cast<T*>(a.out) + m * a.ldo + n, s);
  }
}

template <int XDT, int ODT, int NW, int R, int U>
void launch_rows_of(const MxRowsArgs& a, hipStream_t s) {
  const dim3 grid(((a.N + 15) / 16 + R - 1) / R), block(64 * NW);
  if (a.M <= 4) hipLaunchKernelGGL((k_mx_rows<XDT, ODT, NW, R, U, 1>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_mx_rows<XDT, ODT, NW, R, U, 4>), grid, block, 0, s, a);
}

// Row tiles of b a block and waves along the contraction, measured on MI355X
// with b from memory, us (4 tiles x 8 waves | 1 x 16 | 1 x 8):
//   1 x 2560 x 10240 (x rows, K, b rows): 5.2 | 5.9 | 5.4;  16 rows 6.6 | 11.2 | 8.7
//   1 x 10240 x 2560: 10.0 | 6.2 | 8.9;  13 rows 14.4 | 10.6 | 13.2
//   1 x 768 x 768: 2.5 | 2.1 | 2.0;  16 x 768 x 2304: 3.6 | 3.2 | 3.1
// Many rows of b amortise x; a long contraction with few of them needs the waves.
// In between (bf16, graph of launches, 1 x row | 16 rows of x):
//   4096 x 4096: 5.7 | 4.3 | 5.0 and 7.5 | 6.3 | 6.7;  2560 x 4096: 3.8 | 3.4 | 3.5 and 4.8 | 4.4 | 4.4
//   6144 x 6144: 8.4 | 7.3 | 7.9 and 10.5 | 13.3 | 11.9;  2560 x 6144: 4.9 | 4.3 | 4.6 and 6.1 | 7.8 | 6.7
//   6144 x 8192: 9.1 | 8.4 | 8.6 and 11.3 | 14.5 | 12.5;  768 x 8192: 3.2 | 3.0 | 3.0 and 3.8 | 4.8 | 3.7
//   10240 x 10240: 13.1 | 14.6 | 13.8 and 18.5 | 29.2 | 26.2
// So one row would take the sixteen waves up to about 9000 rows of b, sixteen rows
// the four tiles from about 5000 on; between those and 8192 the rule is up to 1.3
// times slower for sixteen rows, and up to 1.1 times at 8192 for one.
// b with at most MUON_MX_FEW_ROWS_MAX_N rows keeps the grid below 2^32 threads.
template <int XDT, int ODT>
hipError_t launch_rows(const MxRowsArgs& a, hipStream_t s) {
  if (a.N >= 8192) launch_rows_of<XDT, ODT, 8, 4, 1>(a, s);
  else if (a.K >= 4096) launch_rows_of<XDT, ODT, 16, 1, 2>(a, s);
  else launch_rows_of<XDT, ODT, 8, 1, 1>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, int odt, int tile_m, bool keep, hipStream_t s) {
  return a.n == 1 ? launch_gemm_of(list_of_one(a), odt, tile_m, keep, s)
                  : launch_gemm_of(a, odt, tile_m, keep, s);
}

hipError_t launch_mx_rows(const MxRowsArgs& a, int xdt, int odt, hipStream_t s) {
  if (xdt == kBF16) return odt == kBF16 ? launch_rows<kBF16, kBF16>(a, s) : launch_rows<kBF16, kF32>(a, s);
  return odt == kBF16 ? launch_rows<kF32, kBF16>(a, s) : launch_rows<kF32, kF32>(a, s);
}

hipError_t launch_mx_reduce(const MxReduceArgs& a, int odt, int64_t blocks, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (odt == kBF16) hipLaunchKernelGGL((k_mx_reduce<MxReduceArgs, kBF16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mx_reduce<MxReduceArgs, kF32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
