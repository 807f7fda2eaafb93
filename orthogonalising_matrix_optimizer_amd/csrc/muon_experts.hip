// Products of ragged groups of rows with their experts' matrices on gfx950 MFMA.
//
// The rows of expert e are the sorted slots offsets[e] .. offsets[e+1]-1, which
// only the device knows.  Three products, C = R C^T in the general form, where
// the operand of the output's rows and that of its columns hold the contraction
// either along their rows in memory ("along") or across them ("across"):
//   fwd: out rows = slots, columns = out features; x along, w along
//   dx:  out rows = slots, columns = in features;  dy along, w across
//   dw:  out rows = out features, columns = in features, contraction over the
//        expert's slots; dy across, x across
// A block computes one tile; it finds its expert by a wave's sum over the
// experts' tile counts.  Blocks are dealt to XCDs so that each works on a
// contiguous range of tiles, which share operand panels in its L2.
//
// LDS holds stages of BK contraction elements.  An operand along the
// contraction is kept as rows of 16-byte chunks, XOR-swizzled by row, read by
// 16-byte reads; one across it as contraction rows, from which the transposing
// read builds operands.  Contraction elements past the end are zeros in both
// operands, so that nothing of a neighbour (a NaN, say) enters a sum.
//
// bf16 operands whose rows start at 16 bytes and hold whole 16-byte pieces go
// straight to LDS (LDS-DMA), which zeroes what a lane points past the buffer's
// end.  All others are loaded into registers and checked there.  fp32 operands
// are split there into three bf16 terms, each the rounding of what the terms before
// leave (24 bits in all), and six of the nine products of terms are summed, the largest
// left out being that of the second and third with at most 2^-24 of the first's: an fp32
// product in six bf16 matrix instructions, which together run at 2.7 times the rate
// of the fp32 matrix instruction (which keeps subnormal bf16 operands and fp32 sums).
//
// The four results that the matrix instruction leaves in consecutive registers
// are rows of its first operand, which is that of the output's columns.  Its 32
// rows are taken in an order that leaves a lane 16 consecutive columns of
// one output row.
//
// Measured, 64 experts in bf16: 16384 x 6 slots, 2048 -> 1408 gathered 595 us (0.94 PF;
// 495 on zeros, whose lower power leaves the clock at 2.35 GHz instead of 1.92; the matrix
// instructions alone 407, the loads alone 390); 49146 slots, 1408 -> 2048: fwd 365, dx 355, dw
// into fp32 485 (738 MB of stores).  48 slots: 29, the used matrices once.
#include <atomic>
#include <type_traits>

#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx_device.h"
#include "muon_sparse.h"

namespace muon {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

constexpr uint32_t kPast = kExpertSpan;    // an offset past every buffer: reads as zeros
constexpr int kBatch = 64;                // experts looked at at once

// ---- the tile of a block
struct Tile {
  int e;        // expert
  int part;     // part of a split contraction
  int lo, hi;   // its rows (of a part: the part's)
  int r0, c0;   // first row (fwd, dx: from lo; dw: of the matrix) and column
  bool any;
};

__device__ __forceinline__ int clamp_to(int v, int most) { return v < 0 ? 0 : v < most ? v : most; }

// An expert's rows, whatever the offsets hold.
__device__ __forceinline__ void rows_of(const ExpertArgs& a, int e, int& lo, int& hi) {
  lo = clamp_to(a.offsets[e], a.slots);
  hi = clamp_to(a.offsets[e + 1], a.slots);
  if (hi < lo) hi = lo;
}

// Sum over the lanes below and including this one.
__device__ __forceinline__ int sum_below(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// The experts' rows in pieces of `per`, expert by expert, `across` items a piece:
// XCD x (blocks x, x + 8, ..) has the x-th eighth of the items.
struct Found {
  int e, piece, index, rest;   // expert, piece of it and of all, item of the piece
  bool any;
};
__device__ __forceinline__ int pieces_of(const ExpertArgs& a, int e, int per) {
  int lo = 0, hi = 0;
  if (e < a.experts) rows_of(a, e, lo, hi);
  return (hi - lo + per - 1) / per;
}
__device__ __forceinline__ Found find_piece(const ExpertArgs& a, int per, int across, int lane) {
  int all = 0;
  for (int e0 = 0; e0 < a.experts; e0 += kBatch) all += __shfl(sum_below(pieces_of(a, e0 + lane, per), lane), 63, 64);
  const int64_t items = static_cast<int64_t>(all) * across;
  const int x = blockIdx.x & 7;
  const int64_t item = items * x / 8 + (blockIdx.x >> 3);
  Found f{0, 0, 0, 0, false};
  if (item >= items * (x + 1) / 8) return f;
  f.index = __builtin_amdgcn_readfirstlane(static_cast<int>(item / across));
  f.rest = __builtin_amdgcn_readfirstlane(static_cast<int>(item % across));
  int want = f.index;
  for (int e0 = 0; e0 < a.experts; e0 += kBatch) {
    const int own = pieces_of(a, e0 + lane, per), upto = sum_below(own, lane);
    const uint64_t past = __ballot(upto > want);
    if (past) {
      const int l = __builtin_ctzll(past);
      f.e = __builtin_amdgcn_readfirstlane(e0 + l);
      f.piece = __builtin_amdgcn_readfirstlane(want - __shfl(upto - own, l, 64));
      f.any = true;
      break;
    }
    want -= __shfl(upto, 63, 64);
  }
  return f;
}

// fwd, dx: tiles of TM rows, all columns of a row tile after each other.
template <int TM, int TN>
__device__ __forceinline__ Tile row_tile(const ExpertArgs& a, int lane) {
  const Found f = find_piece(a, TM, (a.cols + TN - 1) / TN, lane);
  Tile t{f.e, 0, 0, 0, f.piece * TM, f.rest * TN, f.any};
  if (t.any) {
    rows_of(a, t.e, t.lo, t.hi);
    t.lo = __builtin_amdgcn_readfirstlane(t.lo);
    t.hi = __builtin_amdgcn_readfirstlane(t.hi);
  }
  return t;
}

// Split contractions of dw: parts of a.chunk rows, all tiles of a part after each
// other.
template <int TM, int TN>
__device__ __forceinline__ Tile part_tile(const ExpertArgs& a, int lane) {
  const int across = (a.cols + TN - 1) / TN, tiles = (a.rows + TM - 1) / TM * across;
  const Found f = find_piece(a, a.chunk, tiles, lane);
  Tile t{f.e, f.index, 0, 0, f.rest / across * TM, f.rest % across * TN, f.any && f.index < a.parts};
  if (t.any) {
    rows_of(a, t.e, t.lo, t.hi);
    t.lo = __builtin_amdgcn_readfirstlane(t.lo) + f.piece * a.chunk;
    t.hi = __builtin_amdgcn_readfirstlane(t.hi);
    t.hi = t.hi < t.lo + a.chunk ? t.hi : t.lo + a.chunk;
  }
  return t;
}

// dw: an eighth of each expert's tiles to an XCD, in turn from another one, so
// that unequal experts load them alike.  (Whole experts on one XCD, the largest
// first, read less but were slower: 49146 rows of 64 experts, 2048 x 1408, 530 against
// 499 us.)
template <int TM, int TN>
__device__ __forceinline__ Tile matrix_tile(const ExpertArgs& a) {
  const int across = (a.cols + TN - 1) / TN, tiles = (a.rows + TM - 1) / TM * across;
  const int share = (tiles + 7) / 8;
  const int i = blockIdx.x >> 3, e = i / share;
  const int at = ((blockIdx.x + e) & 7) * share + i % share;
  Tile t{e, 0, 0, 0, at / across * TM, at % across * TN, e < a.experts && at < tiles};
  if (t.any) {
    rows_of(a, e, t.lo, t.hi);
    t.lo = __builtin_amdgcn_readfirstlane(t.lo);
    t.hi = __builtin_amdgcn_readfirstlane(t.hi);
  }
  return t;
}

// ---- operands
//
// LDS layout of a plane of one operand's stage.  Along the contraction: row r,
// chunk c of BK / 8; 256 bytes (all banks) hold two rows (BK 64) or four (BK
// 32), and the chunk index is XOR-ed so that the 16 rows that 16 lanes read
// together fall into different 16-byte slots: rows 0-15 of the rows' operand,
// and 0-7 and 16-23 of the columns' operand, in whose order the lanes take them.
template <int BK, bool COLS>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (BK == 64) return COLS ? ((r >> 1) & 3) | (r >> 2 & 4) : (r >> 1) & 7;
  else return COLS ? (r >> 2 & 1) | (r >> 3 & 2) : (r >> 2) & 3;
}
template <int BK, bool COLS>
__device__ __forceinline__ int along_off(int r, int c) {
  return r * (BK * 2) + ((c ^ swizzle<BK, COLS>(r)) << 4);
}
// Across: contraction row k, element p; the chunk index XOR-ed so that the 64 bytes
// of four rows that 32 lanes read together fall into different quarters of the
// banks (with 64 elements a row, two rows share the 256 bytes).
template <int R>
__device__ __forceinline__ int turn(int k) {
  return R == 64 ? 4 * (k >> 1 & 1) : 4 * (k & 3);
}
template <int R>
__device__ __forceinline__ int across_off(int k, int p) {
  return k * (R * 2) + (((p >> 3) ^ turn<R>(k)) << 4) + (p & 7) * 2;
}

// fp32 -> three bf16 terms of eight elements, v = h + m 2^-8 + l 2^-16.  The scales keep
// m and l among the numbers that bf16 has: unscaled, the last bits of what is below 2^-110
// would be lost (a sixteenth of a number of 2^-130).  They cost two multiplications an
// element: 1001 x 2 slots, 333 -> 777 with gradients 59 us without, 63 with; 16384 x 2,
// 2048 -> 1024 2590 | 2680.
__device__ __forceinline__ void split8(const float* v, u32x4_t& h, u32x4_t& m, u32x4_t& l) {
  float w[8], r[8];
  h = narrow8(v);
  widen8(h, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (v[e] - w[e]) * 256.f;
  m = narrow8(r);
  widen8(m, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (r[e] - w[e]) * 256.f;
  l = narrow8(r);
}

// A piece of eight bf16 elements moved down by n elements (0 .. 8), zeros behind.
__device__ __forceinline__ u32x4_t moved(u32x4_t q, int n) {
  const bool one = n & 1, two = n & 2, four = n & 4;
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t next = i < 3 ? q[i + 1] : 0;
    r[i] = one ? q[i] >> 16 | next << 16 : q[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = two ? (i < 3 ? r[i + 1] : 0) : r[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = four ? (i < 2 ? r[i + 2] : 0) : r[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = n >= 8 ? 0 : r[i];
  return r;
}

// What a block takes of one operand.
struct Panel {
  const uint8_t* base;   // along: the tile's first row (gathered: the matrix); across: the expert's first row
  int64_t pitch;         // bytes from row to row
  const int32_t* tokens; // gathered: of the expert's (across) or the tile's (along) rows
  int src;               // gathered: rows of the matrix
  int rows;              // along: rows of the tile; across: the contraction length
  int cols;              // along: the contraction length; across: columns of the matrix
  int c0;                // across: the tile's first column
};

// One operand of a block's stages: ROWS rows of the output (or columns, COLS) by BK
// contraction elements, loaded by NW waves.  A wave's share is kPer pieces of 1
// KiB, in which a lane has 16 bytes of LDS: eight elements.
template <int ROWS, int NW, int BK, bool ACROSS, bool COLS, int DT, bool DMA>
struct Side {
  static constexpr int kES = DT == kBF16 ? 2 : 4;
  static constexpr int kPlane = ROWS * BK * 2;                // bytes of a plane of a stage
  static constexpr int kPlanes = DT == kBF16 ? 1 : 3;
  static constexpr int kBytes = kPlane * kPlanes;
  static constexpr int kPer = kPlane / 1024 / NW;
  static constexpr int kReads = ACROSS ? 2 : 1;               // LDS reads of an operand
  static_assert(kPer * NW * 1024 == kPlane && !(DMA && DT != kBF16), "load split");
  Panel p;
  // Along: the lane's rows of the tile (of the matrix when gathered), or -1; for
  // buffer loads their offsets.
  int row[ACROSS ? 1 : kPer];
  int next;               // across, gathered: one of the wave's rows of the next stage, see look()
  u32x4_t q[DMA ? 1 : kPer][DT == kBF16 ? 1 : 2];             // loaded, not yet in LDS
  int move[DMA || DT == kF32 ? 1 : kPer];                     // of bf16 in registers: see load()
  bool moves;
  u32x4_t desc;                                               // LDS-DMA, along and gathered: the buffer
  static constexpr bool kBuffer = !DMA && DT == kF32;         // loads into registers by buffer instructions

  // Place of the lane's piece u: row of the stage and 16-byte chunk in it.
  static __device__ __forceinline__ void place(int u, int wave, int lane, int& r, int& c) {
    constexpr int CPR = (ACROSS ? ROWS : BK) / 8;
    const int slot = (wave + NW * u) * 64 + lane;
    r = slot / CPR;
    c = slot % CPR;
    if constexpr (ACROSS) c ^= turn<ROWS>(r);
    else c ^= swizzle<BK, COLS>(r);
  }
  __device__ __forceinline__ int source(int r) const {   // the matrix's row of a gathered row
    const int t = r < p.rows ? p.tokens[r] : -1;
    return t < p.src ? t : -1;
  }
  __device__ __forceinline__ void plan(const Panel& panel, int wave, int lane) {
    p = panel;
    if constexpr (DMA || kBuffer) {
      const int n = p.tokens ? p.src : p.rows < ROWS ? p.rows : ROWS;
      const int64_t bytes = (n - 1) * p.pitch + int64_t(p.cols) * kES;
      desc = make_desc(p.base, static_cast<uint32_t>(bytes));
    }
    if constexpr (!ACROSS) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        int r, c;
        place(u, wave, lane, r, c);
        row[u] = p.tokens ? source(r) : r < p.rows ? r : -1;
        if constexpr (DMA || kBuffer)
          row[u] = static_cast<int>(row[u] < 0 ? kPast : static_cast<uint32_t>(row[u]) * static_cast<uint32_t>(p.pitch) + c * 8 * kES);
      }
    }
    look(0, wave, lane);
  }
  // Across, gathered: finds the rows of the stage from contraction row k on, each by
  // one lane (row i % kRows of the wave's piece i / kRows).
  static constexpr int kRows = ACROSS ? 512 / ROWS : 1;       // rows of a piece
  static_assert(kPer * kRows <= 64, "a lane for each row");
  __device__ __forceinline__ void look(int k, int wave, int lane) {
    if constexpr (ACROSS) {
      if (p.tokens && k < p.rows && lane < kPer * kRows) next = source(k + (wave + NW * (lane / kRows)) * kRows + lane % kRows);
    }
  }
  // The matrix's row of the lane's piece u, or -1.
  __device__ __forceinline__ int found(int u, int lane) const {
    if constexpr (ACROSS) return __shfl(next, u * kRows + lane / (64 / kRows), 64);
    else return row[u];
  }
  // Whether the stage from contraction element k on is all there, so that its pieces
  // are loaded whole without a look at each.
  __device__ __forceinline__ bool whole(int k) const {
    if constexpr (DMA || (kBuffer && ACROSS)) return true;
    else if constexpr (ACROSS) return k + BK <= p.rows && p.c0 + ROWS <= p.cols;
    else return k + BK <= p.cols;
  }
  // Starts the loads of the stage from contraction element k on; with LDS-DMA to
  // `lds`, else into registers.  (The caller branches on WHOLE, for both operands at
  // once: a join of the two ways between their loads makes the compiler wait there
  // for the loads just issued.)
  template <bool WHOLE>
  __device__ __forceinline__ void load(int k, int wave, int lane, uint32_t lds) {
    if constexpr (DMA) {
      const uint32_t pitch = static_cast<uint32_t>(p.pitch);
      auto issue = [&](const u32x4_t& d, uint32_t soff, auto&& offset) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          int r, c;
          place(u, wave, lane, r, c);
          dma16(d, lds + (wave + NW * u) * 1024, offset(u, r, c), soff);
        }
      };
      if constexpr (!ACROSS) {
        const int left = p.cols - k;
        issue(desc, static_cast<uint32_t>(k) * 2, [&](int u, int, int c) { return c * 8 < left ? static_cast<uint32_t>(row[u]) : kPast; });
      } else if (p.tokens) {
        issue(desc, 0, [&](int u, int, int c) {
          const int at = found(u, lane);
          return at >= 0 && p.c0 + c * 8 < p.cols ? static_cast<uint32_t>(at) * pitch + (p.c0 + c * 8) * 2 : kPast;
        });
      } else {
        const int n = p.rows - k < BK ? p.rows - k : BK;
        issue(make_desc(p.base + k * p.pitch + p.c0 * 2, static_cast<uint32_t>(n - 1) * pitch + static_cast<uint32_t>(p.cols - p.c0) * 2),
              0, [&](int, int r, int c) { return static_cast<uint32_t>(r) * pitch + c * 16; });
      }
    } else if constexpr (kBuffer) {
      // whole pieces by buffer loads, which cost no address arithmetic and read as zeros
      // where a row is not there; columns past the matrix are its next row's, of results
      // that are not stored
      const uint32_t pitch = static_cast<uint32_t>(p.pitch);
      auto fetch = [&](const u32x4_t& d, int u, uint32_t voff, uint32_t soff) {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<void*>(static_cast<uint64_t>(d[1]) << 32 | d[0]), 0, static_cast<int>(d[2]), static_cast<int>(d[3]));
        q[u][0] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff, soff, 0);
        q[u][1] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff + 16, soff, 0);
      };
      if constexpr (ACROSS) {
        const int n = p.rows - k < BK ? p.rows - k : BK;
        const u32x4_t d = p.tokens ? desc
                                   : make_desc(p.base + k * p.pitch, static_cast<uint32_t>(n - 1) * pitch + static_cast<uint32_t>(p.cols) * 4);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          int r, c;
          place(u, wave, lane, r, c);
          const uint32_t at = (p.c0 + c * 8) * 4;
          const int from = p.tokens ? found(u, lane) : r;
          fetch(d, u, from < 0 ? kPast : static_cast<uint32_t>(from) * pitch + at, 0);
        }
      } else if constexpr (WHOLE) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) fetch(desc, u, static_cast<uint32_t>(row[u]), static_cast<uint32_t>(k) * 4);
      } else {
        const uint8_t* base = p.base + static_cast<int64_t>(k) * 4;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          int r, c;
          place(u, wave, lane, r, c);
          const uint32_t voff = static_cast<uint32_t>(row[u]);
          const uint32_t* from = reinterpret_cast<const uint32_t*>(base + (voff == kPast ? 0 : voff));
#pragma unroll
          for (int i = 0; i < 8; ++i) q[u][i / 4][i % 4] = voff != kPast && k + c * 8 + i < p.cols ? glb(from)[i] : 0;
        }
      }
    } else {
      // A row of the tile that is not there reads as its first, a piece that the row's
      // end cuts as the row's last eight elements: put() moves them down, and zeroes what
      // is no element.  (Results of columns past the matrix are not stored.)
      bool any = false;
      const uint8_t* base = ACROSS && !p.tokens ? p.base + k * p.pitch : p.base;
      const int c0 = ACROSS ? p.c0 : k, last = p.cols - 8;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        int r, c;
        place(u, wave, lane, r, c);
        c = c0 + c * 8;
        int at = ACROSS && !p.tokens ? (WHOLE || k + r < p.rows ? r : -1) : found(u, lane);
        const int from = WHOLE || c <= last ? c : last < 0 ? 0 : last;
        move[u] = at < 0 ? 8 : WHOLE ? 0 : c - from < 8 ? c - from : 8;
        any = any || at < 0;
        at = at < 0 ? 0 : at;
        const uint16_t* s = reinterpret_cast<const uint16_t*>(
            base + static_cast<uint64_t>(static_cast<uint32_t>(at)) * static_cast<uint32_t>(p.pitch)) + from;
        if (WHOLE || last >= 0) {
          q[u][0] = load16b(s);
        } else {   // rows of less than eight elements
          q[u][0] = u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (i < p.cols) q[u][0][i / 2] |= static_cast<uint32_t>(glb(s)[i]) << (16 * (i & 1));
        }
      }
      moves = !WHOLE || __ballot(any) != 0;
    }
  }
  // Writes what load() brought into registers to a stage in LDS.
  __device__ __forceinline__ void put(int wave, int lane, uint8_t* stage) {
    if constexpr (!DMA) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        uint8_t* to = stage + (wave + NW * u) * 1024 + lane * 16;
        if constexpr (DT == kBF16) {
          *reinterpret_cast<u32x4_t*>(to) = moves ? moved(q[u][0], move[u]) : q[u][0];
        } else {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(q[u][i / 4][i % 4]);
          u32x4_t h, m, l;
          split8(v, h, m, l);
          *reinterpret_cast<u32x4_t*>(to) = h;
          *reinterpret_cast<u32x4_t*>(to + kPlane) = m;
          *reinterpret_cast<u32x4_t*>(to + 2 * kPlane) = l;
        }
      }
    }
  }
  // The matrix instruction's operand of 32 rows from row0 on, contraction
  // elements 16 kk .. 16 kk + 15, from a plane.
  static __device__ __forceinline__ bf16x8_t frag(const uint8_t* plane, int row0, int kk, int lane) {
    if constexpr (ACROSS) {
      const int g = lane >> 4, i = lane & 15, q = i & 3;
      const int k = 16 * kk + 8 * (g >> 1) + (i >> 2);
      const int col = row0 + (COLS ? 16 * (q & 1) + 8 * (g & 1) + 4 * (q >> 1) : 16 * (g & 1) + 4 * q);
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(plane + across_off<ROWS>(k, col)));
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(plane + across_off<ROWS>(k + 4, col)));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int l = lane & 31;
      const int r = row0 + (COLS ? 16 * (l >> 2 & 1) + 4 * (l >> 3) + (l & 3) : l);
      return *reinterpret_cast<const bf16x8_t*>(plane + along_off<BK, COLS>(r, 2 * kk + (lane >> 5)));
    }
  }
};

// ---- output
//
// A lane holds 16 consecutive columns of its row: four 16-byte pieces of fp32, two
// of bf16 (of two neighbouring operands four).  Stored as they are, an instruction
// would write 16 bytes here and there in 32 rows; so lanes 8 and 16 apart exchange
// pieces first, after which an instruction writes whole lines of 128 bytes: slot
// 2 u + v of a lane has a piece of row 8 u + 16 v + (lane & 7).  (dw of 64 experts'
// 2048 x 1408 in fp32, 738 MB, from 49146 rows: 499 us without, 485 with; past the
// caches 463.)
__device__ __forceinline__ void exchange(u32x4_t (&q)[4], int lane) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      const auto r = __builtin_amdgcn_permlane16_swap(q[u][e], q[u + 1][e], false, false);
      q[u][e] = r[0];
      q[u + 1][e] = r[1];
    }
  const bool up = lane & 8;
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t got = __builtin_amdgcn_update_dpp(0, up ? q[v][e] : q[v + 2][e], 0x128 /* row_ror:8 */, 0xf, 0xf, false);
      q[v][e] = up ? got : q[v][e];
      q[v + 2][e] = up ? q[v + 2][e] : got;
    }
}

// The first n elements of a 16-byte piece, past the caches for outputs that would
// only push the operands out of them.
__device__ __forceinline__ void put_piece(float* o, u32x4_t q, int n, bool past) {
  if (n >= 4) {
    if (past) stream16b(o, q);
    else store16b(o, q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) glb(o)[i] = __uint_as_float(q[i]);
  }
}
__device__ __forceinline__ void put_piece(uint16_t* o, u32x4_t q, int n, bool past) {
  if (n >= 8) {
    if (past) stream16b(o, q);
    else store16b(o, q);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) glb(o)[i] = static_cast<uint16_t>(q[i / 2] >> (16 * (i & 1)));
  }
}

// 16 consecutive columns of a row, n of them there, added to what is.
template <class T>
__device__ __forceinline__ void add16(T* o, const float* v, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (n >= 8 * h + 8) {
      float w[8];
      load8(o + 8 * h, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] += v[8 * h + i];
      store8(o + 8 * h, w);
    } else {
#pragma unroll
      for (int i = 8 * h; i < 8 * h + 8; ++i)
        if (i < n) store1(o + i, load1(o + i) + v[i]);
    }
  }
}

// Puts a step's LDS reads between the products of the step before, two to one of
// them: left alone, the compiler puts them right before their use.
template <int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
  if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS < 2 ? 1 : 2, 0);
  if constexpr (PRODUCTS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    interleave<(READS > 2 ? READS - 2 : 0), PRODUCTS - 1>();
  } else if constexpr (READS > 2) {
    interleave<READS - 2, 0>();
  }
}

// TM x TN tiles by WM x WN waves, a ring of NST stages of BK.
//
// The operands of a step of 16 are read from LDS while the step before is
// multiplied.  Before the last step of a stage the block meets: then its stage has
// been read by all (its slot takes the stage NST further on), the next one is
// there, and its first operands are read beside the last step's products.
template <int OP, int DT, bool DMA, class T, int TM, int TN, int WM, int WN, int BK, int NST>
__global__ __launch_bounds__(64 * WM * WN) void k_experts(ExpertArgs a) {
  constexpr int NW = WM * WN;
  using Rows = Side<TM, NW, BK, OP >= kExpertDw, false, DT, DMA>;
  using Cols = Side<TN, NW, BK, OP != kExpertFwd, true, DT, DMA>;
  constexpr int kStage = Rows::kBytes + Cols::kBytes, PL = Rows::kPlanes;
  constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t lds = lds_addr(smem);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;

  Tile tile;
  if constexpr (OP == kExpertDw) tile = matrix_tile<TM, TN>(a);
  else if constexpr (OP == kExpertPart) tile = part_tile<TM, TN>(a, lane);
  else tile = row_tile<TM, TN>(a, lane);
  if (!tile.any) return;
  const int depth = OP >= kExpertDw ? tile.hi - tile.lo : a.depth;
  const int64_t es = DT == kBF16 ? 2 : 4;
  const uint8_t* rbase = static_cast<const uint8_t*>(a.r);
  const uint8_t* cbase = static_cast<const uint8_t*>(a.c);
  Rows rows;
  Cols cols;
  if constexpr (OP >= kExpertDw) {
    rows.plan({rbase + tile.lo * a.ldr * es, a.ldr * es, nullptr, 0, depth, a.rows, tile.r0}, wave, lane);
    cols.plan({a.tokens ? cbase : cbase + tile.lo * a.ldc * es, a.ldc * es,
               a.tokens ? a.tokens + tile.lo : nullptr, a.src, depth, a.cols, tile.c0}, wave, lane);
  } else {
    const int first = tile.lo + tile.r0;
    rows.plan({a.tokens ? rbase : rbase + first * a.ldr * es, a.ldr * es,
               a.tokens ? a.tokens + first : nullptr, a.src, tile.hi - first, depth, 0}, wave, lane);
    const uint8_t* w = cbase + tile.e * a.wstride * es;
    if constexpr (OP == kExpertFwd)
      cols.plan({w + tile.c0 * a.ldc * es, a.ldc * es, nullptr, 0, a.cols - tile.c0, depth, 0}, wave, lane);
    else
      cols.plan({w, a.ldc * es, nullptr, 0, depth, a.cols, tile.c0}, wave, lane);
  }

  // fp32: the products of each scale have sums of their own, so that the smaller ones add
  // nothing to the rounding of the largest
  constexpr int SETS = PL;
  f32x16_t acc[SETS][FN][FM];
#pragma unroll
  for (int n = 0; n < SETS; ++n)
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[n][i][j] = f32x16_t{};

  const int stages = (depth + BK - 1) / BK;
  constexpr int PER = Rows::kPer + Cols::kPer, KK = BK / 16;
  static_assert(KK % 2 == 0 && (DMA || NST == 2), "steps and stages");
  auto load = [&](int k, int slot) {     // LDS-DMA: all the way; else into registers
    if (k >= stages) return;
    if (rows.whole(k * BK) && cols.whole(k * BK)) {
      rows.template load<true>(k * BK, wave, lane, lds + slot * kStage);
      cols.template load<true>(k * BK, wave, lane, lds + slot * kStage + Rows::kBytes);
    } else {
      rows.template load<false>(k * BK, wave, lane, lds + slot * kStage);
      cols.template load<false>(k * BK, wave, lane, lds + slot * kStage + Rows::kBytes);
    }
    rows.look((k + 1) * BK, wave, lane);
    cols.look((k + 1) * BK, wave, lane);
  };
  auto put = [&](int k, int slot) {
    if (DMA || k >= stages) return;
    rows.put(wave, lane, smem + slot * kStage);
    cols.put(wave, lane, smem + slot * kStage + Rows::kBytes);
  };
  struct Frags { bf16x8_t c[PL][FN], r[PL][FM]; } f[2];
  auto read = [&](Frags& g, int slot, int kk) {
    const uint8_t* sr = smem + slot * kStage;
    const uint8_t* sc = sr + Rows::kBytes;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
#pragma unroll
      for (int i = 0; i < FN; ++i) g.c[p][i] = Cols::frag(sc + p * Cols::kPlane, (wn * FN + i) * 32, kk, lane);
#pragma unroll
      for (int j = 0; j < FM; ++j) g.r[p][j] = Rows::frag(sr + p * Rows::kPlane, (wm * FM + j) * 32, kk, lane);
    }
  };
  auto multiply = [&](const Frags& g) {   // the terms' products, the smallest first
#pragma unroll
    for (int sum = PL == 1 ? 0 : 2; sum >= 0; --sum)
#pragma unroll
      for (int p = 0; p < PL; ++p) {
        const int o = sum - p;
        if (o < 0 || o >= PL) continue;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[sum][i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(g.c[p][i], g.r[o][j], acc[sum][i][j], 0, 0, 0);
      }
  };
  if (stages) {
    if constexpr (DMA) {
#pragma unroll
      for (int k = 0; k < NST; ++k) load(k, k);
      wait_ahead<NST - 1, PER>(stages - 1);
    } else {
      load(0, 0);
      put(0, 0);
      load(1, 1);
      put(1, 1);
      load(2, 0);
    }
    lds_barrier();
    read(f[0], 0, 0);
  }
  constexpr int READS = PL * (FN * Cols::kReads + FM * Rows::kReads), PRODUCTS = (PL == 1 ? 1 : 6) * FN * FM;
  int slot = 0;
  for (int k = 0; k < stages; ++k) {
#pragma unroll
    for (int kk = 0; kk + 1 < KK; ++kk) {
      read(f[(kk + 1) & 1], slot, kk + 1);
      multiply(f[kk & 1]);
      interleave<READS, PRODUCTS>();
    }
    // (behind the last stage this reads operands that are not used: a branch around
    // the products would double the accumulators)
    const int free = slot;
    slot = slot + 1 == NST ? 0 : slot + 1;
    if constexpr (DMA) wait_ahead<NST - 2, PER>(stages - 2 - k);
    lds_barrier();
    put(k + 2, free);
    load(DMA ? k + NST : k + 3, free);
    __builtin_amdgcn_sched_barrier(0);
    read(f[0], slot, 0);
    multiply(f[1]);
    interleave<READS, PRODUCTS>();
    __builtin_amdgcn_sched_barrier(0);
  }

  if constexpr (SETS > 1) {
    // where the first terms' sum is an infinity or NaN that is the result: an operand that
    // is one has no further terms, and the others' sums say nothing more
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float big = acc[0][i][j][q];
          const float rest = (acc[SETS > 1 ? 1 : 0][i][j][q] + acc[SETS > 2 ? 2 : 0][i][j][q] * 0x1p-8f) * 0x1p-8f;
          acc[0][i][j][q] = fabsf(big) < __builtin_inff() ? big + rest : big;
        }
  }
  const int most = OP >= kExpertDw ? a.rows : tile.hi - tile.lo;
  T* out = static_cast<T*>(a.out) + (OP == kExpertPart ? tile.part * a.ostride : OP == kExpertDw ? tile.e * a.ostride : tile.lo * a.ldo);
  if (OP == kExpertDw && a.accumulate) {
    if (depth == 0) return;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = tile.r0 + (wm * FM + j) * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int c = tile.c0 + (wn * FN + i) * 32 + 16 * (lane >> 5);
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = acc[0][i][j][q];
        if (r < most && c < a.cols) add16(out + r * a.ldo + c, v, a.cols - c);
      }
    }
    return;
  }
  constexpr bool PAIR = sizeof(T) == 2 && FN % 2 == 0;   // two operands' pieces make a line
  constexpr int EACH = 16 / sizeof(T);                   // elements of a piece
  const int u = lane >> 3 & 1, v = lane >> 4 & 1, h = lane >> 5;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int r0 = tile.r0 + (wm * FM + j) * 32;
#pragma unroll
    for (int i = 0; i < FN; i += PAIR ? 2 : 1) {
      const int c0 = tile.c0 + (wn * FN + i) * 32;
      if constexpr (sizeof(T) == 4 || PAIR) {
        u32x4_t q[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float w[8];
#pragma unroll
          for (int e = 0; e < EACH; ++e) w[e] = PAIR ? acc[0][i + n / 2 * PAIR][j][8 * (n & 1) + e] : acc[0][i][j][(4 * n + e) & 15];
          if constexpr (PAIR) q[n] = narrow8(w);
          else q[n] = bits4(w);
        }
        exchange(q, lane);
        const int c = c0 + (PAIR ? 32 * u + 16 * h + 8 * v : 16 * h + 8 * u + 4 * v);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int r = r0 + 8 * (n >> 1) + 16 * (n & 1) + (lane & 7);
          if (r < most && c < a.cols) put_piece(out + r * a.ldo + c, q[n], a.cols - c, a.past);
        }
      } else {
        const int r = r0 + (lane & 31), c = c0 + 16 * h;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = acc[0][i][j][8 * n + e];
          if (r < most && c + 8 * n < a.cols) put_piece(out + r * a.ldo + c + 8 * n, narrow8(w), a.cols - c - 8 * n, a.past);
        }
      }
    }
  }
}

template <int OP, int DT, bool DMA, class T, int TM, int TN, int WM, int WN, int BK, int NST>
hipError_t launch_tiles(const ExpertArgs& a, hipStream_t s) {
  constexpr int NW = WM * WN;
  using Rows = Side<TM, NW, BK, OP >= kExpertDw, false, DT, DMA>;
  using Cols = Side<TN, NW, BK, OP != kExpertFwd, true, DT, DMA>;
  constexpr int lds = NST * (Rows::kBytes + Cols::kBytes);
  static_assert(lds <= 160 * 1024, "LDS");
  auto* k = &k_experts<OP, DT, DMA, T, TM, TN, WM, WN, BK, NST>;
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
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(expert_blocks(a, OP, TM, TN))), dim3(64 * NW), lds, s, a);
  return hipGetLastError();
}

template <int OP, class T>
hipError_t launch_op(const ExpertArgs& a, int dt, bool aligned, int tile, hipStream_t s) {
  if (tile == 64) {
    if (dt == kF32) return launch_tiles<OP, kF32, false, T, 64, 64, 2, 2, 32, 2>(a, s);
    if (!aligned) return launch_tiles<OP, kBF16, false, T, 64, 64, 2, 2, 64, 2>(a, s);
    return launch_tiles<OP, kBF16, true, T, 64, 64, 2, 2, 64, 3>(a, s);
  }
  if constexpr (OP != kExpertPart) {   // always 64
    if (dt == kF32) return launch_tiles<OP, kF32, false, T, 128, 128, 2, 4, 32, 2>(a, s);
    if (!aligned) return launch_tiles<OP, kBF16, false, T, 128, 128, 2, 2, 64, 2>(a, s);
    if (tile == 128) return launch_tiles<OP, kBF16, true, T, 128, 128, 2, 2, 64, 2>(a, s);
    return launch_tiles<OP, kBF16, true, T, 256, 256, 2, 4, 64, 2>(a, s);
  }
  return hipErrorInvalidValue;
}

// Sums the parts of the experts' split contractions in order: a block takes 2048
// elements of expert blockIdx.y's matrix, a thread eight of a row.  An expert's first part
// is found as the tiles find theirs.
template <class T>
__global__ __launch_bounds__(256) void k_experts_join(ExpertArgs a, const float* in, T* out, int64_t ldo, int64_t ostride,
                                                     bool whole) {
  const int e = blockIdx.y, lane = threadIdx.x & 63;
  int first = 0;
  for (int e0 = 0; e0 < e; e0 += kBatch)
    first += __shfl(sum_below(e0 + lane < e ? pieces_of(a, e0 + lane, a.chunk) : 0, lane), 63, 64);
  int last = first + pieces_of(a, e, a.chunk);
  last = last < a.parts ? last : a.parts;
  if (a.accumulate && first >= last) return;
  const int wide = (a.cols + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int r = static_cast<int>(i / wide), c = static_cast<int>(i - static_cast<int64_t>(r) * wide) * 8;
  if (r >= a.rows) return;
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = 0.f;
  const float* from = in + r * a.ldo + c;
#pragma unroll 4
  for (int p = first; p < last; ++p) {
    float w[8];
    load8(from + p * a.ostride, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += w[q];
  }
  T* o = out + e * ostride + r * ldo + c;
  if (whole && c + 8 <= a.cols) {
    if (a.accumulate) {
      float w[8];
      load8(o, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += w[q];
    }
    store8(o, v);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < a.cols) store1(o + q, a.accumulate ? load1(o + q) + v[q] : v[q]);
  }
}

}  // namespace

hipError_t launch_experts_join(const ExpertArgs& a, void* out, int64_t ldo, int64_t ostride, int odt, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((int64_t(a.rows) * ((a.cols + 7) / 8) + 255) / 256);
  const float* in = static_cast<const float*>(a.out);
  const int64_t size = odt == kBF16 ? 2 : 4;
  const bool whole = ((reinterpret_cast<uintptr_t>(out) | ldo * size | ostride * size) & 15) == 0;
  if (odt == kBF16)
    hipLaunchKernelGGL((k_experts_join<uint16_t>), dim3(blocks, a.experts), dim3(256), 0, s, a, in,
                       static_cast<uint16_t*>(out), ldo, ostride, whole);
  else
    hipLaunchKernelGGL((k_experts_join<float>), dim3(blocks, a.experts), dim3(256), 0, s, a, in,
                       static_cast<float*>(out), ldo, ostride, whole);
  return hipGetLastError();
}

hipError_t launch_experts(const ExpertArgs& a, int op, int dt, int odt, bool aligned, int tile, hipStream_t s) {
  auto with = [&](auto z) {
    using T = decltype(z);
    if (op == kExpertFwd) return launch_op<kExpertFwd, T>(a, dt, aligned, tile, s);
    if (op == kExpertDx) return launch_op<kExpertDx, T>(a, dt, aligned, tile, s);
    return launch_op<kExpertDw, T>(a, dt, aligned, tile, s);
  };
  if (op == kExpertPart) return launch_op<kExpertPart, float>(a, dt, aligned, tile, s);
  return odt == kBF16 ? with(uint16_t{}) : with(float{});
}

}  // namespace muon
