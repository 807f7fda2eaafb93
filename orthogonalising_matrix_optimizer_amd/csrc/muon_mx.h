// Shared host/device definitions of the 4-bit (MXFP4) operators and dropout.
//
// Storage of a rows x cols matrix (blocks of 32 along the columns, the
// contraction index of every product):
//   codes : tiles of 16 rows x 128 columns, 1 KiB each, tile (r / 16, k / 128)
//           at ((k / 128) * R + r / 16) * 1024 for R = ceil(rows / 16): the
//           tiles of a row panel and one step along the contraction are
//           contiguous, so the panels that many blocks read at once spread
//           over all L2 channels.  Inside a tile the 16 bytes of the block
//           (r % 16, (k % 128) / 32) are at 16 * (16 * ((k % 128) / 32) + r % 16):
//           16 consecutive bytes per lane in the order in which a wave feeds
//           v_mfma_scale_f32_16x16x128_f8f6f4, so a tile is one contiguous
//           load and one conflict-free LDS read.
//   scales: one byte per block; a dword holds the four row tiles of 64 rows:
//           byte ((k / 128) * ceil(rows / 64) + r / 64) * 256 + 4 * (16 *
//           ((k % 128) / 32) + r % 16) + (r % 64) / 16, so one dword per lane
//           serves four MFMA operands, which pick their byte by an immediate.
// Blocks past the last column have zero codes and an ordinary scale; rows past
// the last row of a tile are never stored from any product, and may hold anything.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int kMxTileR = 16;       // rows of a code tile
constexpr int kMxTileK = 128;      // columns of a code tile
constexpr int kMxTileBytes = 1024;
constexpr int kMxScaleRows = 64;   // rows of a scale tile (256 bytes)
constexpr int kMxScaleBytes = 256;
constexpr uint32_t kMxNan = 255;   // scale byte of a block that is NaN

// third counter word of the generator: what the numbers are for
constexpr uint32_t kTagDropout = 0x44524F50u, kTagRound = 0x53523430u, kTagRoundT = 0x53523431u;

// Descriptors travel as kernel arguments (under the 4 KiB limit), so the calls
// need no device table, no workspace for one and no staging memory.  A call on
// one matrix passes a list of one: kernel arguments are read from host memory,
// and small ones keep the shortest launches short.
constexpr int kMxMaxList = 36;

// A seed given by value, or by the device address of one (then read by the
// kernel: a replayed graph can be given new numbers).
struct MxSeed {
  uint64_t value;
  const uint64_t* dev;   // or null
};

struct MxDrop {
  uint32_t threshold;    // in steps of 2^-16; 0: no dropout
  float scale;
  MxSeed seed;
};

// Arguments of a grouped launch: what all matrices share, the matrices, and
// the first block (work item) of each.
template <class Common, class Mat, int CAP>
struct MxList {
  static constexpr int kCap = CAP;
  Common c;
  int32_t n;
  int32_t _pad;
  Mat m[CAP];
  uint32_t base[CAP];
};

template <class Common, class Mat, int CAP>
MxList<Common, Mat, 1> list_of_one(const MxList<Common, Mat, CAP>& a) {
  MxList<Common, Mat, 1> o;
  o.c = a.c;
  o.n = 1;
  o._pad = 0;
  o.m[0] = a.m[0];
  o.base[0] = a.base[0];
  return o;
}

struct MxQuantMat {
  const void* in;        // rows x cols, row pitch ld elements
  uint8_t* codes;        // the matrix in 4 bits, or null
  uint8_t* scales;
  uint8_t* codes_t;      // its transpose in 4 bits, or null
  uint8_t* scales_t;
  int64_t ld;
  int32_t rows, cols;
  int32_t index;         // place in the caller's list (fourth counter word)
  int32_t _pad;
};
struct MxQuantCommon {
  MxSeed seed;           // stochastic rounding
  MxDrop drop;
};
template <int CAP> using MxQuantList = MxList<MxQuantCommon, MxQuantMat, CAP>;
using MxQuantArgs = MxQuantList<kMxMaxList>;

struct MxDequantMat {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  int64_t ld;
  int32_t rows, cols;
};
struct MxDequantCommon {};
template <int CAP> using MxDequantList = MxList<MxDequantCommon, MxDequantMat, CAP>;
using MxDequantArgs = MxDequantList<kMxMaxList>;

// out (M x N) = a (M x K) * b (N x K)^T, or with a split contraction the
// partial products over `chunk` code tiles each, `stride` elements apart
struct MxProduct {
  const uint8_t* ac;
  const uint8_t* as;
  const uint8_t* bc;
  const uint8_t* bs;
  void* out;
  int64_t ld;
  int64_t stride;
  int32_t M, N;
  int32_t kt;              // code tiles along the contraction
  int32_t chunk;           // ... of one work item
  int32_t tiles;           // output tiles; item = split * tiles + tile
  int32_t index;           // place in the caller's list
};
struct MxGemmCommon {
  MxDrop drop;
  int32_t xcd[9];          // items [xcd[x], xcd[x + 1]) are XCD x's: as many stages each
  int32_t accumulate;      // out += product
};
template <int CAP> using MxGemmList = MxList<MxGemmCommon, MxProduct, CAP>;
using MxGemmArgs = MxGemmList<kMxMaxList>;

// out (M x N) = sum over the splits of the partial products (fp32, row pitch
// ldp, `stride` elements apart)
struct MxReduce {
  const float* in;
  void* out;
  int64_t ld;
  int64_t stride;
  int32_t M, N, ldp;
  int32_t splits;
  int32_t index;
  int32_t _pad;
};
struct MxReduceCommon {
  MxDrop drop;
  int32_t accumulate;
  int32_t _pad;
};
template <int CAP> using MxReduceList = MxList<MxReduceCommon, MxReduce, CAP>;
using MxReduceArgs = MxReduceList<kMxMaxList>;

static_assert(sizeof(MxQuantArgs) <= 4096 && sizeof(MxGemmArgs) <= 4096 && sizeof(MxReduceArgs) <= 4096 &&
              sizeof(MxDequantArgs) <= 4096, "kernel argument limit");

struct MxDropArgs {
  const void* in;
  void* out;
  int64_t ldi, ldo;
  int32_t rows, cols;
  MxDrop drop;
};

// out (M x N) = x (M x K, not in 4 bits) * b (N x K)^T, M <= 16
struct MxRowsArgs {
  const void* x;
  const uint8_t* bc;
  const uint8_t* bs;
  void* out;
  int64_t ldx, ldo;
  int32_t M, N, K;
  int32_t _pad;
};

hipError_t launch_mx_quantize(const MxQuantArgs& a, int dt, bool rows, bool cols, bool stochastic,
                              int64_t blocks, hipStream_t s);
hipError_t launch_mx_dequantize(const MxDequantArgs& a, int dt, int64_t blocks, hipStream_t s);
// tile_m: rows of the output tiles (256 or 128; always 128 columns)
// keep: the outputs go into the caches, not past them
hipError_t launch_mx_gemm(const MxGemmArgs& a, int odt, int tile_m, bool keep, hipStream_t s);
hipError_t launch_mx_reduce(const MxReduceArgs& a, int odt, int64_t blocks, hipStream_t s);
hipError_t launch_mx_rows(const MxRowsArgs& a, int xdt, int odt, hipStream_t s);
hipError_t launch_dropout(const MxDropArgs& a, int dt, int64_t blocks, hipStream_t s);

// Work of one block of each kernel (the host sizes the grids with these).
constexpr int kMxQuantTile = 128;              // quantise, dequantise: square tile edge
constexpr int kDropItems = 256;                // dropout: groups of 8 elements per block

}  // namespace muon
