// Kernel arguments and launchers of the embedding table and the expert layers
// (see include/muon.h for the operators).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon_common.h"

namespace muon {

// Calls f with an element of a type.
template <class F>
hipError_t with_type(int dt, F&& f) {
  return dt == kBF16 ? f(uint16_t{}) : f(float{});
}

// ---- stable counting sort (muon_route.hip)
//
// Sorts positions 0 .. n-1 by an integer key, by position among equal keys, in
// passes of kSortBits (or kSortWide) bits, the lowest first.
constexpr int kSortThreads = 1024;
constexpr int kSortBits = 8, kSortWide = 10;
// blocks up to which each counts all keys itself (one launch a pass)
constexpr int kSortSelf = 4;

// Bits of the keys 0 .. limit, and how they are sorted.
inline int key_bits(int64_t limit) {
  int b = 1;
  while (limit >> b) ++b;
  return b;
}
inline int sort_bits(int bits) {
  return bits <= kSortBits || (bits > kSortWide && bits <= 2 * kSortBits) ? kSortBits : kSortWide;
}
// Positions a thread takes: more where the blocks' counts, which every block of a pass reads,
// would be many.  us with 1 | 4, of 64 experts' slots (8 bits): 131072 11 | 15, 262144 14 | 16,
// 524288 25 | 18, 1048576 63 | 22; of 512 experts' (10 bits): 98304 21 | 19, 131072 25 | 19, 262144
// 39 | 22, 1048576 260 | 38; a table's gradient of 50257 ids (two passes of 8): 262144 72 | 81,
// 524288 123 | 114, 1048576 255 | 179.
inline int sort_each(int64_t n, int64_t limit) {
  return n <= (int64_t(1) << (sort_bits(key_bits(limit)) == kSortBits ? 18 : 17)) ? 1 : 4;
}

struct SortArgs {
  const void* ids;      // n integers of id_bytes (of the first pass)
  int32_t id_bytes;
  int32_t n;
  int32_t limit;        // keys are 0 .. limit: ids outside 0 .. limit-1 have key `limit`
  int32_t passes;
  int32_t* key[2];      // keys and positions between passes; the last pass writes
  int32_t* pos[2];      // into key[passes & 1 ^ 1] and pos[...] where they are not null
  int32_t* counts;      // blocks x bins, for more than kSortSelf blocks
  // where the sorted positions are a plan's slots (one pass): its arrays, or null
  int32_t* offsets;
  int32_t* tokens;
  int32_t* place;
  int32_t k;
};
hipError_t launch_sort(const SortArgs& a, hipStream_t s);

// ---- routing (muon_route.hip)
struct RouteArgs {
  const void* logits;
  int64_t ld;
  float* gates;
  int32_t* chosen;
  int32_t tokens, experts, k, normalize;
};
// sort: of the slots of a.chosen
hipError_t launch_route(const RouteArgs& a, const SortArgs& sort, int dt, hipStream_t s);

struct RouteGradArgs {
  const float* dgates;
  const void* logits;
  const float* gates;
  const int32_t* chosen;
  void* dlogits;
  int64_t ld, ldd;
  int32_t tokens, experts, k, normalize;
};
hipError_t launch_route_grad(const RouteGradArgs& a, int dt, int ddt, hipStream_t s);

// ---- rows moved by index (muon_rows.hip)
struct CombineArgs {
  const void* y;          // slots' rows
  const void* dout;       // tokens' rows (gradient)
  const float* gates;     // or null: ones
  const int32_t* place;
  const int32_t* rows;    // gradient: the rows' tokens
  void* out;              // forward: tokens' rows; gradient: slots' rows, or null
  float* dgates;          // or null
  int64_t ldy, ldd, ldo;
  int32_t tokens, k, slots, cols;
};
hipError_t launch_combine(const CombineArgs& a, int dt, int odt, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs& a, int dt, hipStream_t s);

struct EmbedArgs {
  const void* ids;
  const void* w;
  void* out;
  int64_t ldw, ldo, rows;   // rows of w
  float scale;
  int32_t id_bytes, tokens, cols;
};
hipError_t launch_embedding(const EmbedArgs& a, int dt, hipStream_t s);

// Sums of dy's rows over runs of equal sorted keys.  A wave takes `chunk` consecutive
// sorted positions; a run inside them is written at once, one that crosses their edges
// goes to `part` (two rows a chunk) and is joined by a second launch.
constexpr int kEmbedZeroRows = 64;   // rows of dw that a wave looks over for zeroing, one a lane
struct EmbedGradArgs {
  const void* dy;
  const int32_t* key;     // sorted ids (the last ones `rows`: no gradient)
  const int32_t* pos;     // their tokens
  void* dw;
  float* part;            // chunks x 2 rows
  int64_t ldy, ldw;
  float scale;
  int32_t tokens, rows, cols, accumulate;
  int32_t chunk, chunks;  // sorted positions a wave sums, and how many such chunks
  int32_t ldp;            // floats from one row of part to the next, a multiple of 8
};
// Without a sort, for few tokens (key, pos, part and the chunks are not used).  us without |
// with a sort, of 256 tokens: 333 rows of 77 10 | 16, 4096 of 1024 11 | 38, 50257 of 768 30 | 40,
// 50257 of 2560 121 | 109; of 512 (with masks for 1024): 18 | 16, 24 | 39, 77 | 40, 197 | 114.
constexpr int kFewTokens = 256;
hipError_t launch_embedding_few(const EmbedGradArgs& a, const void* ids, int id_bytes, int dt, int odt, hipStream_t s);
hipError_t launch_embedding_grad(const EmbedGradArgs& a, int dt, int odt, hipStream_t s);

// ---- experts' products (muon_experts.hip)
// kExpertPart: dw with split contractions, which takes tiles of 64 alone.
enum ExpertOp : int32_t { kExpertFwd = 0, kExpertDx = 1, kExpertDw = 2, kExpertPart = 3 };
struct ExpertArgs {
  const void* r;            // operand of the output's rows: x, dy, dy
  const void* c;            // operand of the output's columns: w, w, x
  void* out;
  const int32_t* offsets;
  const int32_t* tokens;    // gathered x: the rows' tokens, else null
  int64_t ldr, ldc, ldo;    // elements
  int64_t wstride, ostride; // elements between experts' matrices: of c, of out (dw)
  int32_t experts, slots;
  int32_t rows, cols;       // dw: rows of a matrix; columns of the output
  int32_t depth;            // contraction length (fwd, dx)
  int32_t src;              // rows of x when gathered
  int32_t accumulate;       // dw
  int32_t past;             // write past the caches
  int32_t chunk, parts;     // split dw: rows of a part, parts that out has room for
};
// Blocks of a launch with tm x tn tiles.  How the slots are split is known to the
// device alone: a full tile for every tm slots and a part of one an expert at most.
inline int64_t expert_blocks(const ExpertArgs& a, int op, int tm, int tn) {
  const int64_t across = (int64_t(a.cols) + tn - 1) / tn;
  if (op >= kExpertDw) {
    const int64_t tiles = (int64_t(a.rows) + tm - 1) / tm * across;
    if (op == kExpertPart) return 8 * ((tiles * a.parts + 7) / 8);
    return 8 * a.experts * ((tiles + 7) / 8);
  }
  const int64_t tiles = a.slots / tm + (a.experts < a.slots ? a.experts : a.slots);
  return 8 * ((tiles * across + 7) / 8);
}
// Bytes that a buffer's descriptor spans at most: an offset from here on reads as
// zeros and, with the offset along a row added, stays below 2^32.
constexpr uint32_t kExpertSpan = 0xf0000000u;
// Largest row pitch (elements): a tile's 256 rows of bf16, 128 of fp32, are in a span.
constexpr int64_t kExpertPitch = int64_t(1) << 22;
// aligned: every row of the operands starts at 16 bytes (and holds whole ones along
// the contraction), so that loads go straight to LDS
// tile: 64, 128 or, aligned, 256
hipError_t launch_experts(const ExpertArgs& a, int op, int dt, int odt, bool aligned, int tile, hipStream_t s);

// Sums the parts that a launch of kExpertPart wrote to a.out (fp32) into the experts'
// matrices.
hipError_t launch_experts_join(const ExpertArgs& a, void* out, int64_t ldo, int64_t ostride, int odt, hipStream_t s);

}  // namespace muon
