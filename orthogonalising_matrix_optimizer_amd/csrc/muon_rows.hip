// Rows moved by index: the embedding table's lookup and gradient, and the sum
// of experts' rows back to tokens with its gradients.  All of it is bound by
// memory; sums are in fp32.
#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx_device.h"
#include "muon_sparse.h"

namespace muon {
namespace {

constexpr int kRowThreads = 256;

// Eight columns from c of a row, those past `cols` as zeros, and back.
template <class T>
__device__ __forceinline__ void load_cols(const T* row, int c, int cols, float* v) {
  if (c + 8 <= cols) {
    load8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? load1(row + c + e) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store_cols(T* row, int c, int cols, const float* v) {
  if (c + 8 <= cols) {
    store8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < cols) store1(row + c + e, v[e]);
  }
}

__device__ __forceinline__ int64_t id_at(const void* ids, int bytes, int i) {
  return bytes == 8 ? glb(static_cast<const int64_t*>(ids))[i]
                    : static_cast<int64_t>(glb(static_cast<const int32_t*>(ids))[i]);
}

// ---- embedding: a thread takes eight columns of kEmbedEach tokens, so that as many
// rows are on their way.  Bound by memory: 65537 tokens x 2560 in bf16, 672 MB, 124 us.
constexpr int kEmbedEach = 4;
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_embedding(EmbedArgs a) {
  const int wide = (a.cols + 7) / 8;
  const int64_t items = static_cast<int64_t>(a.tokens) * wide;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRowThreads * kEmbedEach + threadIdx.x;
  float v[kEmbedEach][8];
#pragma unroll
  for (int u = 0; u < kEmbedEach; ++u) {
    const int64_t i = first + u * kRowThreads;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
    if (i >= items) continue;
    const int t = static_cast<int>(i / wide), c = static_cast<int>(i - static_cast<int64_t>(t) * wide) * 8;
    const int64_t id = id_at(a.ids, a.id_bytes, t);
    if (id >= 0 && id < a.rows) load_cols(static_cast<const T*>(a.w) + id * a.ldw, c, a.cols, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kEmbedEach; ++u) {
    const int64_t i = first + u * kRowThreads;
    if (i >= items) continue;
    const int t = static_cast<int>(i / wide), c = static_cast<int>(i - static_cast<int64_t>(t) * wide) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] *= a.scale;
    store_cols(static_cast<T*>(a.out) + t * a.ldo, c, a.cols, v[u]);
  }
}

// ---- the table's gradient
//
// Tokens are sorted by id.  A wave takes `chunk` sorted positions and 512
// columns, eight a lane, and adds the rows of each run of equal ids in order.  A
// run inside the chunk is written at once.  One that came in from the chunk
// before goes to the chunk's first partial row, one that only leaves it to its
// second; k_embedding_join adds a run's partial rows.  Waves behind those look
// over 64 rows of the table each and zero the ones without tokens.  Fixed chunks,
// not a wave for each row of the table: half of a text's tokens may share a few ids
// (65536 of them: 43 us, 120 by owners).  65537 x 2560 bf16 into 50257 fp32 rows, 851 MB:
// 245 us and 15 for the join, mostly stores; 16384 x 768 into 50257: 37 and 5.
constexpr int kGradBatch = 8;   // rows in flight

template <class T, class D>
__device__ __forceinline__ void embed_sum(const EmbedGradArgs& a, int chunk, int strip, int lane) {
  const int c = strip * 512 + lane * 8;
  const int p0 = chunk * a.chunk, p1 = p0 + a.chunk < a.tokens ? p0 + a.chunk : a.tokens;
  const bool mine = c < a.cols;
  // keys of this chunk and its neighbours: lane l holds position p0 + l
  const int at = p0 + lane < p1 ? p0 + lane : p1 - 1;
  const int keys = a.key[at], from = a.pos[at];
  const int prev = p0 > 0 ? a.key[p0 - 1] : -1, next = p1 < a.tokens ? a.key[p1] : -1;
  const int n = p1 - p0;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool came = __builtin_amdgcn_readlane(keys, 0) == prev;
  for (int i0 = 0; i0 < n; i0 += kGradBatch) {
    float v[kGradBatch][8];
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u) {
      const int i = i0 + u < n ? i0 + u : n - 1;
      const int64_t t = __builtin_amdgcn_readlane(from, i);   // (of padding there is no token)
      if (mine && i0 + u < n && __builtin_amdgcn_readlane(keys, i) < a.rows) load_cols(static_cast<const T*>(a.dy) + t * a.ldy, c, a.cols, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      const int k = __builtin_amdgcn_readlane(keys, i);
      if (k >= a.rows) return;   // padding is last
      if (mine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
      }
      const int then = i + 1 < n ? __builtin_amdgcn_readlane(keys, i + 1) : next;
      if (then == k && i + 1 < n) continue;
      if (mine) {
        if (came || then == k) {
          store8(a.part + (static_cast<int64_t>(chunk) * 2 + (came ? 0 : 1)) * a.ldp + c, acc);
        } else {
          D* o = static_cast<D*>(a.dw) + k * a.ldw;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = 0.f;
          if (a.accumulate) load_cols(o, c, a.cols, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] += a.scale * acc[e];
          store_cols(o, c, a.cols, w);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
      came = false;
    }
  }
}

template <class D>
__device__ __forceinline__ void embed_zero(const EmbedGradArgs& a, int block, int lane, volatile uint8_t* list) {
  const int v = block * kEmbedZeroRows + lane;
  int lo = 0, hi = a.tokens;
  while (lo < hi) {   // the first position whose key is at least v
    const int mid = (lo + hi) >> 1;
    if (a.key[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  const bool absent = v < a.rows && !(lo < a.tokens && a.key[lo] == v);
  // the pieces of all rows without tokens, one after the other
  const uint64_t mask = __ballot(absent);
  if (absent) list[below(mask)] = static_cast<uint8_t>(lane);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int wide = (a.cols + 7) / 8, items = __popcll(mask) * wide;
  const float zeros[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i = lane; i < items; i += 64) {
    const int n = i / wide;
    D* o = static_cast<D*>(a.dw) + (static_cast<int64_t>(block) * kEmbedZeroRows + list[n]) * a.ldw;
    store_cols(o, (i - n * wide) * 8, a.cols, zeros);
  }
}

template <class T, class D>
__global__ __launch_bounds__(kRowThreads) void k_embedding_grad(EmbedGradArgs a, int strips) {
  const int unit = blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, sums = a.chunks * strips;
  __shared__ uint8_t list[kRowThreads / 64][64];
  if (unit < sums) {
    embed_sum<T, D>(a, unit / strips, unit % strips, lane);
  } else if (!a.accumulate) {
    const int z = unit - sums;
    if (z < (a.rows + kEmbedZeroRows - 1) / kEmbedZeroRows) embed_zero<D>(a, z, lane, list[threadIdx.x >> 6]);
  }
}

// Joins the run that leaves chunk blockIdx.x without having come into it: the
// chunk's second partial row and the first ones of the chunks that it reaches, a
// quarter of them by each wave, 256 columns a block.
template <class D>
__global__ __launch_bounds__(kRowThreads) void k_embedding_join(EmbedGradArgs a) {
  constexpr int WAVES = kRowThreads / 64;
  __shared__ float4 sums[WAVES][64];
  const int chunk = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p0 = chunk * a.chunk, p1 = p0 + a.chunk;
  if (p1 >= a.tokens) return;
  const int k = a.key[p1 - 1];
  if (k >= a.rows || a.key[p1] != k) return;
  if (p0 > 0 && a.key[p0] == k && a.key[p0 - 1] == k) return;   // it came in
  int last = chunk + 1;                                         // chunks chunk + 1 .. last hold the rest
  for (;; last += 64) {
    const int c = last + 1 + lane;
    const bool on = c < a.chunks && a.key[c * a.chunk] == k;
    const uint64_t off = ~__ballot(on);
    if (off) {
      last += __builtin_ctzll(off);
      break;
    }
  }
  const int c = blockIdx.y * 256 + lane * 4, n = last - chunk;
  const int share = (n + WAVES - 1) / WAVES;
  const int i0 = wave * share < n ? wave * share : n, i1 = i0 + share < n ? i0 + share : n;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  auto row = [&](int64_t r) {
    return c < a.cols ? *reinterpret_cast<const float4*>(a.part + r * a.ldp + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto add = [&](float4 q) { v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w; };
  if (wave == 0) add(row(static_cast<int64_t>(chunk) * 2 + 1));
  for (int i = i0; i < i1; i += kGradBatch) {
    float4 q[kGradBatch];
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u) q[u] = row(static_cast<int64_t>(chunk + 1 + (i + u < i1 ? i + u : i1 - 1)) * 2);
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u)
      if (i + u < i1) add(q[u]);
  }
  sums[wave][lane] = make_float4(v[0], v[1], v[2], v[3]);
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    const float4 q = sums[w][lane];
    v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
  }
  D* o = static_cast<D*>(a.dw) + k * a.ldw;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < a.cols) store1(o + c + e, (a.accumulate ? load1(o + c + e) : 0.f) + a.scale * v[e]);
}

// Up to kFewTokens tokens, in one launch and without a sort: a wave takes a row of
// the table, finds the tokens that have it by ballots over all ids and adds their
// rows in order.  (37 tokens, 333 rows of 77: 3.2 us where sort, sums and join take 15.)
template <class T, class D>
__global__ __launch_bounds__(kRowThreads) void k_embedding_few(EmbedGradArgs a, const void* ids, int id_bytes) {
  constexpr int MASKS = kFewTokens / 64;
  const int v = blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (v >= a.rows) return;
  uint64_t mask[MASKS];
  bool any = false;
#pragma unroll
  for (int m = 0; m < MASKS; ++m) {
    const int t = m * 64 + lane;
    mask[m] = m * 64 < a.tokens ? __ballot(t < a.tokens && id_at(ids, id_bytes, t < a.tokens ? t : 0) == v) : 0;
    any = any || mask[m];
  }
  if (!any && a.accumulate) return;
  D* o = static_cast<D*>(a.dw) + v * a.ldw;
  for (int c = lane * 8; c < a.cols; c += 512) {
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
    for (int m = 0; m < MASKS; ++m) {
      uint64_t left = mask[m];
      while (left) {
        float x[kGradBatch][8];
        int n = 0;
#pragma unroll
        for (int u = 0; u < kGradBatch; ++u)
          if (left) {
            const int64_t t = m * 64 + __builtin_ctzll(left);
            left &= left - 1;
            ++n;
            load_cols(static_cast<const T*>(a.dy) + t * a.ldy, c, a.cols, x[u]);
          }
#pragma unroll
        for (int u = 0; u < kGradBatch; ++u)
          if (u < n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[u][e];
          }
      }
    }
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.f;
    if (a.accumulate) load_cols(o, c, a.cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] += a.scale * acc[e];
    store_cols(o, c, a.cols, w);
  }
}

// ---- combine: a thread takes eight columns of a token, the rows of up to
// kSlotBatch slots in flight.  Bound by the rows of y, read once here and there: 16384
// tokens x 6 x 2048 in bf16, 470 MB, 112 us.
constexpr int kSlotBatch = 8;
template <class T, class D>
__global__ __launch_bounds__(kRowThreads) void k_combine(CombineArgs a) {
  const int wide = (a.cols + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int t = static_cast<int>(i / wide), c = static_cast<int>(i - static_cast<int64_t>(t) * wide) * 8;
  if (t >= a.tokens) return;
  const int64_t slot = static_cast<int64_t>(t) * a.k;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += kSlotBatch) {
    int row[kSlotBatch];
    float g[kSlotBatch], v[kSlotBatch][8];
#pragma unroll
    for (int u = 0; u < kSlotBatch; ++u) {
      const bool in = j0 + u < a.k;
      const int r = in ? a.place[slot + j0 + u] : -1;
      row[u] = r < a.slots ? r : -1;
      g[u] = a.gates && in ? a.gates[slot + j0 + u] : 1.f;
    }
#pragma unroll
    for (int u = 0; u < kSlotBatch; ++u)
      if (row[u] >= 0) load_cols(static_cast<const T*>(a.y) + row[u] * a.ldy, c, a.cols, v[u]);
#pragma unroll
    for (int u = 0; u < kSlotBatch; ++u)
      if (row[u] >= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += g[u] * v[u][e];
      }
  }
  store_cols(static_cast<D*>(a.out) + t * a.ldo, c, a.cols, acc);
}

__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// A wave takes a row of y and dy, in order: these are the bytes that count, and the
// tokens' rows of dout, read once for each slot, come from the last cache (827 MB pass
// L2, 470 of which are y and dout once).  (A wave for
// each token, which reads dout once and k rows of y here and there: 16384 tokens x 6
// x 2048 in bf16 309 us, 203 in this order.)  The row's slot is that of its
// token's which lies there; rows that are only gathered need none.
constexpr int kChunkBatch = 4;   // pieces of 512 columns in flight
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_combine_grad(CombineArgs a) {
  const int r = blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= a.slots) return;
  const int t = a.rows[r];
  if (a.dgates) {
    // slot r gets its number from the wave of its row, if that is one of its token's, else 0
    const int at = a.place[r], of = at >= 0 && at < a.slots ? a.rows[at] : -1;
    const int64_t own = static_cast<int64_t>(of) * a.k;
    if (lane == 0 && !(of >= 0 && of < a.tokens && r >= own && r < own + a.k)) a.dgates[r] = 0.f;
  }
  if (t < 0 || t >= a.tokens) return;
  const int64_t first = static_cast<int64_t>(t) * a.k;
  uint64_t here = 0;   // the token's slots that lie here: one, in a plan of expert_plan's
  float g = 1.f;
  if (a.gates || a.dgates) {
    here = __ballot(lane < a.k && a.place[first + (lane < a.k ? lane : 0)] == r);
    if (!here) return;
    if (a.gates) {
      g = a.gates[first + __builtin_ctzll(here)];
      for (uint64_t more = here & (here - 1); more; more &= more - 1) g += a.gates[first + __builtin_ctzll(more)];
    }
  }
  const T* d = static_cast<const T*>(a.dout) + t * a.ldd;
  const T* y = static_cast<const T*>(a.y) + r * a.ldy;
  T* out = static_cast<T*>(a.out) + r * a.ldo;
  float dot = 0.f;
  for (int c0 = lane * 8; c0 < a.cols; c0 += 512 * kChunkBatch) {
    float x[kChunkBatch][8], v[kChunkBatch][8];
#pragma unroll
    for (int u = 0; u < kChunkBatch; ++u) {
      const int c = c0 + 512 * u;
      if (c >= a.cols) break;
      load_cols(d, c, a.cols, x[u]);
      if (a.dgates) load_cols(y, c, a.cols, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kChunkBatch; ++u) {
      const int c = c0 + 512 * u;
      if (c >= a.cols) break;
      if (a.dgates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += x[u][e] * v[u][e];
      }
      if (a.out) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] *= g;
        store_cols(out, c, a.cols, x[u]);
      }
    }
  }
  if (a.dgates) {
    dot = lanes_sum(dot);
    if (here >> lane & 1) a.dgates[first + lane] = dot;
  }
}

unsigned blocks_of(int64_t items, int64_t per) { return static_cast<unsigned>((items + per - 1) / per); }

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a, int dt, hipStream_t s) {
  const unsigned blocks = blocks_of(int64_t(a.tokens) * ((a.cols + 7) / 8), kRowThreads * kEmbedEach);
  return with_type(dt, [&](auto z) {
    hipLaunchKernelGGL((k_embedding<decltype(z)>), dim3(blocks), dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, int dt, int odt, hipStream_t s) {
  const int strips = (a.cols + 511) / 512;
  const int64_t units = int64_t(a.chunks) * strips + (a.accumulate ? 0 : blocks_of(a.rows, kEmbedZeroRows));
  return with_type(odt, [&](auto o) {
    using D = decltype(o);
    if (units) {
      const hipError_t e = with_type(dt, [&](auto z) {
        hipLaunchKernelGGL((k_embedding_grad<decltype(z), D>), dim3(blocks_of(units, kRowThreads / 64)),
                           dim3(kRowThreads), 0, s, a, strips);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
    }
    if (a.chunks > 1)
      hipLaunchKernelGGL((k_embedding_join<D>), dim3(a.chunks - 1, blocks_of(a.cols, 256)), dim3(kRowThreads),
                         0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_embedding_few(const EmbedGradArgs& a, const void* ids, int id_bytes, int dt, int odt, hipStream_t s) {
  return with_type(dt, [&](auto z) {
    return with_type(odt, [&](auto o) {
      hipLaunchKernelGGL((k_embedding_few<decltype(z), decltype(o)>), dim3(blocks_of(a.rows, kRowThreads / 64)),
                         dim3(kRowThreads), 0, s, a, ids, id_bytes);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine(const CombineArgs& a, int dt, int odt, hipStream_t s) {
  const unsigned blocks = blocks_of(int64_t(a.tokens) * ((a.cols + 7) / 8), kRowThreads);
  return with_type(dt, [&](auto z) {
    return with_type(odt, [&](auto o) {
      hipLaunchKernelGGL((k_combine<decltype(z), decltype(o)>), dim3(blocks), dim3(kRowThreads), 0, s, a);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine_grad(const CombineArgs& a, int dt, hipStream_t s) {
  return with_type(dt, [&](auto z) {
    hipLaunchKernelGGL((k_combine_grad<decltype(z)>), dim3(blocks_of(a.slots, kRowThreads / 64)),
                       dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace muon
