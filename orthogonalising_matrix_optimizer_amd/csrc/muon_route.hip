// Routing of tokens to experts, its gradient, and the stable counting sort that
// orders slots by expert and tokens by id.
//
// Sort.  A block takes 1024 (or 4096) consecutive positions.  Within a wave the
// lanes with the same digit are found by ballots over the digit's bits, so a
// position's rank among equals is a population count and one lane adds the wave's
// count: no atomics on hot bins (half of a text's tokens share a high digit), and
// the order depends on nothing but the keys.  A position goes to
//   (positions with smaller digits) + (equal digits in earlier blocks)
//   + (in earlier waves of the block) + (earlier in the wave).
// Up to kSortSelf blocks, each counts the digits of all keys itself, which costs
// less than a launch of its own for it; beyond, a launch writes the blocks' counts
// (us a pass with 16 blocks: 18.6 | 9.8).
#include <type_traits>

#include "muon_common.h"
#include "muon_device.h"
#include "muon_mx_device.h"
#include "muon_sparse.h"

namespace muon {
namespace {

constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int32_t first_key(const SortArgs& a, int i) {
  const int64_t id = a.id_bytes == 8 ? glb(static_cast<const int64_t*>(a.ids))[i]
                                     : glb(static_cast<const int32_t*>(a.ids))[i];
  return id >= 0 && id < a.limit ? static_cast<int32_t>(id) : a.limit;
}

// Lanes of the wave with the same digit, of those for which `in` holds.
template <int BITS>
__device__ __forceinline__ uint64_t peers_of(int digit, bool in) {
  uint64_t same = __ballot(in);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = digit >> b & 1;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  return same;
}

template <int BITS>
struct SortShared {
  uint16_t count[kSortWaves][1 << BITS];   // a wave's, then the earlier waves'
  int32_t total[1 << BITS];                // all positions', then those with smaller digits
  int32_t before[1 << BITS];               // positions of earlier blocks
  int32_t sums[kSortWaves];
};

// Exclusive sums over sh.total in place.
template <int BITS>
__device__ __forceinline__ void scan_bins(SortShared<BITS>& sh, int t) {
  constexpr int BINS = 1 << BITS, PER = BINS > kSortThreads ? BINS / kSortThreads : 1;
  int32_t v[PER], own = 0;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    v[u] = t * PER + u < BINS ? sh.total[t * PER + u] : 0;
    own += v[u];
  }
  int32_t up = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(up, d, 64);
    if ((t & 63) >= d) up += o;
  }
  if ((t & 63) == 63) sh.sums[t >> 6] = up;
  __syncthreads();
  int32_t at = up - own;
  for (int w = 0; w < (t >> 6); ++w) at += sh.sums[w];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (t * PER + u < BINS) sh.total[t * PER + u] = at;
    at += v[u];
  }
  __syncthreads();
}

// One pass over the digit at `shift`; SELF: the blocks count for themselves.
template <int BITS, int EACH, bool SELF>
__device__ __forceinline__ void sort_pass(const SortArgs& a, int pass, SortShared<BITS>& sh) {
  constexpr int BINS = 1 << BITS, SPAN = kSortThreads * EACH;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int shift = pass * BITS, n = a.n, start = blockIdx.x * SPAN;
  const bool first = pass == 0, last = pass + 1 == a.passes;
  const int32_t* kin = first ? nullptr : a.key[(pass - 1) & 1];
  const int32_t* pin = first ? nullptr : a.pos[(pass - 1) & 1];
  auto key_at = [&](int i) { return first ? first_key(a, i) : kin[i]; };

  for (int i = t; i < kSortWaves * BINS; i += kSortThreads) (&sh.count[0][0])[i] = 0;
  for (int i = t; i < BINS; i += kSortThreads) sh.total[i] = sh.before[i] = 0;
  __syncthreads();

  int32_t key[EACH], rank[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int i = start + wave * 64 * EACH + e * 64 + lane;
    const bool in = i < n;
    key[e] = in ? key_at(i) : 0;
    const int d = key[e] >> shift & (BINS - 1);
    const uint64_t peers = peers_of<BITS>(d, in);
    const int mine = below(peers);
    volatile uint16_t* c = &sh.count[wave][d];
    const int had = in ? *c : 0;
    rank[e] = had + mine;
    if (in && mine == 0) *c = static_cast<uint16_t>(had + __popcll(peers));
  }
  if constexpr (SELF) {
    // all positions' digits; this block's and later ones only in the total
    const int blocks = gridDim.x;
    if (blocks > 1)
      for (int j = wave * 64; j < n; j += kSortThreads) {
        const int i = j + lane;
        const bool in = i < n;
        const int d = in ? key_at(i) >> shift & (BINS - 1) : 0;
        const uint64_t peers = peers_of<BITS>(d, in);
        if (in && below(peers) == 0) {
          const int32_t c = __popcll(peers);
          atomicAdd(&sh.total[d], c);
          if (j < start) atomicAdd(&sh.before[d], c);
        }
      }
  } else {
    // the blocks' counts, their sums split over the threads of a bin
    constexpr int STRANDS = BINS < kSortThreads ? kSortThreads / BINS : 1;
    const int me = blockIdx.x, blocks = gridDim.x;
    for (int bin = t % BINS; bin < BINS; bin += kSortThreads) {
      int32_t all = 0, early = 0;
#pragma unroll 8
      for (int b = t / BINS; b < blocks; b += STRANDS) {
        const int32_t c = a.counts[int64_t(b) * BINS + bin];
        all += c;
        early += b < me ? c : 0;
      }
      if (STRANDS == 1) {
        sh.total[bin] = all;
        sh.before[bin] = early;
      } else {
        atomicAdd(&sh.total[bin], all);
        atomicAdd(&sh.before[bin], early);
      }
    }
  }
  __syncthreads();
  for (int bin = t; bin < BINS; bin += kSortThreads) {
    int32_t run = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = sh.count[w][bin];
      sh.count[w][bin] = static_cast<uint16_t>(run);
      run += c;
    }
    if (SELF && gridDim.x == 1) sh.total[bin] = run;
  }
  __syncthreads();
  scan_bins<BITS>(sh, t);
  if (last && a.offsets && blockIdx.x == 0)
    for (int e = t; e <= a.limit; e += kSortThreads) a.offsets[e] = sh.total[e];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int i = start + wave * 64 * EACH + e * 64 + lane;
    if (i >= n) continue;
    const int d = key[e] >> shift & (BINS - 1);
    const int to = sh.total[d] + sh.before[d] + sh.count[wave][d] + rank[e];
    const int32_t from = first ? i : pin[i];
    if (a.key[pass & 1]) a.key[pass & 1][to] = key[e];
    if (a.pos[pass & 1]) a.pos[pass & 1][to] = from;
    if (last && a.tokens) {
      const bool used = key[e] < a.limit;
      a.tokens[to] = used ? from / a.k : -1;
      a.place[from] = used ? to : -1;
    }
  }
}

template <int BITS, int EACH, bool SELF>
__global__ __launch_bounds__(kSortThreads) void k_sort(SortArgs a, int pass) {
  __shared__ SortShared<BITS> sh;
  sort_pass<BITS, EACH, SELF>(a, pass, sh);
}

// All passes of what one block sorts.
template <int BITS>
__global__ __launch_bounds__(kSortThreads) void k_sort_one(SortArgs a) {
  __shared__ SortShared<BITS> sh;
  for (int pass = 0; pass < a.passes; ++pass) {
    if (pass) __syncthreads();
    sort_pass<BITS, 1, true>(a, pass, sh);
  }
}

// counts[block][digit] of a pass.
template <int BITS, int EACH>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs a, int pass) {
  constexpr int BINS = 1 << BITS, SPAN = kSortThreads * EACH;
  __shared__ int32_t total[BINS];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int32_t* kin = pass == 0 ? nullptr : a.key[(pass - 1) & 1];
  for (int i = t; i < BINS; i += kSortThreads) total[i] = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int i = blockIdx.x * SPAN + wave * 64 * EACH + e * 64 + lane;
    const bool in = i < a.n;
    const int32_t key = !in ? 0 : pass == 0 ? first_key(a, i) : kin[i];
    const int d = key >> (pass * BITS) & (BINS - 1);
    const uint64_t peers = peers_of<BITS>(d, in);
    if (in && below(peers) == 0) atomicAdd(&total[d], static_cast<int32_t>(__popcll(peers)));
  }
  __syncthreads();
  for (int i = t; i < BINS; i += kSortThreads) a.counts[int64_t(blockIdx.x) * BINS + i] = total[i];
}

template <int BITS, int EACH>
hipError_t launch_sort_of(const SortArgs& a, hipStream_t s) {
  const int blocks = (a.n + kSortThreads * EACH - 1) / (kSortThreads * EACH);
  if constexpr (EACH == 1) {   // more positions a thread are only for many blocks
    if (blocks <= 1) {
      hipLaunchKernelGGL((k_sort_one<BITS>), dim3(1), dim3(kSortThreads), 0, s, a);
      return hipGetLastError();
    }
    if (blocks <= kSortSelf) {
      for (int pass = 0; pass < a.passes; ++pass)
        hipLaunchKernelGGL((k_sort<BITS, EACH, true>), dim3(blocks), dim3(kSortThreads), 0, s, a, pass);
      return hipGetLastError();
    }
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    hipLaunchKernelGGL((k_sort_count<BITS, EACH>), dim3(blocks), dim3(kSortThreads), 0, s, a, pass);
    hipLaunchKernelGGL((k_sort<BITS, EACH, false>), dim3(blocks), dim3(kSortThreads), 0, s, a, pass);
  }
  return hipGetLastError();
}

// ---- routing: a wave takes a token, a lane the experts lane, lane + 64, ...  Each of the
// k maxima is a chain of cross-lane steps, which bounds it: 16384 tokens, 6 of 64 in
// 8.3 us, the gradient in 7.7 (4 MB of logits are 1).

// Largest of a value over the wave, and the sum of one, in all lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MUON_STEP(ctrl) \
  v = umax(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, 0xf, 0xf, false)))
  MUON_STEP(0x111); MUON_STEP(0x112); MUON_STEP(0x114); MUON_STEP(0x118);   // within rows of 16
  MUON_STEP(0x142); MUON_STEP(0x143);                                       // across them
#undef MUON_STEP
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
#define MUON_STEP(ctrl) \
  v += __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), ctrl, 0xf, 0xf, false)))
  MUON_STEP(0x111); MUON_STEP(0x112); MUON_STEP(0x114); MUON_STEP(0x118);
  MUON_STEP(0x142); MUON_STEP(0x143);
#undef MUON_STEP
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), 63)));
}

// Unsigned integers in the order of the numbers: NaN first among them, both
// zeros equal, 0 for -inf, which is never chosen.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u == 0xff800000u ? 0u : u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_rank(uint32_t u) {
  return u == 0xffffffffu ? __uint_as_float(0x7fc00000u)
                          : __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
}

// Chooses token t's experts; V = experts a lane holds.
template <class T, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int lane) {
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float x[V];
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * 64 + lane;
    x[v] = i < a.experts ? load1(row + i) : __uint_as_float(0xff800000u);
    key[v] = rank_of(x[v]);
  }
  float top = 0.f, value = 0.f;
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = umax(m, key[v]);
    m = wave_max(m);
    if (m == 0) break;
    if (j == 0) top = of_rank(m);
    bool found = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t at = __ballot(key[v] == m);
      if (!found && at) {
        found = true;
        const int l = __builtin_ctzll(at);
        if (lane == l) key[v] = 0;
        if (lane == j) {
          mine = v * 64 + l;
          value = of_rank(m);
        }
      }
    }
  }
  // sum of exp(x - top) over all experts, or the chosen ones; 0 where none is there
  const float e = mine >= 0 ? expf(value - top) : 0.f;
  float sum = e;
  if (!a.normalize) {
    sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += rank_of(x[v]) == 0 ? 0.f : expf(x[v] - top);
  }
  sum = wave_sum(sum);
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(t) * a.k + lane;
    a.gates[at] = mine >= 0 ? e / sum : 0.f;
    a.chosen[at] = mine;
  }
}

constexpr int kRouteWaves = 4;
template <class T, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(RouteArgs a) {
  const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t < a.tokens) route_token<T, V>(a, t, threadIdx.x & 63);
}

// The same and the sort of the slots, for what one block sorts: one launch.
template <class T, int V, int BITS>
__global__ __launch_bounds__(kSortThreads) void k_route_sort(RouteArgs a, SortArgs s) {
  __shared__ SortShared<BITS> sh;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int t = wave; t < a.tokens; t += kSortWaves) route_token<T, V>(a, t, threadIdx.x & 63);
  __syncthreads();
  sort_pass<BITS, 1, true>(s, 0, sh);
}

template <class T, class D, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_grad(RouteGradArgs a) {
  const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.tokens) return;
  const int64_t at = static_cast<int64_t>(t) * a.k + lane;
  int chosen = -1;
  float g = 0.f, dg = 0.f;
  if (lane < a.k) {
    chosen = a.chosen[at];
    if (chosen >= 0 && chosen < a.experts) {
      g = a.gates[at];
      dg = a.dgates[at];
    } else {
      chosen = -1;
    }
  }
  const float inner = wave_sum(g * dg);
  const bool any = __ballot(chosen >= 0) != 0;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  D* out = static_cast<D*>(a.dlogits) + t * a.ldd;
  float p[V], d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = d[v] = 0.f;
  if (!a.normalize && any) {
    float x[V];
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * 64 + lane;
      x[v] = i < a.experts ? load1(row + i) : __uint_as_float(0xff800000u);
      m = umax(m, rank_of(x[v]));
    }
    const float top = of_rank(wave_max(m));
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = rank_of(x[v]) == 0 ? 0.f : expf(x[v] - top);
      sum += p[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] /= sum;
  }
  for (int j = 0; j < a.k; ++j) {
    const int c = __builtin_amdgcn_readlane(chosen, j);
    if (c < 0) continue;
    const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(dg), j));
    const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c == v * 64 + lane) {
        d[v] += dj;
        if (a.normalize) p[v] = gj;
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * 64 + lane;
    if (i < a.experts) store1(out + i, any ? p[v] * (d[v] - inner) : 0.f);
  }
}

// Calls f with the number of experts a lane holds.
template <class F>
hipError_t with_width(int experts, F&& f) {
  if (experts <= 64) return f(std::integral_constant<int, 1>{});
  if (experts <= 128) return f(std::integral_constant<int, 2>{});
  if (experts <= 256) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
  const bool wide = sort_bits(key_bits(a.limit)) == kSortWide;
  if (sort_each(a.n, a.limit) == 1)
    return wide ? launch_sort_of<kSortWide, 1>(a, s) : launch_sort_of<kSortBits, 1>(a, s);
  return wide ? launch_sort_of<kSortWide, 4>(a, s) : launch_sort_of<kSortBits, 4>(a, s);
}

hipError_t launch_route(const RouteArgs& a, const SortArgs& sort, int dt, hipStream_t s) {
  return with_width(a.experts, [&](auto v) {
    return with_type(dt, [&](auto z) {
      using T = decltype(z);
      constexpr int V = decltype(v)::value;
      if (a.tokens <= 4 * kSortWaves && sort.n <= kSortThreads) {
        if (sort_bits(key_bits(a.experts)) == kSortBits)
          hipLaunchKernelGGL((k_route_sort<T, V, kSortBits>), dim3(1), dim3(kSortThreads), 0, s, a, sort);
        else
          hipLaunchKernelGGL((k_route_sort<T, V, kSortWide>), dim3(1), dim3(kSortThreads), 0, s, a, sort);
        return hipGetLastError();
      }
      const int blocks = (a.tokens + kRouteWaves - 1) / kRouteWaves;
      hipLaunchKernelGGL((k_route<T, V>), dim3(blocks), dim3(64 * kRouteWaves), 0, s, a);
      const hipError_t e = hipGetLastError();
      return e == hipSuccess ? launch_sort(sort, s) : e;
    });
  });
}

hipError_t launch_route_grad(const RouteGradArgs& a, int dt, int ddt, hipStream_t s) {
  const int blocks = (a.tokens + kRouteWaves - 1) / kRouteWaves;
  return with_width(a.experts, [&](auto v) {
    return with_type(dt, [&](auto z) {
      return with_type(ddt, [&](auto y) {
        hipLaunchKernelGGL((k_route_grad<decltype(z), decltype(y), decltype(v)::value>), dim3(blocks),
                           dim3(64 * kRouteWaves), 0, s, a);
        return hipGetLastError();
      });
    });
  });
}

}  // namespace muon
