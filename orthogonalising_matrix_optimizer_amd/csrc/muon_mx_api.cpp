// C ABI of the 4-bit (MXFP4) operators and dropout: validation and launches.
//
// The operators are stated in include/muon.h.  Descriptors travel as kernel
// arguments, at most kMxMaxList matrices a launch, so a call needs neither a
// device table nor staging memory and may run under stream capture.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "../../include/muon.h"
#include "muon_check.h"
#include "muon_common.h"
#include "muon_mx.h"
#include "muon_span.h"

using namespace muon;

namespace {

// where an fp32 sum of equal terms stops growing; it also keeps the parts of a
// split contraction (kMinChunk code tiles at least) to 2^13
constexpr int64_t kMaxCols = int64_t(1) << 24;
// a grid has fewer than 2^32 threads: blocks of 256, and of the quantiser's 1024
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;
constexpr int64_t kMaxQuantBlocks = (int64_t(1) << 22) - 1;

bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMaxRows && cols <= kMaxCols;
}

int check_mx(const muon_mx& m) {
  if (!shape_ok(m.rows, m.cols)) return MUON_E_SHAPE;
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (!m.codes || !m.scales) return MUON_E_NULL;
  if (reinterpret_cast<uintptr_t>(m.codes) % 16 || reinterpret_cast<uintptr_t>(m.scales) % 16)
    return MUON_E_ALIGN;
  return MUON_OK;
}

void add_span(std::vector<Span>& v, const muon_mx& m, bool write) {
  if (m.rows == 0 || m.cols == 0) return;
  add_span(v, m.codes, muon_mx_codes_bytes(m.rows, m.cols), write);
  add_span(v, m.scales, muon_mx_scales_bytes(m.rows, m.cols), write);
}

// Dropout probability -> threshold in steps of 2^-16 and the kept elements' factor.
int drop_of(float p, uint64_t seed, const uint64_t* dev, MxDrop* d) {
  if (!(p >= 0.f && p < 1.f)) return MUON_E_HPARAM;
  const uint32_t t = uint32_t(std::floor(double(p) * 65536.0 + 0.5));
  if (t >= 65536) return MUON_E_HPARAM;
  if (reinterpret_cast<uintptr_t>(dev) % 8) return MUON_E_ALIGN;
  d->threshold = t;
  d->scale = 65536.f / float(65536 - t);
  d->seed = {seed, t ? dev : nullptr};
  return MUON_OK;
}

int64_t round_up(int64_t v, int64_t a) { return ceil_div(v, a) * a; }

// Whether `bytes` of outputs are written past the caches.  The memory side's
// cache holds 256 MiB: outputs of half of it and more push out what the next
// call reads, smaller ones may be read from it.  A quantisation and a product
// after each other, K = 2560, N = 10240, into the caches | past them: 4096 rows
// (80 MiB) 71 | 72 us, 8192 (160) 139 | 122, 12288 (240) 204 | 182, 16384 (320)
// 280 | 259; a layer's step of 8192 rows 462 | 453, of 16384 with dropout 882 | 877.
bool past_caches(int64_t bytes) { return bytes > int64_t(128) << 20; }

// How a list of products is run: the tile height, and the contraction length
// (in code tiles) above which a product is split, 0 for none; per product the
// workspace offset of its partial products.
constexpr int64_t kTileN = 128;
constexpr int64_t kMinChunk = 16;
struct ProductPlan {
  int tile_m = 256;
  int64_t chunk = 0;
  size_t bytes = 0;
  std::vector<size_t> offset;
};

// The splits of a contraction of kt code tiles have the same length (but the last).
int64_t even_chunk(int64_t kt, int64_t chunk) {
  return kt ? ceil_div(kt, ceil_div(kt, chunk)) : 1;
}

// Blocks that sum the parts of a split M x N product.
int64_t reduce_blocks(int64_t M, int64_t N) { return ceil_div(M * (round_up(N, 8) / 8), 256); }

// Microseconds a stage (128 columns) of a work item takes with 1, 2, 3 blocks
// on its CU, measured on MI355X: 256 x 128 tiles (two blocks a CU) and 128 x
// 128 (three).  Of the two the cheaper is taken, e.g. K = 2560, N = 2560: M =
// 2048 18 us with 128-high tiles and 20 with 256-high ones, 6000 29.5 and 27.5,
// 8192 35 and 43 (640 tall tiles leave half of the CUs one short); M = 8191, N
// = 10240: 132 and 121.
constexpr double kStage256[3] = {0.72, 1.10, 1.10}, kStage128[3] = {0.45, 0.68, 0.88};

// Time of a list whose items have `work` stages in all, the longest `longest`.
double list_us(const double* t, int per_cu, double items, double work, double longest) {
  if (items == 0) return 0;
  const int n = int(std::ceil(items / 256));             // items on a CU
  const double rounds = (n / per_cu) * t[per_cu - 1] + (n % per_cu ? t[n % per_cu - 1] : 0);
  return std::max(work / items * rounds, longest * t[std::min(n, per_cu) - 1]);
}

ProductPlan plan_products(const muon_mx* a, const muon_mx* b, int n) {
  ProductPlan p;
  double i256 = 0, i128 = 0, w256 = 0, w128 = 0, longest = 0;
  for (int i = 0; i < n; ++i) {
    const double tn = ceil_div(b[i].rows, kTileN), kt = ceil_div(a[i].cols, kMxTileK);
    const double n256 = ceil_div(a[i].rows, 256) * tn, n128 = ceil_div(a[i].rows, 128) * tn;
    i256 += n256;
    i128 += n128;
    w256 += n256 * kt;
    w128 += n128 * kt;
    if (n128 > 0) longest = std::max(longest, kt);
  }
  const double t256 = list_us(kStage256, 2, i256, w256, longest);
  double best = list_us(kStage128, 3, i128, w128, longest);
  p.tile_m = t256 < best ? 256 : 128;
  best = std::min(best, t256);
  // Splitting adds the partial products' way through the caches and back (8
  // TB/s) and a launch (5 us); it pays for few tiles with a long contraction and
  // for lists with one much longer than the rest, us (whole | split): 768 x 768
  // x 8192 33 | 20, 128 x 2560 x 10240 40 | 18, 1408 x 2048 x 16384 65 | 50,
  // twelve 768 x 768 with K of 1630 to 23201 100 | 66; but 2560 x 2560 x 16384
  // 81 | 88 and 512 x 2048 x 4096 19 | 20.
  for (int64_t c = kMinChunk; c < longest; c += c / 2) {
    double items = 0, bytes = 0, part = 0;
    bool fits = true;   // every product's items and sum in a launch of their own
    for (int i = 0; i < n; ++i) {
      const int64_t kt = ceil_div(a[i].cols, kMxTileK), splits = std::max<int64_t>(1, ceil_div(kt, c));
      const double own = double(splits) * ceil_div(a[i].rows, 128) * ceil_div(b[i].rows, kTileN);
      fits = fits && own <= kMaxBlocks && reduce_blocks(a[i].rows, b[i].rows) <= kMaxBlocks;
      part = std::max(part, double(even_chunk(kt, c)));
      items += own;
      bytes += 8.0 * splits * a[i].rows * b[i].rows;
    }
    if (!fits) continue;
    const double t = list_us(kStage128, 3, items, w128, part) + bytes / 8e6 + 5;
    if (t < 0.9 * best) {
      best = t / 0.9;
      p.chunk = c;
      p.tile_m = 128;
    }
  }
  if (p.chunk) {
    p.offset.assign(n, 0);
    for (int i = 0; i < n; ++i) {
      const int64_t kt = ceil_div(a[i].cols, kMxTileK);
      const int64_t splits = std::max<int64_t>(1, ceil_div(kt, even_chunk(kt, p.chunk)));
      p.offset[i] = p.bytes;
      p.bytes += size_t(splits) * a[i].rows * round_up(b[i].rows, 8) * 4;
      p.bytes = round_up(p.bytes, 256);
    }
  }
  return p;
}

// Deals a launch's work items to the eight XCDs: contiguous ranges (items that
// follow each other share operands) with an eighth of the stages each.  An empty
// item counts as one stage.
void share_out(MxGemmArgs& g, int64_t items) {
  auto own = [&](int i) { return (i + 1 < g.n ? g.base[i + 1] : items) - int64_t(g.base[i]); };
  auto per_item = [&](int i) { return std::max(1.0, double(g.m[i].tiles) * g.m[i].kt / own(i)); };
  double stages = 0;
  for (int i = 0; i < g.n; ++i) stages += own(i) * per_item(i);
  int64_t at = 0;
  double before = 0;
  int x = 0;
  g.c.xcd[0] = 0;
  for (int i = 0; i < g.n && x < 7; ++i) {
    const double per = per_item(i), part = own(i) * per;
    while (x < 7 && before + part >= stages * (x + 1) / 8) {
      const double want = (stages * (x + 1) / 8 - before) / per;
      g.c.xcd[++x] = int32_t(at + std::min<int64_t>(own(i), std::max<int64_t>(0, int64_t(want + 0.5))));
    }
    at += own(i);
    before += part;
  }
  while (x < 8) g.c.xcd[++x] = int32_t(items);
}

// Shapes and types of one product of a list.
int check_product(const muon_mx& a, const muon_mx& b, const muon_mat& out, const muon_mat& first) {
  if (out.dtype != first.dtype) return MUON_E_DTYPE;
  if (a.cols != b.cols || out.rows != a.rows || out.cols != b.rows) return MUON_E_SHAPE;
  if (ceil_div(a.rows, 128) * ceil_div(b.rows, kTileN) > kMaxBlocks) return MUON_E_SHAPE;
  return MUON_OK;
}

// Arguments of a launch of products and of the launch that sums their parts.
struct ProductLaunch {
  MxGemmArgs g;
  MxReduceArgs red;
  int64_t items, blocks, written;   // work items, blocks of the sum, bytes of output
  ProductLaunch() { std::memset(this, 0, sizeof(*this)); }
};

// Fills l with the list's products and calls run() for each launch.  With a
// split contraction every product of the list writes fp32 partials, so that one
// launch holds them all.
template <class Run>
int build_launches(const muon_mx* a, const muon_mx* b, const muon_mat* out, int32_t n,
                   const ProductPlan& plan, char* workspace, ProductLaunch& l, Run run) {
  const bool split = plan.chunk != 0;
  int rc;
  auto flush = [&]() {
    if (l.g.n == 0) return int(MUON_OK);
    share_out(l.g, l.items);
    const int code = run();
    l.g.n = l.red.n = 0;
    l.items = l.blocks = l.written = 0;
    return code;
  };
  for (int i = 0; i < n; ++i) {
    const int64_t M = a[i].rows, N = b[i].rows, kt = ceil_div(a[i].cols, kMxTileK);
    const int64_t tiles = ceil_div(M, plan.tile_m) * ceil_div(N, kTileN);
    if (tiles == 0) continue;
    const int64_t chunk = split ? even_chunk(kt, plan.chunk) : std::max<int64_t>(kt, 1);
    const int64_t splits = std::max<int64_t>(1, ceil_div(kt, chunk));
    const int64_t nb = split ? reduce_blocks(M, N) : 0;
    if (l.g.n == kMxMaxList || l.items + tiles * splits > kMaxBlocks || l.blocks + nb > kMaxBlocks)
      if ((rc = flush()) != MUON_OK) return rc;
    MxProduct& p = l.g.m[l.g.n];
    p.ac = static_cast<const uint8_t*>(a[i].codes);
    p.as = static_cast<const uint8_t*>(a[i].scales);
    p.bc = static_cast<const uint8_t*>(b[i].codes);
    p.bs = static_cast<const uint8_t*>(b[i].scales);
    p.out = out[i].ptr;
    p.ld = out[i].ld;
    p.stride = 0;
    p.M = int32_t(M);
    p.N = int32_t(N);
    p.kt = int32_t(kt);
    p.chunk = int32_t(chunk);
    p.tiles = int32_t(tiles);
    p.index = i;
    if (split) {
      MxReduce& r = l.red.m[l.g.n];
      std::memset(&r, 0, sizeof(r));
      r.ldp = int32_t(round_up(N, 8));
      r.stride = M * r.ldp;
      r.in = workspace ? reinterpret_cast<const float*>(workspace + plan.offset[i]) : nullptr;
      r.out = out[i].ptr;
      r.ld = out[i].ld;
      r.M = p.M;
      r.N = p.N;
      r.splits = int32_t(splits);
      r.index = i;
      l.red.base[l.g.n] = uint32_t(l.blocks);
      l.red.n = l.g.n + 1;
      p.out = const_cast<float*>(r.in);
      p.ld = r.ldp;
      p.stride = r.stride;
    }
    l.g.base[l.g.n++] = uint32_t(l.items);
    l.items += tiles * splits;
    l.blocks += nb;
    l.written += M * N * esize(out[i].dtype);
  }
  return flush();
}

}  // namespace

extern "C" {

void muon_mx_default_options(muon_mx_options* o) {
  if (o) std::memset(o, 0, sizeof(*o));
}

size_t muon_mx_codes_bytes(int64_t rows, int64_t cols) {
  if (!shape_ok(rows, cols)) return 0;
  return size_t(ceil_div(rows, kMxTileR)) * size_t(ceil_div(cols, kMxTileK)) * kMxTileBytes;
}

size_t muon_mx_scales_bytes(int64_t rows, int64_t cols) {
  if (!shape_ok(rows, cols)) return 0;
  return size_t(ceil_div(rows, kMxScaleRows)) * size_t(ceil_div(cols, kMxTileK)) * kMxScaleBytes;
}

int muon_mx_quantize(const muon_mat* in, const muon_mx* out, const muon_mx* out_t, int32_t n,
                     const muon_mx_options* opt, void* stream) try {
  if (n < 0) return MUON_E_SHAPE;
  if (n == 0) return MUON_OK;
  if (!in || (!out && !out_t)) return MUON_E_NULL;
  muon_mx_options o;
  muon_mx_default_options(&o);
  if (opt) o = *opt;
  MxQuantArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc;
  if ((rc = drop_of(o.dropout, o.dropout_seed, o.dropout_seed_dev, &a.c.drop)) != MUON_OK) return rc;
  if (reinterpret_cast<uintptr_t>(o.seed_dev) % 8) return MUON_E_ALIGN;
  a.c.seed = {o.seed, o.stochastic ? o.seed_dev : nullptr};
  std::vector<Span> spans;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_dense(in[i])) != MUON_OK) return rc;
    if (in[i].dtype != in[0].dtype) return MUON_E_DTYPE;
    const int64_t r = in[i].rows, c = in[i].cols;
    if (out) {
      if ((rc = check_mx(out[i])) != MUON_OK) return rc;
      if (out[i].rows != r || out[i].cols != c) return MUON_E_SHAPE;
      add_span(spans, out[i], true);
    }
    if (out_t) {
      if ((rc = check_mx(out_t[i])) != MUON_OK) return rc;
      if (out_t[i].rows != c || out_t[i].cols != r) return MUON_E_SHAPE;
      add_span(spans, out_t[i], true);
    }
    if (ceil_div(r, kMxQuantTile) * ceil_div(c, kMxQuantTile) > kMaxQuantBlocks) return MUON_E_SHAPE;
    add_span(spans, in[i], false);
  }
  add_span(spans, a.c.seed.dev, sizeof(uint64_t), false);
  add_span(spans, a.c.drop.seed.dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;

  hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t blocks = 0;
  auto flush = [&]() {
    if (a.n && launch_mx_quantize(a, in[0].dtype, out, out_t, o.stochastic, blocks, s) != hipSuccess)
      return MUON_E_HIP;
    a.n = 0;
    blocks = 0;
    return MUON_OK;
  };
  for (int i = 0; i < n; ++i) {
    const int64_t nb = ceil_div(in[i].rows, kMxQuantTile) * ceil_div(in[i].cols, kMxQuantTile);
    if (nb == 0) continue;
    if (a.n == kMxMaxList || blocks + nb > kMaxQuantBlocks)
      if ((rc = int(flush())) != MUON_OK) return rc;
    MxQuantMat& m = a.m[a.n];
    std::memset(&m, 0, sizeof(m));
    m.in = in[i].ptr;
    m.ld = in[i].ld;
    m.rows = int32_t(in[i].rows);
    m.cols = int32_t(in[i].cols);
    m.index = i;
    if (out) {
      m.codes = static_cast<uint8_t*>(out[i].codes);
      m.scales = static_cast<uint8_t*>(out[i].scales);
    }
    if (out_t) {
      m.codes_t = static_cast<uint8_t*>(out_t[i].codes);
      m.scales_t = static_cast<uint8_t*>(out_t[i].scales);
    }
    a.base[a.n++] = uint32_t(blocks);
    blocks += nb;
  }
  return flush();
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_mx_dequantize(const muon_mx* in, const muon_mat* out, int32_t n, void* stream) try {
  if (n < 0) return MUON_E_SHAPE;
  if (n == 0) return MUON_OK;
  if (!in || !out) return MUON_E_NULL;
  std::vector<Span> spans;
  int rc;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_mx(in[i])) != MUON_OK || (rc = check_dense(out[i])) != MUON_OK) return rc;
    if (out[i].dtype != out[0].dtype) return MUON_E_DTYPE;
    if (in[i].rows != out[i].rows || in[i].cols != out[i].cols) return MUON_E_SHAPE;
    if (ceil_div(in[i].rows, kMxQuantTile) * ceil_div(in[i].cols, kMxQuantTile) > kMaxBlocks)
      return MUON_E_SHAPE;
    add_span(spans, in[i], false);
    add_span(spans, out[i], true);
  }
  if (conflict(spans)) return MUON_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  MxDequantArgs a;
  std::memset(&a, 0, sizeof(a));
  int64_t blocks = 0;
  auto flush = [&]() {
    if (a.n && launch_mx_dequantize(a, out[0].dtype, blocks, s) != hipSuccess) return MUON_E_HIP;
    a.n = 0;
    blocks = 0;
    return MUON_OK;
  };
  for (int i = 0; i < n; ++i) {
    const int64_t nb = ceil_div(in[i].rows, kMxQuantTile) * ceil_div(in[i].cols, kMxQuantTile);
    if (nb == 0) continue;
    if (a.n == kMxMaxList || blocks + nb > kMaxBlocks)
      if ((rc = int(flush())) != MUON_OK) return rc;
    MxDequantMat& m = a.m[a.n];
    m.codes = static_cast<const uint8_t*>(in[i].codes);
    m.scales = static_cast<const uint8_t*>(in[i].scales);
    m.out = out[i].ptr;
    m.ld = out[i].ld;
    m.rows = int32_t(in[i].rows);
    m.cols = int32_t(in[i].cols);
    a.base[a.n++] = uint32_t(blocks);
    blocks += nb;
  }
  return flush();
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

size_t muon_mx_matmul_workspace_bytes(const muon_mx* a, const muon_mx* b, int32_t n) try {
  if (n <= 0 || !a || !b) return 0;
  for (int i = 0; i < n; ++i)
    if (!shape_ok(a[i].rows, a[i].cols) || !shape_ok(b[i].rows, b[i].cols) || a[i].cols != b[i].cols)
      return 0;
  return plan_products(a, b, n).bytes;
} catch (...) {   // an allocation of the host's failed
  return 0;
}

int muon_mx_matmul(const muon_mx* a, const muon_mx* b, const muon_mat* out, int32_t n,
                   const muon_mx_options* opt, void* workspace, size_t workspace_bytes,
                   void* stream) try {
  if (n < 0) return MUON_E_SHAPE;
  if (n == 0) return MUON_OK;
  if (!a || !b || !out) return MUON_E_NULL;
  muon_mx_options o;
  muon_mx_default_options(&o);
  if (opt) o = *opt;
  MxReduceCommon red_common;
  std::memset(&red_common, 0, sizeof(red_common));
  int rc;
  if ((rc = drop_of(o.dropout, o.dropout_seed, o.dropout_seed_dev, &red_common.drop)) != MUON_OK) return rc;
  red_common.accumulate = o.accumulate != 0;
  std::vector<Span> spans;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_mx(a[i])) != MUON_OK || (rc = check_mx(b[i])) != MUON_OK ||
        (rc = check_dense(out[i])) != MUON_OK)
      return rc;
    if ((rc = check_product(a[i], b[i], out[i], out[0])) != MUON_OK) return rc;
    add_span(spans, a[i], false);
    add_span(spans, b[i], false);
    add_span(spans, out[i], true);
  }
  const ProductPlan plan = plan_products(a, b, n);
  if (plan.bytes) {
    if (!workspace || workspace_bytes < plan.bytes) return MUON_E_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return MUON_E_ALIGN;
    add_span(spans, workspace, plan.bytes, true);
  }
  add_span(spans, red_common.drop.seed.dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);

  ProductLaunch l;
  l.red.c = red_common;
  l.g.c.accumulate = plan.chunk ? 0 : red_common.accumulate;
  if (!plan.chunk) l.g.c.drop = red_common.drop;
  return build_launches(a, b, out, n, plan, static_cast<char*>(workspace), l, [&]() {
    if (launch_mx_gemm(l.g, plan.chunk ? int(kF32) : out[0].dtype, plan.tile_m,
                       plan.chunk || !past_caches(l.written), s) != hipSuccess)
      return MUON_E_HIP;
    if (l.red.n && launch_mx_reduce(l.red, out[0].dtype, l.blocks, s) != hipSuccess)
      return MUON_E_HIP;
    return MUON_OK;
  });
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_mx_plan_info(const muon_mx* a, const muon_mx* b, const muon_mat* out, int32_t n,
                      int32_t* tile_rows, int32_t* parts, int32_t* past, int32_t* xcd_items) try {
  if (n <= 0) return MUON_E_SHAPE;
  if (!a || !b || !out) return MUON_E_NULL;
  int rc;
  for (int i = 0; i < n; ++i) {
    if (out[i].dtype != MUON_BF16 && out[i].dtype != MUON_F32) return MUON_E_DTYPE;
    if (!shape_ok(a[i].rows, a[i].cols) || !shape_ok(b[i].rows, b[i].cols)) return MUON_E_SHAPE;
    if ((rc = check_product(a[i], b[i], out[i], out[0])) != MUON_OK) return rc;
  }
  const ProductPlan plan = plan_products(a, b, n);
  if (tile_rows) *tile_rows = plan.tile_m;
  if (past) *past = 0;
  if (xcd_items) std::fill(xcd_items, xcd_items + 9, 0);
  if (parts) std::fill(parts, parts + n, 0);
  ProductLaunch l;
  bool first = true;
  return build_launches(a, b, out, n, plan, nullptr, l, [&]() {
    for (int j = 0; j < l.g.n && parts; ++j)
      parts[l.g.m[j].index] = std::max(1, int(ceil_div(l.g.m[j].kt, l.g.m[j].chunk)));
    if (first) {
      if (past) *past = !plan.chunk && past_caches(l.written);
      if (xcd_items) std::copy(l.g.c.xcd, l.g.c.xcd + 9, xcd_items);
    }
    first = false;
    return MUON_OK;
  });
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_mx_matmul_rows(const muon_mat* x, const muon_mx* b, const muon_mat* out,
                        void* stream) try {
  if (!x || !b || !out) return MUON_E_NULL;
  int rc;
  if ((rc = check_dense(*x)) != MUON_OK || (rc = check_mx(*b)) != MUON_OK ||
      (rc = check_dense(*out)) != MUON_OK)
    return rc;
  if (x->rows > MUON_MX_FEW_ROWS || x->cols != b->cols || out->rows != x->rows || out->cols != b->rows)
    return MUON_E_SHAPE;
  if (b->rows > MUON_MX_FEW_ROWS_MAX_N) return MUON_E_SHAPE;
  std::vector<Span> spans;
  add_span(spans, *x, false);
  add_span(spans, *b, false);
  add_span(spans, *out, true);
  if (conflict(spans)) return MUON_E_ALIAS;
  if (out->rows == 0 || out->cols == 0) return MUON_OK;
  MxRowsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x->ptr;
  a.ldx = x->ld;
  a.bc = static_cast<const uint8_t*>(b->codes);
  a.bs = static_cast<const uint8_t*>(b->scales);
  a.out = out->ptr;
  a.ldo = out->ld;
  a.M = int32_t(x->rows);
  a.N = int32_t(b->rows);
  a.K = int32_t(x->cols);
  return launch_mx_rows(a, x->dtype, out->dtype, static_cast<hipStream_t>(stream)) == hipSuccess
             ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_dropout(const muon_mat* in, const muon_mat* out, float p, uint64_t seed,
                 const uint64_t* seed_dev, void* stream) try {
  if (!in || !out) return MUON_E_NULL;
  MxDropArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc;
  if ((rc = drop_of(p, seed, seed_dev, &a.drop)) != MUON_OK) return rc;
  if ((rc = check_dense(*in)) != MUON_OK || (rc = check_dense(*out)) != MUON_OK) return rc;
  if (in->dtype != out->dtype) return MUON_E_DTYPE;
  if (in->rows != out->rows || in->cols != out->cols) return MUON_E_SHAPE;
  if (in->rows == 0 || in->cols == 0) return MUON_OK;
  const int64_t blocks = ceil_div(in->rows * ceil_div(in->cols, 8), kDropItems);
  if (blocks > kMaxBlocks) return MUON_E_SHAPE;
  std::vector<Span> spans;
  add_span(spans, *out, true);
  // in place is allowed: every element is read by the lane that writes it
  if (!(in->ptr == out->ptr && in->ld == out->ld)) add_span(spans, *in, false);
  add_span(spans, a.drop.seed.dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;
  a.in = in->ptr;
  a.out = out->ptr;
  a.ldi = in->ld;
  a.ldo = out->ld;
  a.rows = int32_t(in->rows);
  a.cols = int32_t(in->cols);
  return launch_dropout(a, in->dtype, blocks, static_cast<hipStream_t>(stream)) == hipSuccess
             ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

}  // extern "C"
