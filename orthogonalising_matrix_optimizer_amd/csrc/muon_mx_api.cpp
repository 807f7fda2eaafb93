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
#include "muon_common.h"
#include "muon_mx.h"

using namespace muon;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
// the products address a panel of 256 rows with 32-bit offsets
constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;   // of 256 threads: the grid limit

int esize(int dt) { return dt == MUON_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMaxRows && cols <= kMaxCols;
}

// A matrix of any size, zero included; rows need only element alignment.
int check_dense(const muon_mat& m) {
  if (m.dtype != MUON_BF16 && m.dtype != MUON_F32) return MUON_E_DTYPE;
  if (m.rows < 0 || m.cols < 0 || m.rows > kMaxRows || m.cols > kMaxRows) return MUON_E_SHAPE;
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (m.ld < m.cols || m.ld > (int64_t(1) << 40)) return MUON_E_SHAPE;
  if (!m.ptr) return MUON_E_NULL;
  if (reinterpret_cast<uintptr_t>(m.ptr) % esize(m.dtype)) return MUON_E_ALIGN;
  return MUON_OK;
}

int check_mx(const muon_mx& m) {
  if (!shape_ok(m.rows, m.cols)) return MUON_E_SHAPE;
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (!m.codes || !m.scales) return MUON_E_NULL;
  if (reinterpret_cast<uintptr_t>(m.codes) % 16 || reinterpret_cast<uintptr_t>(m.scales) % 16)
    return MUON_E_ALIGN;
  return MUON_OK;
}

bool vec_ok(const muon_mat& m) {
  return reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && (m.ld * esize(m.dtype)) % 16 == 0;
}

// Memory that a call reads or writes: `width` bytes in every `pitch` from lo
// on, up to hi.
struct Span {
  uintptr_t lo, hi;
  size_t pitch, width;
  bool write;
};

void add_span(std::vector<Span>& v, const void* p, size_t bytes, bool write) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (p && bytes) v.push_back({a, a + bytes, bytes, bytes, write});
}

void add_span(std::vector<Span>& v, const muon_mat& m, bool write) {
  if (m.rows == 0 || m.cols == 0) return;
  const uintptr_t a = reinterpret_cast<uintptr_t>(m.ptr);
  const size_t es = esize(m.dtype);
  v.push_back({a, a + (size_t(m.rows - 1) * m.ld + m.cols) * es, size_t(m.ld) * es,
               size_t(m.cols) * es, write});
}

void add_span(std::vector<Span>& v, const muon_mx& m, bool write) {
  if (m.rows == 0 || m.cols == 0) return;
  add_span(v, m.codes, muon_mx_codes_bytes(m.rows, m.cols), write);
  add_span(v, m.scales, muon_mx_scales_bytes(m.rows, m.cols), write);
}

// Whether two spans share a byte; column slices of one buffer do not.
bool share(const Span& a, const Span& b) {
  if (b.lo >= a.hi || a.lo >= b.hi) return false;
  if (a.pitch != b.pitch) return true;
  const size_t d = (a.lo < b.lo ? b.lo - a.lo : a.lo - b.lo) % a.pitch;
  const size_t first = a.lo < b.lo ? a.width : b.width, second = a.lo < b.lo ? b.width : a.width;
  return d < first || d + second > a.pitch;
}

// Whether something written is also read or written through another argument.
bool conflict(std::vector<Span>& v) {
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  // the spans still open at the next one's start: only they can share bytes with it
  std::vector<Span> open;
  for (const Span& s : v) {
    size_t kept = 0;
    for (const Span& o : open)
      if (o.hi > s.lo) {
        if ((o.write || s.write) && share(o, s)) return true;
        open[kept++] = o;
      }
    open.resize(kept);
    // equal spans that are only read count once
    if (!(kept && !s.write && open[kept - 1].lo == s.lo && open[kept - 1].hi == s.hi &&
          !open[kept - 1].write))
      open.push_back(s);
  }
  return false;
}

// Dropout probability -> threshold in steps of 2^-16 and the kept elements' factor.
int drop_of(float p, uint32_t* thr, float* scale) {
  if (!(p >= 0.f && p < 1.f)) return MUON_E_HPARAM;
  const uint32_t t = uint32_t(std::floor(double(p) * 65536.0 + 0.5));
  if (t >= 65536) return MUON_E_HPARAM;
  *thr = t;
  *scale = 65536.f / float(65536 - t);
  return MUON_OK;
}

int seed_ok(const uint64_t* dev) {
  return reinterpret_cast<uintptr_t>(dev) % 8 ? MUON_E_ALIGN : MUON_OK;
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
  uint32_t thr = 0;
  float scale = 1.f;
  int rc;
  if ((rc = drop_of(o.dropout, &thr, &scale)) != MUON_OK) return rc;
  if ((rc = seed_ok(o.seed_dev)) != MUON_OK || (rc = seed_ok(o.dropout_seed_dev)) != MUON_OK) return rc;
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
    if (ceil_div(r, kMxQuantTile) * ceil_div(c, kMxQuantTile) > kMaxBlocks) return MUON_E_SHAPE;
    add_span(spans, in[i], false);
  }
  if (o.stochastic) add_span(spans, o.seed_dev, sizeof(uint64_t), false);
  if (thr) add_span(spans, o.dropout_seed_dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;

  hipStream_t s = static_cast<hipStream_t>(stream);
  MxQuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.drop = thr;
  a.drop_scale = scale;
  a.seed = {o.seed, o.stochastic ? o.seed_dev : nullptr};
  a.drop_seed = {o.dropout_seed, thr ? o.dropout_seed_dev : nullptr};
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
    if (a.n == kMxMaxList || blocks + nb > kMaxBlocks)
      if ((rc = int(flush())) != MUON_OK) return rc;
    MxQuantMat& m = a.m[a.n];
    std::memset(&m, 0, sizeof(m));
    m.in = in[i].ptr;
    m.ld = in[i].ld;
    m.rows = int32_t(in[i].rows);
    m.cols = int32_t(in[i].cols);
    m.vec = vec_ok(in[i]);
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
    m.vec = vec_ok(out[i]);
    a.base[a.n++] = uint32_t(blocks);
    blocks += nb;
  }
  return flush();
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_mx_matmul(const muon_mx* a, const muon_mx* b, const muon_mat* out, int32_t n,
                   const muon_mx_options* opt, void* stream) try {
  if (n < 0) return MUON_E_SHAPE;
  if (n == 0) return MUON_OK;
  if (!a || !b || !out) return MUON_E_NULL;
  muon_mx_options o;
  muon_mx_default_options(&o);
  if (opt) o = *opt;
  MxGemmArgs g;
  std::memset(&g, 0, sizeof(g));
  int rc;
  if ((rc = drop_of(o.dropout, &g.drop, &g.drop_scale)) != MUON_OK) return rc;
  if ((rc = seed_ok(o.dropout_seed_dev)) != MUON_OK) return rc;
  g.accumulate = o.accumulate != 0;
  g.drop_seed = {o.dropout_seed, g.drop ? o.dropout_seed_dev : nullptr};
  std::vector<Span> spans;
  const int ts = 128;
  for (int i = 0; i < n; ++i) {
    if ((rc = check_mx(a[i])) != MUON_OK || (rc = check_mx(b[i])) != MUON_OK ||
        (rc = check_dense(out[i])) != MUON_OK)
      return rc;
    if (out[i].dtype != out[0].dtype) return MUON_E_DTYPE;
    if (a[i].cols != b[i].cols || out[i].rows != a[i].rows || out[i].cols != b[i].rows)
      return MUON_E_SHAPE;
    if (ceil_div(a[i].rows, ts) * ceil_div(b[i].rows, ts) > kMaxBlocks) return MUON_E_SHAPE;
    add_span(spans, a[i], false);
    add_span(spans, b[i], false);
    add_span(spans, out[i], true);
  }
  if (g.drop) add_span(spans, o.dropout_seed_dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t blocks = 0;
  auto flush = [&]() {
    if (g.n && launch_mx_gemm(g, out[0].dtype, ts, blocks, s) != hipSuccess) return MUON_E_HIP;
    g.n = 0;
    blocks = 0;
    return MUON_OK;
  };
  for (int i = 0; i < n; ++i) {
    const int64_t nb = ceil_div(a[i].rows, ts) * ceil_div(b[i].rows, ts);
    if (nb == 0) continue;
    if (g.n == kMxMaxList || blocks + nb > kMaxBlocks)
      if ((rc = int(flush())) != MUON_OK) return rc;
    MxProduct& p = g.p[g.n];
    p.ac = static_cast<const uint8_t*>(a[i].codes);
    p.as = static_cast<const uint8_t*>(a[i].scales);
    p.bc = static_cast<const uint8_t*>(b[i].codes);
    p.bs = static_cast<const uint8_t*>(b[i].scales);
    p.out = out[i].ptr;
    p.ld = out[i].ld;
    p.M = int32_t(a[i].rows);
    p.N = int32_t(b[i].rows);
    p.kt = int32_t(ceil_div(a[i].cols, kMxTileK));
    p.index = i;
    g.base[g.n++] = uint32_t(blocks);
    blocks += nb;
  }
  return flush();
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_dropout(const muon_mat* in, const muon_mat* out, float p, uint64_t seed,
                 const uint64_t* seed_dev, void* stream) try {
  if (!in || !out) return MUON_E_NULL;
  MxDropArgs a;
  std::memset(&a, 0, sizeof(a));
  int rc;
  if ((rc = drop_of(p, &a.drop, &a.scale)) != MUON_OK || (rc = seed_ok(seed_dev)) != MUON_OK) return rc;
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
  if (a.drop) add_span(spans, seed_dev, sizeof(uint64_t), false);
  if (conflict(spans)) return MUON_E_ALIAS;
  a.in = in->ptr;
  a.out = out->ptr;
  a.ldi = in->ld;
  a.ldo = out->ld;
  a.rows = int32_t(in->rows);
  a.cols = int32_t(in->cols);
  a.vec = vec_ok(*in) && vec_ok(*out);
  a.seed = {seed, a.drop ? seed_dev : nullptr};
  return launch_dropout(a, in->dtype, blocks, static_cast<hipStream_t>(stream)) == hipSuccess
             ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

}  // extern "C"
