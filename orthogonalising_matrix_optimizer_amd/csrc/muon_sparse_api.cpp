// C ABI of the embedding table and the expert layers: validation and launches.
// The operators are stated in include/muon.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../../include/muon.h"
#include "muon_check.h"
#include "muon_sparse.h"
#include "muon_span.h"

using namespace muon;

namespace {

// a grid has fewer than 2^32 threads, in blocks of at most 512 here
constexpr int64_t kMaxBlocks = (int64_t(1) << 23) - 1;
constexpr int64_t kMaxCols = int64_t(1) << 24;

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// A matrix whose rows are as long as these kernels take.
int check_rows(const muon_mat& m) {
  const int rc = check_dense(m);
  return rc == MUON_OK && m.cols > kMaxCols ? int(MUON_E_SHAPE) : rc;
}

int check_stack(const muon_stack& w) {
  if (w.dtype != MUON_BF16 && w.dtype != MUON_F32) return MUON_E_DTYPE;
  if (w.count < 1 || w.count > MUON_MAX_EXPERTS || w.rows < 0 || w.cols < 0 || w.rows > kMaxCols || w.cols > kMaxCols)
    return MUON_E_SHAPE;
  if (w.rows == 0 || w.cols == 0) return MUON_OK;
  if (w.ld < w.cols || w.ld > (int64_t(1) << 40) || !fits(w.rows, w.ld, w.cols)) return MUON_E_SHAPE;
  const int64_t one = (w.rows - 1) * w.ld + w.cols;
  if (w.count > 1 && (w.stride < one || !fits(w.count, w.stride, one))) return MUON_E_SHAPE;
  if (!w.ptr) return MUON_E_NULL;
  if (misaligned(w.ptr, esize(w.dtype))) return MUON_E_ALIGN;
  return MUON_OK;
}

void add_span(std::vector<Span>& v, const muon_stack& w, bool write) {
  const muon_mat m = {w.ptr, w.rows, w.cols, w.ld, w.dtype, 0};
  if (w.count > 1 && w.stride == w.rows * w.ld) {
    muon_mat all = m;
    all.rows *= w.count;
    muon::add_span(v, all, write);
    return;
  }
  for (int64_t e = 0; e < w.count; ++e) {
    muon_mat one = m;
    one.ptr = static_cast<char*>(w.ptr) + e * w.stride * esize(w.dtype);
    muon::add_span(v, one, write);
  }
}

int check_counts(int64_t n_tokens, int64_t k, int64_t experts) {
  if (n_tokens < 0 || k < 1 || k > MUON_MAX_K || experts < 1 || experts > MUON_MAX_EXPERTS) return MUON_E_SHAPE;
  return n_tokens > MUON_MAX_SLOTS / k ? MUON_E_SHAPE : MUON_OK;
}

int64_t slots_of(const muon_slots& s) { return s.n_tokens * s.k; }

int check_slots(const muon_slots* s) {
  if (!s) return MUON_E_NULL;
  const int rc = check_counts(s->n_tokens, s->k, s->experts);
  if (rc != MUON_OK) return rc;
  if (!s->offsets || (s->n_tokens && (!s->tokens || !s->place))) return MUON_E_NULL;
  if (misaligned(s->offsets, 4) || misaligned(s->tokens, 4) || misaligned(s->place, 4)) return MUON_E_ALIGN;
  return MUON_OK;
}

void add_span(std::vector<Span>& v, const muon_slots& s, bool write) {
  muon::add_span(v, s.offsets, (size_t(s.experts) + 1) * 4, write);
  muon::add_span(v, s.tokens, size_t(slots_of(s)) * 4, write);
  muon::add_span(v, s.place, size_t(slots_of(s)) * 4, write);
}

int check_ids(const muon_ids* ids) {
  if (!ids) return MUON_E_NULL;
  if (ids->bytes != 4 && ids->bytes != 8) return MUON_E_DTYPE;
  if (ids->n < 0 || ids->n > MUON_MAX_SLOTS) return MUON_E_SHAPE;
  if (ids->n && !ids->ptr) return MUON_E_NULL;
  return misaligned(ids->ptr, ids->bytes) ? int(MUON_E_ALIGN) : int(MUON_OK);
}

int check_workspace(std::vector<Span>& v, void* ws, size_t have, size_t need) {
  if (!need) return MUON_OK;
  if (!ws || have < need) return MUON_E_WORKSPACE;
  if (misaligned(ws, 16)) return MUON_E_ALIGN;
  muon::add_span(v, ws, need, true);
  return MUON_OK;
}

// ---- sort

int64_t sort_blocks(int64_t n, int64_t limit) { return ceil_div(n, kSortThreads * sort_each(n, limit)); }
int sort_passes(int64_t limit) { return int(ceil_div(key_bits(limit), sort_bits(key_bits(limit)))); }

// Bytes of a sort's counts.
size_t count_bytes(int64_t n, int64_t limit) {
  const int64_t blocks = sort_blocks(n, limit);
  return blocks <= kSortSelf ? 0 : size_t(blocks) * 4 << sort_bits(key_bits(limit));
}

SortArgs slots_sort(const void* choice, int id_bytes, const muon_slots& s, void* workspace) {
  SortArgs a;
  std::memset(&a, 0, sizeof(a));
  a.ids = choice;
  a.id_bytes = id_bytes;
  a.n = int32_t(slots_of(s));
  a.limit = s.experts;
  a.passes = 1;                       // an expert's number is one digit
  a.counts = static_cast<int32_t*>(workspace);
  a.offsets = s.offsets;
  a.tokens = s.tokens;
  a.place = s.place;
  a.k = s.k;
  return a;
}

// ---- products

// Rows of 16-byte pieces that start at 16 bytes.
bool pieces(const void* p, int64_t ld, int64_t inner) {
  return !misaligned(p, 16) && ld % 8 == 0 && inner % 8 == 0;
}

// Shared checks of the three products: rows operand, columns operand, slots.
int check_products(const muon_mat& r, int dt, const muon_slots* s, std::vector<Span>& v) {
  int rc;
  if ((rc = check_slots(s)) != MUON_OK || (rc = check_rows(r)) != MUON_OK) return rc;
  if (r.dtype != dt) return MUON_E_DTYPE;
  add_span(v, *s, false);
  add_span(v, r, false);
  return MUON_OK;
}

// Whether `rows` rows of a gathered x can be addressed.
bool spans(const muon_mat& x) {
  return x.rows == 0 || ((x.rows - 1) * x.ld + x.cols) * esize(x.dtype) < int64_t(kExpertSpan);
}

// Output tile of a product (64, 128 or 256 on a side) by an estimate of its time: the
// rounds of tiles that the device's 256 CUs take, times the stages of 64 contraction
// elements of a tile at what each costs, measured on MI355X with 1, 2 and 3 blocks a
// CU, us: 256: 1.7, 128: 1.2 (0.8 alone), 64: 0.6; fp32 (one block, three) 128: 3.1, 64:
// 3.1 (2.4 alone); and a tile's own start and end.  A launch's last round of tiles with
// a CU to themselves counts whole.  fwd, us with tiles of 64 | 128 |
// 256: 4096 slots, 8 experts, 1024 -> 2048: 39 | 38 | 34; 16384 slots, 1024 -> 1024: 62
// | 52 | 61; 48 slots, 64 experts, 2048 -> 1408: 37 | 32 | 49, 12000: 170 | 128 | 131; fp32
// 8192 slots, 32 experts, 1024 -> 1024: 150 | 140; 32768, 8, 2048 -> 1024: 965 | 813.
int tile_of(const ExpertArgs& a, int op, int dt, bool aligned) {
  if (op == kExpertPart) return 64;
  if (const char* e = std::getenv("MUON_EXPERT_TILE")) {
    const int t = std::atoi(e);
    if (t == 64 || t == 128 || (t == 256 && aligned)) return t;
  }
  // of the experts, those that a few slots can reach
  const double used = std::min<double>(a.experts, a.slots);
  const double depth = op == kExpertDw ? 1.5 * a.slots / a.experts : a.depth;
  const double stages = std::ceil(depth / 64);
  auto time = [&](int t, double slots, double each, double alone, double own) {
    const double across = double(ceil_div(a.cols, t));
    // half a tile too many for an expert, on average
    const double high = op == kExpertDw ? double(a.experts) * ceil_div(a.rows, t) : double(a.slots) / t + 0.5 * used;
    const double rounds = high * across / slots;
    const double whole = rounds <= 1 ? 1 : slots == 256 ? std::ceil(rounds) : rounds + 0.3;
    return whole * (stages * (rounds <= 0.5 ? alone : each) + own);
  };
  if (dt == MUON_F32) return time(64, 768, 3.1, 2.4, 3) <= time(128, 256, 3.1, 3.1, 4) ? 64 : 128;
  const double t64 = time(64, 768, 0.6, 0.5, 3), t128 = time(128, 512, 1.2, 0.8, 3);
  if (!aligned) return t64 < t128 ? 64 : 128;
  const double t256 = time(256, 256, 1.7, 1.7, 5);
  return t256 < std::min(t64, t128) ? 256 : t64 < t128 ? 64 : 128;
}

// Outputs that are larger than half of the memory side's cache (256 MiB) go past
// the caches.
bool past_caches(const ExpertArgs& a, int op, int odt) {
  const int64_t rows = op == kExpertDw ? int64_t(a.experts) * a.rows : a.slots;
  return rows * a.cols * esize(odt) > int64_t(128) << 20;
}

int run_products(ExpertArgs a, int op, int dt, int odt, bool aligned, void* stream) {
  if (std::max(a.ldr, a.ldc) > kExpertPitch) return MUON_E_SHAPE;
  a.past = op != kExpertPart && past_caches(a, op, odt);   // parts are read again
  const int tile = tile_of(a, op, dt, aligned);
  if (expert_blocks(a, op, tile, tile) > kMaxBlocks) return MUON_E_SHAPE;
  return launch_experts(a, op, dt, odt, aligned, tile, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
}

// Contractions of dw that are split: where an expert has few tiles and many rows, the
// chip would stand idle while each tile goes through all of its expert's rows.  Parts
// of `chunk` rows have fp32 results of their own that a second launch sums in order.
// A stage of 64 rows takes about 0.8 us, the second launch 6 us, a 64 x 64 tile of a
// part 0.011 us to write and read again; of the two the sum is least where both are
// alike.  us of a call that gathers, whole | split: 2 experts of 2048 rows, 256 x 128: 22 | 12
// (fp32 62 | 16); 1 of 16384, 128 x 128: 181 | 17; 8 of 2048, 512 x 256: 29 | 25 to 34, and,
// left whole by the rule, 8 of 2048, 256 x 1024: 34 | 39, 16 of 512, 256 x 256: 9.3 | 17.
struct Split {
  int64_t chunk = 0, parts = 0, ld = 0;
  size_t bytes = 0;
};
Split plan_split(int64_t slots, const muon_stack& dw) {
  Split p;
  const int64_t tiles = ceil_div(dw.rows, 64) * ceil_div(dw.cols, 64), each = slots / dw.count;
  if (tiles == 0) return p;
  const double sum = double(slots) * double(tiles);
  const int64_t chunk = ceil_div(int64_t(std::max(std::sqrt(0.88 * sum), sum / 768)) + 1, 64) * 64;
  if (0.8 * chunk / 64 + 6 + 0.011 * sum / chunk >= 0.8 * each / 64) return p;
  p.chunk = chunk;
  p.parts = slots / chunk + dw.count;
  p.ld = int64_t(round_up(size_t(dw.cols), 8));
  p.bytes = size_t(p.parts) * dw.rows * p.ld * 4;
  return p;
}

int check_gates(const float* gates, const muon_slots& s, std::vector<Span>& v, bool write) {
  if (misaligned(gates, 4)) return MUON_E_ALIGN;
  muon::add_span(v, gates, size_t(slots_of(s)) * 4, write);
  return MUON_OK;
}

// ---- embedding's gradient

struct GradPlan {
  bool few;                     // without a sort and a workspace
  int64_t chunk, chunks;
  size_t keys, counts, part, bytes;   // offsets: four arrays of n integers, counts, partial rows
};

GradPlan plan_grad(int64_t tokens, int64_t rows, int64_t cols) {
  GradPlan p;
  // short chunks where there are few waves (two a SIMD are wanted), long ones where
  // there are many: each writes up to two partial rows
  p.few = tokens && tokens <= kFewTokens && ceil_div(rows, 4) <= kMaxBlocks;
  p.chunk = 8;
  while (p.chunk < 64 && tokens * ceil_div(cols, 512) >= 4096 * p.chunk) p.chunk *= 2;
  p.chunks = ceil_div(tokens, p.chunk);
  p.keys = round_up(size_t(tokens) * 4, 16);
  p.counts = 4 * p.keys;
  p.part = round_up(p.counts + count_bytes(tokens, rows), 16);
  p.bytes = tokens && !p.few ? p.part + size_t(p.chunks) * 2 * round_up(size_t(cols), 8) * 4 : 0;
  return p;
}

}  // namespace

extern "C" {

size_t muon_expert_plan_workspace_bytes(int64_t n_tokens, int32_t k, int32_t experts) {
  return check_counts(n_tokens, k, experts) == MUON_OK ? count_bytes(n_tokens * k, experts) : 0;
}

int muon_expert_plan(const muon_ids* choice, const muon_slots* slots, void* workspace,
                     size_t workspace_bytes, void* stream) try {
  int rc;
  if ((rc = check_ids(choice)) != MUON_OK || (rc = check_slots(slots)) != MUON_OK) return rc;
  if (choice->n != slots_of(*slots)) return MUON_E_SHAPE;
  std::vector<Span> v;
  muon::add_span(v, choice->ptr, size_t(choice->n) * choice->bytes, false);
  add_span(v, *slots, true);
  if ((rc = check_workspace(v, workspace, workspace_bytes, count_bytes(choice->n, slots->experts))) != MUON_OK) return rc;
  if (conflict(v)) return MUON_E_ALIAS;
  const SortArgs a = slots_sort(choice->ptr, choice->bytes, *slots, workspace);
  return launch_sort(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_route(const muon_mat* logits, int32_t normalize, float* gates, int32_t* chosen,
               const muon_slots* slots, void* workspace, size_t workspace_bytes, void* stream) try {
  if (!logits) return MUON_E_NULL;
  int rc;
  if ((rc = check_slots(slots)) != MUON_OK || (rc = check_rows(*logits)) != MUON_OK) return rc;
  const int64_t n = slots_of(*slots);
  if (logits->rows != slots->n_tokens || logits->cols != slots->experts) return MUON_E_SHAPE;
  if (n && (!gates || !chosen)) return MUON_E_NULL;
  if (misaligned(gates, 4) || misaligned(chosen, 4)) return MUON_E_ALIGN;
  std::vector<Span> v;
  add_span(v, *logits, false);
  muon::add_span(v, gates, size_t(n) * 4, true);
  muon::add_span(v, chosen, size_t(n) * 4, true);
  add_span(v, *slots, true);
  if ((rc = check_workspace(v, workspace, workspace_bytes, count_bytes(n, slots->experts))) != MUON_OK) return rc;
  if (conflict(v)) return MUON_E_ALIAS;
  RouteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits->ptr;
  a.ld = logits->ld;
  a.gates = gates;
  a.chosen = chosen;
  a.tokens = int32_t(slots->n_tokens);
  a.experts = slots->experts;
  a.k = slots->k;
  a.normalize = normalize != 0;
  const SortArgs sort = slots_sort(chosen, 4, *slots, workspace);
  return launch_route(a, sort, logits->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_route_grad(const float* dgates, const muon_mat* logits, const float* gates,
                    const int32_t* chosen, int32_t k, int32_t normalize, const muon_mat* dlogits,
                    void* stream) try {
  if (!logits || !dlogits) return MUON_E_NULL;
  int rc;
  if ((rc = check_rows(*logits)) != MUON_OK || (rc = check_rows(*dlogits)) != MUON_OK ||
      (rc = check_counts(logits->rows, k, logits->cols)) != MUON_OK)
    return rc;
  if (dlogits->rows != logits->rows || dlogits->cols != logits->cols) return MUON_E_SHAPE;
  if (logits->rows == 0) return MUON_OK;
  if (!dgates || !gates || !chosen) return MUON_E_NULL;
  if (misaligned(dgates, 4) || misaligned(gates, 4) || misaligned(chosen, 4)) return MUON_E_ALIGN;
  std::vector<Span> v;
  const size_t n = size_t(logits->rows) * k * 4;
  muon::add_span(v, dgates, n, false);
  muon::add_span(v, gates, n, false);
  muon::add_span(v, chosen, n, false);
  add_span(v, *logits, false);
  add_span(v, *dlogits, true);
  if (conflict(v)) return MUON_E_ALIAS;
  RouteGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dgates = dgates;
  a.logits = logits->ptr;
  a.gates = gates;
  a.chosen = chosen;
  a.dlogits = dlogits->ptr;
  a.ld = logits->ld;
  a.ldd = dlogits->ld;
  a.tokens = int32_t(logits->rows);
  a.experts = int32_t(logits->cols);
  a.k = k;
  a.normalize = normalize != 0;
  return launch_route_grad(a, logits->dtype, dlogits->dtype, static_cast<hipStream_t>(stream)) == hipSuccess
             ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

// fwd and dx: rows of x (dy) times the experts' matrices.
static int row_products(int op, const muon_mat* x, const muon_stack* w, const muon_slots* slots,
                        bool gather, const muon_mat* out, void* stream) {
  if (!x || !w || !out) return MUON_E_NULL;
  int rc;
  std::vector<Span> v;
  if ((rc = check_products(*x, w->dtype, slots, v)) != MUON_OK || (rc = check_stack(*w)) != MUON_OK ||
      (rc = check_rows(*out)) != MUON_OK)
    return rc;
  const int64_t n = slots_of(*slots), depth = op == kExpertFwd ? w->cols : w->rows;
  if (w->count != slots->experts || x->rows != (gather ? slots->n_tokens : n) || x->cols != depth ||
      out->rows != n || out->cols != (op == kExpertFwd ? w->rows : w->cols) || (gather && !spans(*x)))
    return MUON_E_SHAPE;
  add_span(v, *w, false);
  add_span(v, *out, true);
  if (conflict(v)) return MUON_E_ALIAS;
  if (n == 0 || out->cols == 0) return MUON_OK;
  ExpertArgs a;
  std::memset(&a, 0, sizeof(a));
  a.r = x->ptr;
  a.c = w->ptr;
  a.out = out->ptr;
  a.offsets = slots->offsets;
  a.tokens = gather ? slots->tokens : nullptr;
  a.ldr = x->ld;
  a.ldc = w->ld;
  a.ldo = out->ld;
  a.wstride = w->count > 1 ? w->stride : 0;
  a.experts = slots->experts;
  a.slots = int32_t(n);
  a.cols = int32_t(out->cols);
  a.depth = int32_t(depth);
  a.src = int32_t(x->rows);
  const bool aligned = w->dtype == MUON_BF16 && pieces(x->ptr, x->ld, x->cols) &&
                       pieces(w->ptr, w->ld, w->cols) && a.wstride % 8 == 0;
  return run_products(a, op, w->dtype, out->dtype, aligned, stream);
}

int muon_expert_linear(const muon_mat* x, const muon_stack* w, const muon_slots* slots,
                       int32_t gather, const muon_mat* out, void* stream) try {
  return row_products(kExpertFwd, x, w, slots, gather != 0, out, stream);
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_expert_linear_dx(const muon_mat* dy, const muon_stack* w, const muon_slots* slots,
                          const muon_mat* dx, void* stream) try {
  return row_products(kExpertDx, dy, w, slots, false, dx, stream);
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

size_t muon_expert_linear_dw_workspace_bytes(int64_t slots, const muon_stack* dw) {
  if (!dw || slots < 0 || slots > MUON_MAX_SLOTS || dw->count < 1 || dw->count > MUON_MAX_EXPERTS || dw->rows < 0 ||
      dw->rows > kMaxCols || dw->cols < 0 || dw->cols > kMaxCols)
    return 0;
  return plan_split(slots, *dw).bytes;
}

int muon_expert_linear_dw(const muon_mat* dy, const muon_mat* x, const muon_slots* slots,
                          int32_t gather, int32_t accumulate, const muon_stack* dw,
                          void* workspace, size_t workspace_bytes, void* stream) try {
  if (!dy || !x || !dw) return MUON_E_NULL;
  int rc;
  std::vector<Span> v;
  if ((rc = check_products(*dy, x->dtype, slots, v)) != MUON_OK || (rc = check_rows(*x)) != MUON_OK ||
      (rc = check_stack(*dw)) != MUON_OK)
    return rc;
  const int64_t n = slots_of(*slots);
  if (dw->count != slots->experts || dy->rows != n || x->rows != (gather ? slots->n_tokens : n) ||
      dw->rows != dy->cols || dw->cols != x->cols || (gather && !spans(*x)))
    return MUON_E_SHAPE;
  add_span(v, *x, false);
  add_span(v, *dw, true);
  const Split split = plan_split(n, *dw);
  if ((rc = check_workspace(v, workspace, workspace_bytes, split.bytes)) != MUON_OK) return rc;
  if (conflict(v)) return MUON_E_ALIAS;
  if (dw->rows == 0 || dw->cols == 0) return MUON_OK;
  ExpertArgs a;
  std::memset(&a, 0, sizeof(a));
  a.r = dy->ptr;
  a.c = x->ptr;
  a.out = dw->ptr;
  a.offsets = slots->offsets;
  a.tokens = gather ? slots->tokens : nullptr;
  a.ldr = dy->ld;
  a.ldc = x->ld;
  a.ldo = dw->ld;
  a.ostride = dw->count > 1 ? dw->stride : 0;
  a.experts = slots->experts;
  a.slots = int32_t(n);
  a.rows = int32_t(dw->rows);
  a.cols = int32_t(dw->cols);
  a.src = int32_t(x->rows);
  a.accumulate = accumulate != 0;
  const bool aligned = x->dtype == MUON_BF16 && pieces(dy->ptr, dy->ld, dy->cols) && pieces(x->ptr, x->ld, x->cols);
  if (!split.chunk) return run_products(a, kExpertDw, x->dtype, dw->dtype, aligned, stream);
  a.out = workspace;
  a.ldo = split.ld;
  a.ostride = dw->rows * split.ld;
  a.chunk = int32_t(split.chunk);
  a.parts = int32_t(split.parts);
  if ((rc = run_products(a, kExpertPart, x->dtype, MUON_F32, aligned, stream)) != MUON_OK) return rc;
  return launch_experts_join(a, dw->ptr, dw->ld, dw->count > 1 ? dw->stride : 0, dw->dtype,
                             static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_expert_combine(const muon_mat* y, const float* gates, const muon_slots* slots,
                        const muon_mat* out, void* stream) try {
  if (!y || !out) return MUON_E_NULL;
  int rc;
  if ((rc = check_slots(slots)) != MUON_OK || (rc = check_rows(*y)) != MUON_OK || (rc = check_rows(*out)) != MUON_OK) return rc;
  if (y->rows != slots_of(*slots) || out->rows != slots->n_tokens || out->cols != y->cols) return MUON_E_SHAPE;
  std::vector<Span> v;
  add_span(v, *slots, false);
  add_span(v, *y, false);
  add_span(v, *out, true);
  if ((rc = check_gates(gates, *slots, v, false)) != MUON_OK) return rc;
  if (conflict(v)) return MUON_E_ALIAS;
  if (out->rows == 0 || out->cols == 0) return MUON_OK;
  if (ceil_div(out->rows * ceil_div(out->cols, 8), 256) > kMaxBlocks) return MUON_E_SHAPE;
  CombineArgs a;
  std::memset(&a, 0, sizeof(a));
  a.y = y->ptr;
  a.gates = gates;
  a.place = slots->place;
  a.out = out->ptr;
  a.ldy = y->ld;
  a.ldo = out->ld;
  a.tokens = int32_t(out->rows);
  a.k = slots->k;
  a.slots = int32_t(y->rows);
  a.cols = int32_t(y->cols);
  return launch_combine(a, y->dtype, out->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_expert_combine_grad(const muon_mat* dout, const muon_mat* y, const float* gates,
                             const muon_slots* slots, const muon_mat* dy, float* dgates,
                             void* stream) try {
  if (!dout || (dgates && !y)) return MUON_E_NULL;
  int rc;
  if ((rc = check_slots(slots)) != MUON_OK || (rc = check_rows(*dout)) != MUON_OK) return rc;
  const int64_t n = slots_of(*slots);
  if (dout->rows != slots->n_tokens) return MUON_E_SHAPE;
  std::vector<Span> v;
  add_span(v, *slots, false);
  add_span(v, *dout, false);
  if ((rc = check_gates(gates, *slots, v, false)) != MUON_OK || (rc = check_gates(dgates, *slots, v, true)) != MUON_OK) return rc;
  for (const muon_mat* m : {dgates ? y : nullptr, dy}) {
    if (!m) continue;
    if ((rc = check_rows(*m)) != MUON_OK) return rc;
    if (m->dtype != dout->dtype) return MUON_E_DTYPE;
    if (m->rows != n || m->cols != dout->cols) return MUON_E_SHAPE;
    add_span(v, *m, m == dy);
  }
  if (conflict(v)) return MUON_E_ALIAS;
  if (n == 0 || (!dy && !dgates)) return MUON_OK;
  CombineArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dout = dout->ptr;
  a.y = dgates ? y->ptr : nullptr;
  a.gates = gates;
  a.place = slots->place;
  a.rows = slots->tokens;
  a.out = dy && dout->cols ? dy->ptr : nullptr;
  a.dgates = dgates;
  a.ldd = dout->ld;
  a.ldy = dgates ? y->ld : 0;
  a.ldo = dy ? dy->ld : 0;
  a.tokens = int32_t(dout->rows);
  a.k = slots->k;
  a.slots = int32_t(n);
  a.cols = int32_t(dout->cols);
  return launch_combine_grad(a, dout->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

int muon_expert_gather(const muon_mat* x, const muon_slots* slots, const muon_mat* out, void* stream) {
  if (!out) return MUON_E_NULL;
  return muon_expert_combine_grad(x, nullptr, nullptr, slots, out, nullptr, stream);
}

int muon_embedding(const muon_ids* ids, const muon_mat* w, float scale, const muon_mat* out,
                   void* stream) try {
  if (!w || !out) return MUON_E_NULL;
  int rc;
  if ((rc = check_ids(ids)) != MUON_OK || (rc = check_rows(*w)) != MUON_OK || (rc = check_rows(*out)) != MUON_OK) return rc;
  if (w->dtype != out->dtype) return MUON_E_DTYPE;
  if (!std::isfinite(scale)) return MUON_E_HPARAM;
  if (out->rows != ids->n || out->cols != w->cols) return MUON_E_SHAPE;
  std::vector<Span> v;
  muon::add_span(v, ids->ptr, size_t(ids->n) * ids->bytes, false);
  add_span(v, *w, false);
  add_span(v, *out, true);
  if (conflict(v)) return MUON_E_ALIAS;
  if (out->rows == 0 || out->cols == 0) return MUON_OK;
  if (ceil_div(out->rows * ceil_div(out->cols, 8), 1024) > kMaxBlocks) return MUON_E_SHAPE;
  EmbedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.ids = ids->ptr;
  a.w = w->ptr;
  a.out = out->ptr;
  a.ldw = w->ld;
  a.ldo = out->ld;
  a.rows = w->rows;
  a.scale = scale;
  a.id_bytes = ids->bytes;
  a.tokens = int32_t(ids->n);
  a.cols = int32_t(w->cols);
  return launch_embedding(a, w->dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

size_t muon_embedding_grad_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols) {
  if (tokens < 0 || tokens > MUON_MAX_SLOTS || rows < 0 || rows >= kMaxRows || cols < 0 || cols > kMaxCols) return 0;
  return plan_grad(tokens, rows, cols).bytes;
}

int muon_embedding_grad(const muon_mat* dy, const muon_ids* ids, float scale, int32_t accumulate,
                        const muon_mat* dw, void* workspace, size_t workspace_bytes, void* stream) try {
  if (!dy || !dw) return MUON_E_NULL;
  int rc;
  if ((rc = check_ids(ids)) != MUON_OK || (rc = check_rows(*dy)) != MUON_OK || (rc = check_rows(*dw)) != MUON_OK) return rc;
  if (!std::isfinite(scale)) return MUON_E_HPARAM;
  if (dy->rows != ids->n || dw->cols != dy->cols || dw->rows >= kMaxRows) return MUON_E_SHAPE;
  const GradPlan p = plan_grad(ids->n, dw->rows, dw->cols);
  std::vector<Span> v;
  muon::add_span(v, ids->ptr, size_t(ids->n) * ids->bytes, false);
  add_span(v, *dy, false);
  add_span(v, *dw, true);
  if ((rc = check_workspace(v, workspace, workspace_bytes, p.bytes)) != MUON_OK) return rc;
  if (conflict(v)) return MUON_E_ALIAS;
  if (dw->rows == 0 || dw->cols == 0) return MUON_OK;
  const int64_t units = p.chunks * ceil_div(dw->cols, 512) + ceil_div(dw->rows, kEmbedZeroRows);
  if (ceil_div(units, 4) > kMaxBlocks || p.chunks * ceil_div(dw->cols, 256) > kMaxBlocks) return MUON_E_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  EmbedGradArgs a;
  std::memset(&a, 0, sizeof(a));
  if (ids->n && !p.few) {
    SortArgs sort;
    std::memset(&sort, 0, sizeof(sort));
    sort.ids = ids->ptr;
    sort.id_bytes = ids->bytes;
    sort.n = int32_t(ids->n);
    sort.limit = int32_t(dw->rows);
    sort.passes = sort_passes(dw->rows);
    for (int i = 0; i < 2; ++i) {
      sort.key[i] = reinterpret_cast<int32_t*>(ws + (2 * i) * p.keys);
      sort.pos[i] = reinterpret_cast<int32_t*>(ws + (2 * i + 1) * p.keys);
    }
    sort.counts = reinterpret_cast<int32_t*>(ws + p.counts);
    if (launch_sort(sort, s) != hipSuccess) return MUON_E_HIP;
    a.key = sort.key[(sort.passes - 1) & 1];
    a.pos = sort.pos[(sort.passes - 1) & 1];
    a.part = reinterpret_cast<float*>(ws + p.part);
  }
  a.dy = dy->ptr;
  a.dw = dw->ptr;
  a.ldy = dy->ld;
  a.ldw = dw->ld;
  a.scale = scale;
  a.tokens = int32_t(ids->n);
  a.rows = int32_t(dw->rows);
  a.cols = int32_t(dw->cols);
  a.accumulate = accumulate != 0;
  a.chunk = int32_t(p.chunk);
  a.chunks = int32_t(p.chunks);
  a.ldp = int32_t(round_up(size_t(dw->cols), 8));
  const hipError_t e = p.few ? launch_embedding_few(a, ids->ptr, ids->bytes, dy->dtype, dw->dtype, s)
                           : launch_embedding_grad(a, dy->dtype, dw->dtype, s);
  return e == hipSuccess ? MUON_OK : MUON_E_HIP;
} catch (...) {   // an allocation of the host's failed
  return MUON_E_HIP;
}

}  // extern "C"
