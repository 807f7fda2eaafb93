// Memory that a call reads and writes, and whether its arguments may share it
// (host only).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>
#include <vector>

namespace muon {

// Memory that a call reads or writes: `width` bytes in every `pitch` from lo
// on, up to hi.
struct Span {
  uintptr_t lo, hi;
  size_t pitch, width;
  bool write;
};

// Whether the bytes lo .. hi - 1 meet a row of the span.
inline bool meets(const Span& s, uintptr_t lo, uintptr_t hi) {
  if (lo >= s.hi || s.lo >= hi) return false;
  if (lo <= s.lo) return true;
  const size_t in = (lo - s.lo) % s.pitch;                  // place in the row's pitch
  if (in < s.width) return true;
  const uintptr_t next = lo - in + s.pitch;                 // the next row's start
  return next < s.hi && next < hi;
}

// Whether two spans share a byte.  A single row is described by its width alone,
// every n-th row of a buffer by n pitches.
inline bool share(const Span& a, const Span& b) {
  if (b.lo >= a.hi || a.lo >= b.hi) return false;
  auto run = [](const Span& s) { return s.hi - s.lo == s.width || s.pitch == s.width; };
  if (run(a)) return meets(b, a.lo, a.hi);
  if (run(b)) return meets(a, b.lo, b.hi);
  // rows' starts differ by the spans' distance and multiples of the common pitch
  const size_t pitch = std::gcd(a.pitch, b.pitch);
  const Span &first = a.lo < b.lo ? a : b, &second = a.lo < b.lo ? b : a;
  const size_t d = (second.lo - first.lo) % pitch;
  if (d >= first.width && d + second.width <= pitch) return false;
  // else the rows themselves, of the span with fewer of them, where the other is
  const Span &few = a.pitch > b.pitch ? a : b, &many = a.pitch > b.pitch ? b : a;
  uintptr_t row = few.lo;
  if (many.lo > row) row += (many.lo - row) / few.pitch * few.pitch;
  for (; row < few.hi && row < many.hi; row += few.pitch)
    if (meets(many, row, row + few.width)) return true;
  return false;
}

// Whether something written is also read or written through another argument.
inline bool conflict(std::vector<Span>& v) {
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
    auto same = [&](const Span& o) {
      return o.lo == s.lo && o.hi == s.hi && o.pitch == s.pitch && o.width == s.width;
    };
    if (!(kept && !s.write && same(open[kept - 1]) && !open[kept - 1].write)) open.push_back(s);
  }
  return false;
}

}  // namespace muon
