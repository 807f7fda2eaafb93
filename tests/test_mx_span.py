"""Which memory of a call's arguments counts as shared: the host code's rule
against sets of bytes."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "orthogonalising_matrix_optimizer_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "muon_span.h"
using namespace muon;
// lines of "start rows pitch width write" for two spans -> share conflict
int main() {
  long a[5], b[5];
  auto span = [](const long* v) {
    return Span{uintptr_t(v[0]), uintptr_t(v[0] + (v[1] - 1) * v[2] + v[3]), size_t(v[2]), size_t(v[3]), v[4] != 0};
  };
  while (scanf("%ld %ld %ld %ld %ld %ld %ld %ld %ld %ld", a, a + 1, a + 2, a + 3, a + 4, b, b + 1, b + 2, b + 3, b + 4) == 10) {
    std::vector<Span> v = {span(a), span(b)};
    printf("%d %d\n", share(span(a), span(b)), conflict(v));
  }
  return 0;
}
"""

# three spans a line -> conflict
PROGRAM3 = r"""
#include <stdio.h>
#include "muon_span.h"
using namespace muon;
int main() {
  long s[5];
  std::vector<Span> v;
  while (scanf("%ld %ld %ld %ld %ld", s, s + 1, s + 2, s + 3, s + 4) == 5) {
    v.push_back({uintptr_t(s[0]), uintptr_t(s[0] + (s[1] - 1) * s[2] + s[3]), size_t(s[2]), size_t(s[3]), s[4] != 0});
    if (v.size() == 3) {
      printf("%d\n", conflict(v));
      v.clear();
    }
  }
  return 0;
}
"""


def _bytes(s):
    start, rows, pitch, width, _ = s
    return {start + i * pitch + j for i in range(rows) for j in range(width)}


def _program(d, source):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    (d / "span.cpp").write_text(source)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "span.cpp"), "-o", str(d / "span")], check=True)

    def ask(groups):
        text = "\n".join(" ".join(str(v) for span in g for v in span) for g in groups)
        out = subprocess.run([str(d / "span")], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(groups)
        return got
    return ask


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    return _program(tmp_path_factory.mktemp("span"), PROGRAM)


@pytest.fixture(scope="module")
def answers3(tmp_path_factory):
    ask = _program(tmp_path_factory.mktemp("span3"), PROGRAM3)
    return lambda groups: [c for c, in ask(groups)]


def _check(pairs, got):
    for (a, b), (share, conflict) in zip(pairs, got):
        real = bool(_bytes(a) & _bytes(b))
        assert share == real, (a, b)
        assert conflict == (share and (a[4] or b[4])), (a, b)


def _slice(rng, pitch, rows):
    """A slice of a buffer of `rows` rows of `pitch` bytes, as the callers describe it."""
    r0, c0 = rng.randrange(rows), rng.randrange(pitch)
    n, w = rng.randint(1, rows - r0), rng.randint(1, pitch - c0)
    every = rng.choice([1, 1, 2, 3])
    n = -(-n // every)
    # a single row is described by its width alone
    return (1000 + r0 * pitch + c0, n, w if n == 1 else pitch * every, w, rng.randrange(2))


def test_column_slices_of_one_buffer(answers):
    """Slices of one buffer, a single row of it among them, share memory exactly
    where their bytes do."""
    rng = random.Random(1)
    pairs = []
    while len(pairs) < 20000:
        pitch, rows = rng.randint(1, 12), rng.randint(1, 9)
        a, b = _slice(rng, pitch, rows), _slice(rng, pitch, rows)
        pairs.append((a, b))
    _check(pairs, answers(pairs))


def test_strided_rows_beside_a_column_slice(answers):
    pairs = [((1000, 5, 200, 60, 1), (1060, 9, 100, 40, 1)),     # buf[::2, :60], buf[:, 60:]
             ((1000, 5, 200, 61, 1), (1060, 9, 100, 40, 1)),     # ... and one column too many
             ((1100, 1, 30, 30, 1), (1030, 17, 100, 30, 1)),     # buf[1:2, :30], buf[:17, 30:60]
             ((1030, 17, 100, 30, 1), (1100, 1, 30, 30, 1)),
             ((1100, 1, 31, 31, 1), (1030, 17, 100, 30, 1)),
             ((1100, 1, 30, 30, 0), (1100, 1, 30, 30, 0))]
    assert [s for s, _ in answers(pairs)] == [0, 1, 0, 0, 1, 1]
    _check(pairs, answers(pairs))


def test_spans_of_any_pitch(answers):
    rng = random.Random(2)
    pairs = []
    for _ in range(40000):
        a, b = ((1000 + rng.randrange(60), rng.randint(1, 6), p, rng.randint(1, p), rng.randrange(2))
                for p in (rng.randint(1, 14), rng.randint(1, 14)))
        pairs.append((a, b))
    _check(pairs, answers(pairs))


def test_two_operands_that_begin_and_end_alike(answers3):
    """Of two inputs with the same first and last byte one may have gaps that
    the other has not: an output in such a gap overlaps the other."""
    strided, whole, gap = (1000, 3, 100, 50, 0), (1000, 1, 250, 250, 0), (1060, 1, 10, 10, 1)
    assert answers3([(strided, whole, gap), (whole, strided, gap), (strided, strided, gap)]) == [1, 1, 0]
