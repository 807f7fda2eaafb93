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


def _bytes(s):
    start, rows, pitch, width, _ = s
    return {start + i * pitch + j for i in range(rows) for j in range(width)}


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("span")
    (d / "span.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "span.cpp"), "-o", str(d / "span")], check=True)

    def ask(pairs):
        text = "\n".join(" ".join(map(str, (*a, *b))) for a, b in pairs)
        out = subprocess.run([str(d / "span")], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(pairs)
        return got
    return ask


def _check(pairs, got, exact):
    for (a, b), (share, conflict) in zip(pairs, got):
        real = bool(_bytes(a) & _bytes(b))
        assert share >= real, (a, b)
        assert conflict == (share and (a[4] or b[4])), (a, b)
        if exact:
            assert share == real, (a, b)


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
        # every second row against every third is looked at below
        if a[1] == 1 or b[1] == 1 or a[2] == b[2]:
            pairs.append((a, b))
    _check(pairs, answers(pairs), exact=True)


def test_strided_rows_beside_a_column_slice(answers):
    pairs = [((1000, 5, 200, 60, 1), (1060, 9, 100, 40, 1)),     # buf[::2, :60], buf[:, 60:]
             ((1000, 5, 200, 61, 1), (1060, 9, 100, 40, 1)),     # ... and one column too many
             ((1100, 1, 30, 30, 1), (1030, 17, 100, 30, 1)),     # buf[1:2, :30], buf[:17, 30:60]
             ((1030, 17, 100, 30, 1), (1100, 1, 30, 30, 1)),
             ((1100, 1, 31, 31, 1), (1030, 17, 100, 30, 1)),
             ((1100, 1, 30, 30, 0), (1100, 1, 30, 30, 0))]
    assert [s for s, _ in answers(pairs)] == [0, 1, 0, 0, 1, 1]
    _check(pairs, answers(pairs), exact=True)


def test_no_shared_byte_is_missed(answers):
    rng = random.Random(2)
    pairs = []
    for _ in range(40000):
        a, b = ((1000 + rng.randrange(60), rng.randint(1, 6), p, rng.randint(1, p), rng.randrange(2))
                for p in (rng.randint(1, 14), rng.randint(1, 14)))
        pairs.append((a, b))
    _check(pairs, answers(pairs), exact=False)
