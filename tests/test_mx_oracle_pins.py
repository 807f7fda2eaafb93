"""Pins of the 4-bit oracle: published generator outputs, hand-worked blocks,
and statistics that a slip in rounding or scaling would break."""
import math

import numpy as np
import pytest

from oracle import mx_oracle as mx


def test_philox_published_outputs():
    # known answers of Philox 4x32 with ten rounds
    zero = mx.philox(np.zeros((1, 4), np.uint64), 0)[0]
    assert [hex(v) for v in zero] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = mx.philox(np.full((1, 4), 0xFFFFFFFF, np.uint64), (1 << 64) - 1)[0]
    assert [hex(v) for v in ones] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


def test_hand_worked_block():
    x = np.zeros((1, 32))
    x[0, :10] = [6, -5, 5.1, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2500001]
    code, sign, byte = mx.quantize(x)
    assert byte[0, 0] == 127
    # ties: 5 -> 4, 3.5 -> 4, 2.5 -> 2, 1.75 -> 2, 1.25 -> 1, 0.75 -> 1, 0.25 -> 0
    assert code[0, 0, :10].tolist() == [7, 6, 7, 6, 4, 4, 2, 2, 0, 1]
    assert sign[0, 0, 1] and sign[0, 0, 9] and not sign[0, 0, 0]
    v = mx.values(code, sign, byte, 10)
    assert v.tolist() == [[6, -4, 6, 4, 2, 2, 1, 1, 0, -0.5]]


@pytest.mark.parametrize("top,e", [(6.0, 0), (6.0000005, 1), (3.0, -1), (3.1, 0), (1.5, -2), (12.0, 1),
                                   (1e-45, -127), (0.0, -127), (2.0 ** -126, -127)])
def test_scale_is_the_smallest_that_holds_the_block(top, e):
    x = np.zeros((1, 32))
    x[0, 5] = -top
    assert mx.quantize(x)[2][0, 0] == e + 127


def test_non_finite_blocks_and_short_rows():
    x = np.zeros((2, 40))
    x[0, 33] = math.inf
    x[1, 2] = math.nan
    v = mx.rounded(x)
    assert np.isnan(v[0, 32:]).all() and np.isfinite(v[0, :32]).all()
    assert np.isnan(v[1, :32]).all() and np.isfinite(v[1, 32:]).all()
    assert v.shape == (2, 40)


def test_stochastic_rounding_is_between_neighbours_and_unbiased():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 64))
    near = mx.rounded(x)
    tot = np.zeros_like(x)
    n = 64
    for s in range(n):
        v = mx.rounded(x, seed=s)
        tot += v
    scale = np.repeat(np.exp2(mx.quantize(x)[2] - 127.0), 32, 1)
    # one step is at most 2 scales; the mean of n draws has a deviation of at
    # most half a step / sqrt(n), six of them over 4096 elements; 1/512 of a
    # step for the random byte
    assert np.max(np.abs(tot / n - x) / scale) < 6 * 1.0 / math.sqrt(n) + 2 / 512
    assert abs(np.mean((tot / n - x) / scale)) < 6 * 1.0 / math.sqrt(n * x.size) + 2 / 512
    assert np.max(np.abs(near - x) / scale) <= 1.0


def test_quantisation_is_idempotent():
    x = np.random.default_rng(4).standard_normal((8, 96)) * 10.0 ** np.arange(-4, 4)[:, None]
    v = mx.rounded(x)
    assert np.array_equal(mx.rounded(v), v)


def test_dropout_rate_scale_and_place():
    x = np.ones((128, 333), np.float32)
    y = mx.dropout(x, 0.25, 7)
    assert set(np.unique(y)) == {np.float32(0), np.float32(65536) / np.float32(49152)}
    kept = np.mean(y > 0)
    assert abs(kept - 0.75) < 6 * math.sqrt(0.75 * 0.25 / x.size)
    # a function of the place alone: a wider matrix has the same mask in front
    wide = mx.dropout(np.ones((128, 400), np.float32), 0.25, 7)
    assert np.array_equal(wide[:, :333], y)
    assert not np.array_equal(mx.dropout(x, 0.25, 8), y)
    assert not np.array_equal(mx.dropout(x, 0.25, 7, index=1), y)
