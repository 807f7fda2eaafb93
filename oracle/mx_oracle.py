"""Plain CPU oracle for the 4-bit operators and dropout (TEST INFRASTRUCTURE).

Written from the number format (blocks of 32, power-of-two scale, the eight
magnitudes of a 4-bit element) and from the published definition of the
Philox 4x32 generator (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
as easy as 1, 2, 3", 2011), in float64; shares no code with the product.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_BYTE = 255
DROP, ROUND, ROUND_T = (int.from_bytes(s, "big") for s in (b"DROP", b"SR40", b"SR41"))


def philox(counter, seed: int) -> np.ndarray:
    """Four 32-bit words for each counter (array [..., 4])."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def randoms(rows: int, cols: int, bits: int, tag: int, index: int, seed: int) -> np.ndarray:
    """Random integers of `bits` bits per element of a rows x cols matrix."""
    per = 128 // bits
    groups = -(-cols // per)
    ctr = np.zeros((rows, groups, 4), np.uint64)
    ctr[..., 0] = np.arange(groups)
    ctr[..., 1] = np.arange(rows)[:, None]
    ctr[..., 2] = tag
    ctr[..., 3] = index
    w = philox(ctr, seed)
    return w.reshape(rows, groups * 4).view({8: np.uint8, 16: np.uint16}[bits])[:, :cols].astype(np.int64)


def quantize(x: np.ndarray, r8: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(code magnitude 0..7, sign bit, scale byte) of each element / block of x,
    blocks of 32 along the rows; shapes [rows, blocks, 32] and [rows, blocks]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :cols] = x
    v = v.reshape(rows, nb, 32)
    r = np.zeros((rows, nb * 32))
    if r8 is not None:
        r[:, :cols] = r8
    r = r.reshape(v.shape)
    code = np.zeros(v.shape, np.int64)
    byte = np.zeros((rows, nb), np.int64)
    for i in range(rows):
        for b in range(nb):
            blk = v[i, b]
            top = np.max(np.abs(blk)) if np.all(np.isfinite(blk)) else math.inf
            if not math.isfinite(top):
                byte[i, b] = NAN_BYTE
                continue
            e = -127
            if top > 0:
                e = max(-127, math.frexp(top)[1] - 4)
                while top > 6.0 * 2.0 ** e:
                    e += 1
            byte[i, b] = e + 127
            a = np.abs(blk) * 2.0 ** -e
            if r8 is None:
                d = np.abs(a[:, None] - GRID[None, :])
                near = d == d.min(1, keepdims=True)
                # ties to the even code
                pick = np.where(near, np.where(np.arange(8) % 2 == 0, 0, 1), 9)
                code[i, b] = np.argmin(pick, 1)
            else:
                low = np.searchsorted(GRID, a, side="right") - 1
                high = np.minimum(low + 1, 7)
                step = np.where(high > low, GRID[high] - GRID[low], 1.0)
                code[i, b] = low + ((a - GRID[low]) / step * 256 > r[i, b] + 0.5)
    return code, np.signbit(v), byte


def values(code, sign, byte, cols: int) -> np.ndarray:
    """float64 values of codes and scales (2^128 and beyond are kept finite)."""
    scale = np.where(byte == NAN_BYTE, np.nan, np.exp2(byte.astype(np.float64) - 127))
    v = np.where(sign, -1.0, 1.0) * GRID[code] * scale[..., None]
    return v.reshape(v.shape[0], -1)[:, :cols] if v.size else np.zeros((v.shape[0], cols))


def rounded(x, seed: Optional[int] = None, transpose: bool = False, index: int = 0) -> np.ndarray:
    """Values of x (or of its transpose) after quantisation along the rows."""
    x = np.asarray(x, np.float64)
    x = x.T if transpose else x
    r8 = None
    if seed is not None:
        r8 = randoms(x.shape[0], x.shape[1], 8, ROUND_T if transpose else ROUND, index, seed)
    return values(*quantize(x, r8), x.shape[1])


def dropout(x: np.ndarray, p: float, seed: int, index: int = 0) -> np.ndarray:
    """float32 of x with its dropped elements zero and the others scaled, the
    product rounded once to fp32 (a bf16 result rounds that again)."""
    t = math.floor(p * 65536 + 0.5)
    keep = randoms(x.shape[0], x.shape[1], 16, DROP, index, seed) >= t
    scale = np.float32(65536) / np.float32(65536 - t)
    return np.where(keep, np.asarray(x, np.float32) * scale, np.float32(0))


def storage(code, sign, byte):
    """Codes and scale bytes in the tiled storage order (muon_mx layout):
    (codes uint8 [k tiles, row tiles, 1024], scales uint8 [k tiles, row tiles
    of 64, 256], scales' valid mask)."""
    rows, nb = byte.shape
    rt, kt, st = -(-rows // 16), -(-nb // 4), -(-rows // 64)
    codes = np.zeros((kt, rt, 4, 16, 16), np.uint8)
    scales = np.zeros((kt, st, 4, 16, 4), np.uint8)
    valid = np.zeros(scales.shape, bool)
    nib = (code + 8 * sign).astype(np.uint8)
    nib[byte == NAN_BYTE] = 0
    packed = nib[..., 0::2] | (nib[..., 1::2] << 4)
    for r in range(rows):
        for b in range(nb):
            codes[b // 4, r // 16, b % 4, r % 16] = packed[r, b]
            scales[b // 4, r // 64, b % 4, r % 16, r % 64 // 16] = byte[r, b]
            valid[b // 4, r // 64, b % 4, r % 16, r % 64 // 16] = True
    return codes.reshape(kt, rt, 1024), scales.reshape(kt, st, 256), valid.reshape(kt, st, 256)
