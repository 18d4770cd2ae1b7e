"""Plain references of the dropout and adapter operators, used by the tests
only: numpy unsigned integers for the generator, numpy fp32 for what the
operators define in fp32 steps, float64 for sums.  Shares no code with the
library."""
from __future__ import annotations

import numpy as np


def philox4x32(counter, key, rounds):
    """Philox4x32 ("Parallel random numbers: as easy as 1, 2, 3", SC 2011) of
    counter words [4] (arrays of one shape) and key words [2]."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return int(np.rint(float(np.float32(p)) * 65536.0))


def factor(p: float) -> np.float32:
    return np.float32(65536.0 / (65536 - threshold(p)))


def numbers(rows, cols, seed, offset, first_row=0):
    """The 16-bit numbers [rows, cols] of rows first_row .. of a tensor with
    `cols` columns."""
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    e = np.uint64(first_row) * np.uint64(cols // 8) + np.arange(rows * cols // 8, dtype=np.uint64)
    full = lambda v: np.full(e.shape, v, dtype=np.uint64)
    w = philox4x32([e & np.uint64(0xFFFFFFFF), e >> np.uint64(32), full(offset & 0xFFFFFFFF),
                    full(offset >> 32)], (seed & 0xFFFFFFFF, seed >> 32), 7)
    words = np.stack(w, 1).astype("<u4")
    return words.view("<u2").reshape(rows, cols)


def keep_mask(rows, cols, p, seed, offset, first_row=0):
    return numbers(rows, cols, seed, offset, first_row) >= threshold(p)


def bf16_round(v32: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, to nearest even; NaN -> 0x7FC0."""
    u = np.ascontiguousarray(v32, dtype=np.float32).view(np.uint32)
    r = ((u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16))
    return np.where(np.isnan(v32), np.uint32(0x7FC0), r).astype(np.uint16)


def dropout(x32: np.ndarray, mask: np.ndarray, f: np.float32, residual32=None) -> np.ndarray:
    """fp32 product and sum, each rounded: residual + (mask ? x * f : +0)."""
    with np.errstate(all="ignore"):
        t = np.where(mask, x32.astype(np.float32) * f, np.float32(0))
        return t if residual32 is None else residual32.astype(np.float32) + t


def adapter_forward(x, a, b, alpha, ids, base=None, mask=None, f=1.0):
    """float64 (y, h); ids outside [0, count) mark rows without an adapter."""
    rows, count = x.shape[0], a.shape[0]
    xd = x if mask is None else np.where(mask, x, 0.0)
    y = np.zeros((rows, b.shape[1])) if base is None else base.astype(np.float64).copy()
    h = np.zeros((rows, a.shape[1]))
    for i in range(count):
        at = np.nonzero(ids == i)[0]
        if at.size:
            h[at] = alpha[i] * f * (xd[at] @ a[i].T)
            y[at] += h[at] @ b[i].T
    return y, h


def adapter_backward(x, a, b, alpha, ids, dy, h, base=None, mask=None, f=1.0):
    """float64 (dx, da, db, g)."""
    rows, count = x.shape[0], a.shape[0]
    keep = np.ones(x.shape) if mask is None else mask.astype(np.float64)
    xd = np.where(keep > 0, x, 0.0) * f
    dx = np.zeros(x.shape) if base is None else base.astype(np.float64).copy()
    da, db, g = np.zeros(a.shape), np.zeros(b.shape), np.zeros((rows, a.shape[1]))
    for i in range(count):
        at = np.nonzero(ids == i)[0]
        if at.size:
            g[at] = alpha[i] * (dy[at] @ b[i])
            dx[at] += f * keep[at] * (g[at] @ a[i])
            da[i] = g[at].T @ xd[at]
            db[i] = dy[at].T @ h[at]
    return dx, da, db, g
