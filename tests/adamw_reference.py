"""Plain reference of the AdamW step, used by the tests only: numpy fp32 where
the definition rounds every operation, float64 for the update of the
parameters, integers for the codes.  Shares no code with the library."""
from __future__ import annotations

import numpy as np

from tests import op_reference as ref

BLOCK = 256
F = np.float32


def e4m3_values():
    """The value of each of the 256 codes, from the format's fields."""
    code = np.arange(256)
    exponent, mantissa = (code >> 3) & 15, code & 7
    v = np.where(exponent == 0, mantissa / 8.0 * 2.0 ** -6,
                 (1.0 + mantissa / 8.0) * 2.0 ** (exponent.astype(float) - 7))
    v = np.where((code & 0x7F) == 0x7F, np.nan, v)
    return np.where(code & 0x80, -v, v)


VALUES = e4m3_values()


def decode(codes, scales, square=False):
    """The values of codes; of a second moment (square) 0x7F is an infinity."""
    if square:
        return np.where(codes == 0x7F, F(np.inf), decode(codes, scales))
    return (VALUES[codes] * np.repeat(scales.astype(np.float64), BLOCK)[:codes.size]).astype(F)


def scales_of(x):
    """The least power of two, 2^-126 or more, that keeps each block within 448."""
    out = np.empty((x.size + BLOCK - 1) // BLOCK)
    for i in range(out.size):
        b = np.abs(x[i * BLOCK:(i + 1) * BLOCK].astype(np.float64))
        most = b[np.isfinite(b)].max(initial=0.0)
        e = -126
        while most > 448.0 * 2.0 ** e:
            e += 1
        out[i] = 2.0 ** e
    return out.astype(F)


def place(y, u):
    """Codes of the magnitudes y <= 448 (float64): floor(place + u / 65536) in the
    distance of their neighbours."""
    e = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    value = np.floor(y / step + u / 65536.0) * step
    code = np.searchsorted(VALUES[:0x7F], value).astype(np.int64)
    assert (VALUES[code] == value).all()
    return code


def encode(x, u, keep):
    """(codes, scales) of x (fp32) with 16-bit numbers u; keep: above 0 stays so."""
    scales = scales_of(x)
    finite = np.isfinite(x)
    y = np.where(finite, x, 0).astype(np.float64) / np.repeat(scales.astype(np.float64),
                                                             BLOCK)[:x.size]
    code = place(np.abs(y), u)
    if keep:
        code = np.where((code == 0) & (y > 0), 1, code)
    code = code | np.where(np.signbit(y), 0x80, 0)
    return np.where(finite, code, 0x7F).astype(np.uint8), scales


def words(n, per, word1, steps, seed):
    """16-bit numbers of n values, `per` values a group: [n, 8 / per]."""
    groups = (n + per - 1) // per
    e = np.arange(groups, dtype=np.uint64)
    full = lambda v: np.full(e.shape, v, dtype=np.uint64)
    w = ref.philox4x32([e, full(word1), full(steps & 0xFFFFFFFF), full(steps >> 32)],
                       (seed & 0xFFFFFFFF, seed >> 32), 7)
    return np.stack(w, 1).astype("<u4").view("<u2").reshape(groups * per, 8 // per)[:n]


def step(p, g, m, v, t, lr, weight_decay, beta1, beta2, eps, grad_scale=None):
    """One step for values p (float64), g, m, v (fp32): fp32 (m, v), float64 p and
    the update's magnitude."""
    with np.errstate(all="ignore"):
        g = g if grad_scale is None else g * F(grad_scale)
        m = m * F(beta1) + g * F(1.0 - beta1)
        v = v * F(beta2) + (g * F(1.0 - beta2)) * g
        update = (lr / (1.0 - beta1 ** t)) * m.astype(np.float64) / \
            (np.sqrt(v.astype(np.float64)) / np.sqrt(1.0 - beta2 ** t) + eps)
    return m, v, p * (1.0 - lr * weight_decay) - update, np.abs(update)


def stochastic_bf16(p, u):
    """bf16 bits of fp32 p: the bits below the upper half plus u, cut."""
    b = p.astype(F).view(np.uint32)
    out = (b.astype(np.int64) + np.where(np.isfinite(p), u, 0)) >> 16
    return np.where(np.isnan(p), 0x7FC0, out).astype(np.uint16)
