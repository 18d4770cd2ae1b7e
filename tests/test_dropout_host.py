"""Dropout on the CPU: the reference's generator against the published
known-answer vectors of Philox4x32, its rate and independence, and every
refusal of the two entry points (nothing reaches a device)."""
import ctypes

import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import op_reference as ref

NULLS = (0x0, 0x0, 0x0, 0x0), (0x0, 0x0)
ONES = (0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2
DIGITS = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)


@pytest.mark.parametrize("vector, rounds, want", [
    (NULLS, 7, (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
    (NULLS, 10, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (ONES, 10, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    (DIGITS, 10, (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(vector, rounds, want):
    counter, key = vector
    got = ref.philox4x32([np.array([c]) for c in counter], key, rounds)
    assert tuple(int(v[0]) for v in got) == want


def test_rate_and_streams():
    """The kept share is within five standard deviations of 1 - T / 65536, and
    two offsets agree on it by chance only."""
    n, p = 1 << 20, 0.1
    a = ref.keep_mask(1024, 1024, p, 7, 0)
    b = ref.keep_mask(1024, 1024, p, 7, 1)
    q = 1.0 - ref.threshold(p) / 65536.0
    assert abs(a.mean() - q) < 5 * (q * (1 - q) / n) ** 0.5
    both = q * q + (1 - q) * (1 - q)
    assert abs((a == b).mean() - both) < 5 * (both * (1 - both) / n) ** 0.5
    assert abs(np.corrcoef(a[:-1].ravel(), a[1:].ravel())[0, 1]) < 5 / n ** 0.5


def _drop(p=0.1, rng=0x8000, reserved=0):
    return ctypes.byref(dsl._DropoutDesc(rng, p, reserved))


def test_dropout_refusals():
    L = dsl.lib()

    def call(drop=None, x=0x1000, ldx=64, res=None, ldres=0, y=0x2000, ldy=64, dtype=0, rows=16,
             cols=64):
        return L.fp8_dropout(drop or _drop(), x, ldx, res, ldres, y, ldy, dtype, rows, cols, None)

    assert L.fp8_dropout(None, 0x1000, 64, None, 0, 0x2000, 64, 0, 16, 64, None) == -1
    assert call(_drop(rng=0)) == -1
    assert call(_drop(rng=0x8004)) == -3
    assert call(_drop(reserved=1)) == -5
    for p in (-0.1, 1.0, 0.99999999, float("nan"), float("inf")):
        assert call(_drop(p=p)) == -5
    assert call(dtype=2) == -5
    assert call(cols=60) == -2
    assert call(rows=-1) == -2
    assert call(ldx=56) == -2
    assert call(ldx=68) == -2                                  # bf16: not a multiple of 8
    assert call(ldx=66, dtype=1) == -2                         # fp32: not a multiple of 4
    assert call(ldy=60) == -2
    assert call(res=0x3000, ldres=56) == -2
    assert call(rows=(1 << 25) + 1) == -2
    assert call(cols=1 << 27, ldx=1 << 27, ldy=1 << 27) == -2
    assert call(x=None) == -1 and call(y=None) == -1
    assert call(x=0x1008) == -3 and call(y=0x2004) == -3 and call(res=0x3008, ldres=64) == -3
    assert call(rows=0) == 0 and call(cols=0, x=None, y=None) == 0


def test_dropout_cast_refusals():
    L = dsl.lib()
    desc = lambda rows=32, cols=48, fmt=0, data=0x100000, data_t=0x200000: dsl._Desc(
        data, data_t, 0x3000, fmt, 0, rows, cols)

    def call(drop=None, x=0x1000, ldx=48, res=None, ldres=0, y=None, ldy=0, rows=32, cols=48,
             scale=0x4000, out=None, dbias=None, ws=None, ws_bytes=0):
        return L.fp8_dropout_cast_transpose_amax(
            drop or _drop(), x, ldx, res, ldres, y, ldy, rows, cols, scale,
            ctypes.byref(out or desc()), None, dbias, ws, ws_bytes, None, None)

    assert call(_drop(p=2.0)) == -5
    assert call(_drop(rng=0)) == -1
    assert call(rows=30, out=desc(30)) == -2
    assert call(cols=40, ldx=40, out=desc(cols=40)) == -2
    assert call(out=desc(16)) == -2
    assert call(out=desc(fmt=2)) == -4
    assert call(out=desc(data=0, data_t=0)) == -1
    assert call(scale=None) == -1
    assert call(x=None) == -1
    assert call(x=0x1008) == -3
    assert call(ldx=52) == -2
    assert call(res=0x5000, ldres=40) == -2
    assert call(res=0x5008, ldres=48) == -3
    assert call(y=0x6000, ldy=44) == -2
    assert call(y=0x6004, ldy=48) == -3
    assert call(dbias=0x7002, ws=0x8000, ws_bytes=512) == -3
    assert call(dbias=0x7000) == -1                            # no workspace
    assert call(dbias=0x7000, ws=0x8000, ws_bytes=511) == -2
    assert call(dbias=0x7000, ws=0x8008, ws_bytes=512) == -3


def test_binding_refusals():
    rng = torch.zeros(2, dtype=torch.int64)
    drop = dsl.Dropout(0.1, rng)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bf16 or fp32"):
        dsl.fp8_dropout(torch.zeros(4, 8, dtype=torch.float16), drop, bf(4, 8))
    with pytest.raises(ValueError, match="device tensor"):
        dsl.fp8_dropout(bf(4, 8), drop, bf(4, 8))
    with pytest.raises(ValueError, match="shape"):
        dsl._matrix(bf(4, 8), 4, 16, torch.bfloat16, "y")
    with pytest.raises(ValueError, match="two elements"):
        dsl.Dropout(0.1, torch.zeros(3, dtype=torch.int64)).desc()
    with pytest.raises(ValueError, match="device tensor"):
        drop.desc()
    with pytest.raises(ValueError, match="unit stride"):
        dsl._matrix(bf(8, 4).t(), 4, 8, torch.bfloat16, "x")
    with pytest.raises(TypeError, match="must be"):
        dsl._matrix(torch.zeros(4, 8), 4, 8, torch.bfloat16, "y")


def test_binding_overlap():
    """An output is an input itself, or apart from it (columns of one wider
    tensor included); anything else is refused."""
    wide = torch.zeros(8, 48, dtype=torch.bfloat16)
    a, b, c = wide[:, :16], wide[:, 16:32], wide[:, 8:24]

    def check(y, t, same=True):
        dsl._need_apart((y.data_ptr(), y.stride(0)), (t.data_ptr(), t.stride(0)), y.shape[0],
                        y.shape[1], t.shape[1], 2, "y", same=same)

    check(a, a)
    check(a, b)
    check(b, a)
    check(wide[:, 32:], a)
    check(wide[4:], wide[:4])
    dsl._need_apart((a.data_ptr(), 48), dsl._NONE, 8, 16, 16, 2, "y")
    for y, t in ((a, c), (c, a), (c, b), (wide[1:], wide[:-1])):
        with pytest.raises(ValueError, match="overlap"):
            check(y, t)
    with pytest.raises(ValueError, match="overlap"):
        check(a, a, same=False)
