"""GPU parity of fp8_dropout and fp8_dropout_cast_transpose_amax.

Every step of the operator is a rounding the definition names (fp32 product,
fp32 sum, one rounding to the output type), so y, the codes, the transpose,
the amax and the scale-inverse are compared bit for bit.  The bias gradient
sums the stored bf16 values in fp32 in tile order, within the bound that
fp8_cast_transpose_amax_dbias states."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
import oracle
from tests import op_reference as ref
from tests.gpu_util import DEV, bf16_values, bits8, bits16, f32, f32_bits

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x0123456789ABCDEF, 0x7EDCBA9876543210


def _rng(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


def _rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _want(x, res, p, seed=SEED, offset=OFFSET):
    """fp32 values of the result before its rounding, from CPU tensors."""
    rows, cols = x.shape
    mask = ref.keep_mask(rows, cols, p, seed, offset)
    return ref.dropout(x.float().numpy(), mask, ref.factor(p),
                       None if res is None else res.float().numpy())


def _bits(t):
    return bits16(t) if t.dtype == torch.bfloat16 else f32_bits(t)


def _rounded(v, dtype):
    return ref.bf16_round(v) if dtype == torch.bfloat16 else v.view(np.uint32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(1, 8), (3, 24), (33, 8), (17, 520), (5, 2056), (1037, 1160)])
def test_shapes(shape, residual, dtype):
    x = _rand(shape, 1, dtype=dtype)
    res = _rand(shape, 2, dtype=dtype) if residual else None
    y = torch.full(shape, -7.0, dtype=dtype, device=DEV)
    dsl.fp8_dropout(x.to(DEV), dsl.Dropout(0.25, _rng()), y,
                    residual=None if res is None else res.to(DEV))
    np.testing.assert_array_equal(_bits(y), _rounded(_want(x, res, 0.25), dtype))


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.999, 65535 / 65536])
def test_rates(p):
    """p below half a step keeps everything; the largest p keeps about one in 65536."""
    x = _rand((256, 512), 3)
    y = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    dsl.fp8_dropout(x.to(DEV), dsl.Dropout(p, _rng()), y)
    np.testing.assert_array_equal(bits16(y), ref.bf16_round(_want(x, None, p)))


@pytest.mark.parametrize("seed, offset", [(0, 0), (-1, -1), (2 ** 63 - 1, 1), (1, 2 ** 32)])
def test_seed_and_offset_words(seed, offset):
    x = _rand((16, 128), 4)
    y = torch.empty(16, 128, dtype=torch.bfloat16, device=DEV)
    dsl.fp8_dropout(x.to(DEV), dsl.Dropout(0.5, _rng(seed, offset)), y)
    np.testing.assert_array_equal(bits16(y), ref.bf16_round(_want(x, None, 0.5, seed, offset)))


def test_positions_past_32_bits_of_elements():
    """The last rows of a tensor of 2^32 + 2^21 elements (8.6 GB)."""
    rows, cols = (1 << 20) + 512, 4096
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    dsl.fp8_dropout(x, dsl.Dropout(0.5, _rng()), x)
    for first in (0, rows - 8):
        mask = ref.keep_mask(8, cols, 0.5, SEED, OFFSET, first_row=first)
        np.testing.assert_array_equal(x[first:first + 8].float().cpu().numpy(), 2.0 * mask)


def test_strides_and_in_place():
    """Column slices of wider tensors; y equal to x and equal to the residual;
    nothing outside the slice is written."""
    wide = _rand((40, 96), 5)
    x, res = wide[:, 16:56], wide[:, 56:96]
    want = ref.bf16_round(_want(x, res, 0.3))
    for target in ("apart", "x", "residual"):
        w = wide.to(DEV)
        other = torch.zeros(40, 64, dtype=torch.bfloat16, device=DEV)
        y = {"apart": other[:, 8:48], "x": w[:, 16:56], "residual": w[:, 56:96]}[target]
        dsl.fp8_dropout(w[:, 16:56], dsl.Dropout(0.3, _rng()), y, residual=w[:, 56:96])
        np.testing.assert_array_equal(bits16(y), want)
        assert torch.equal(w[:, :16].cpu(), wide[:, :16])
        assert float(other[:, :8].abs().sum() + other[:, 48:].abs().sum()) == 0.0


def test_dropped_infinities_and_nans_leave_nothing():
    x = torch.full((64, 256), float("nan"), dtype=torch.bfloat16)
    x[::2] = float("inf")
    res = _rand((64, 256), 6)
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty(64, 256, dtype=dtype, device=DEV)
        dsl.fp8_dropout(x.to(dtype).to(DEV), dsl.Dropout(0.5, _rng()), y,
                        residual=res.to(dtype).to(DEV))
        mask = ref.keep_mask(64, 256, 0.5, SEED, OFFSET)
        got, base = y.float().cpu().numpy(), res.float().numpy()
        np.testing.assert_array_equal(got[~mask], base[~mask])
        assert np.isnan(got[1::2][mask[1::2]]).all()
        assert (got[::2][mask[::2]] == np.inf).all()


def test_gradient_is_the_same_mask():
    """The call on an output gradient: exactly the derivative of the forward,
    which differences of a linear function give without error (powers of two
    times the factor 2)."""
    x = torch.randint(-8, 9, (32, 64), generator=torch.Generator().manual_seed(1)).float()
    d = dsl.Dropout(0.5, _rng())
    y0, y1, g = (torch.empty(32, 64, device=DEV) for _ in range(3))
    dsl.fp8_dropout(x.to(DEV), d, y0)
    dsl.fp8_dropout((x + 1).to(DEV), d, y1)
    dsl.fp8_dropout(torch.ones(32, 64, device=DEV), d, g)
    assert torch.equal(y1 - y0, g)


def _check_cast(x, res, p, scale, fmt, *, y=True, q=True, qt=True, dbias=False, noop=None):
    rows, cols = x.shape
    dev = lambda t: None if t is None else t.to(DEV)
    out = dsl.Float8Tensor.empty(rows, cols, fmt, data=q, transpose=qt, device=DEV)
    yt = torch.full((rows, cols), -7.0, dtype=torch.bfloat16, device=DEV) if y else None
    amax = torch.zeros(1, device=DEV)
    db = torch.full((cols,), float("nan"), device=DEV) if dbias else None
    ws = torch.full((dsl.fp8_cast_dbias_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8,
                    device=DEV) if dbias else None
    s = torch.tensor([scale], device=DEV)
    dsl.fp8_dropout_cast_transpose_amax(dev(x), dsl.Dropout(p, _rng()), s, out, amax,
                                        residual=dev(res), y=yt, dbias=db, workspace=ws)
    want = ref.bf16_round(_want(x, res, p))
    oq, oqt, oamax, osinv = oracle.cast_transpose_amax(want, scale, fmt)
    if y:
        np.testing.assert_array_equal(bits16(yt), want)
    if q:
        np.testing.assert_array_equal(bits8(out.data), oq)
    if qt:
        np.testing.assert_array_equal(bits8(out.data_t), oqt)
    assert f32_bits(amax)[0] == np.float32(oamax).view(np.uint32)
    assert f32_bits(out.scale_inv)[0] == np.float32(osinv).view(np.uint32)
    if dbias:
        v = bf16_values(want)
        bound = (-(-rows // 128) + 12) * 2.0 ** -24 * np.abs(v).sum(0)
        assert (np.abs(f32(db) - v.sum(0)) <= bound).all()


@pytest.mark.parametrize("shape", [(16, 16), (128, 256), (400, 272), (272, 400), (1024, 2048)])
@pytest.mark.parametrize("fmt", [dsl.E4M3, dsl.E5M2])
@pytest.mark.parametrize("residual, dbias", [(True, False), (False, True), (True, True)])
def test_cast_shapes(shape, fmt, residual, dbias):
    x = _rand(shape, 7)
    res = _rand(shape, 8) if residual else None
    _check_cast(x, res, 0.1, 41.0, fmt, dbias=dbias, y=residual)


@pytest.mark.parametrize("extra", [16, 48, 64, 80, 112])
def test_every_column_residue_of_a_tile(extra):
    _check_cast(_rand((48, 128 + extra), 9), _rand((48, 128 + extra), 10), 0.3, 9.0, dsl.E4M3,
                dbias=True)


@pytest.mark.parametrize("q, qt", [(True, False), (False, True)])
def test_one_layout_only(q, qt):
    _check_cast(_rand((80, 144), 11), None, 0.5, 3.0, dsl.E5M2, q=q, qt=qt, y=False, dbias=True)


@pytest.mark.parametrize("scale", [0.0, float("inf"), float("nan"), -2.0, 2.0 ** 100])
def test_cast_special_scales(scale):
    x = _rand((32, 48), 12)
    x[0, :8] = float("nan")
    x[1, :8] = float("inf")
    _check_cast(x, None, 0.2, scale, dsl.E4M3)


def test_cast_noop_empty_and_amax_accumulation():
    x = _rand((32, 48), 13).to(DEV)
    d, s = dsl.Dropout(0.1, _rng()), torch.tensor([2.0], device=DEV)
    out = dsl.Float8Tensor.empty(32, 48, dsl.E4M3, device=DEV)
    out.data.fill_(0x11)
    amax, flag = torch.full((1,), 1e4, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    dsl.fp8_dropout_cast_transpose_amax(x, d, s, out, amax, noop_flag=flag)
    assert (out.data == 0x11).all() and float(out.scale_inv) == 1.0
    flag.zero_()
    dsl.fp8_dropout_cast_transpose_amax(x, d, s, out, amax, noop_flag=flag)
    assert float(amax) == 1e4 and float(out.scale_inv) == 0.5       # the larger maximum stays
    empty = dsl.Float8Tensor.empty(0, 48, dsl.E4M3, device=DEV)
    db = torch.full((48,), 3.0, device=DEV)
    dsl.fp8_dropout_cast_transpose_amax(x[:0], d, s, empty, amax, dbias=db,
                                        workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert float(empty.scale_inv) == 0.5 and float(db.abs().sum()) == 0.0


def test_dropout_in_a_graph_draws_from_the_device_offset():
    """A captured call reads rng when it runs: the program bumps the offset
    between replays, and every replay equals the eager call at that offset."""
    x = _rand((64, 128), 14)
    xd, rng = x.to(DEV), _rng(5, 0)
    y = torch.empty(64, 128, dtype=torch.bfloat16, device=DEV)
    out = dsl.Float8Tensor.empty(64, 128, dsl.E4M3, device=DEV)
    s, amax = torch.tensor([3.0], device=DEV), torch.zeros(1, device=DEV)
    d = dsl.Dropout(0.4, rng)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        dsl.fp8_dropout_cast_transpose_amax(xd, d, s, out, amax, y=y)
    for offset in range(4):
        rng[1] = offset
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.bf16_round(_want(x, None, 0.4, 5, offset))
        np.testing.assert_array_equal(bits16(y), want)
        np.testing.assert_array_equal(bits8(out.data),
                                      oracle.cast_transpose_amax(want, 3.0, dsl.E4M3)[0])
        assert float((y * 2).sum()) == float((y * 2).sum())          # eager work between replays
