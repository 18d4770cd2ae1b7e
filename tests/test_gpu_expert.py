"""GPU parity of the expert-routing calls.

Plans, gathered rows, codes, transposes and dx are compared bit for bit: each is
a copy, or one fp32 product rounded as the definition says.  Sums:

* y: top_k + 1 fp32 operations of relative error 2^-24 on terms of magnitude
  `size` in all, then half a bf16 step, 2^-8 of the value (2^-134 below the
  normal numbers);
* dweights: a sum of `cols` products in any order, at most cols + 1 roundings of
  2^-24 on terms of magnitude `size` in all.
"""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
import oracle
from tests import expert_reference as ref
from tests.gpu_util import DEV, bf16_values, bits8, bits16, f32

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
F32 = np.float32


def _rand(shape, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16)


def _ids(tokens, top_k, experts, seed, how="mixed"):
    r = np.random.default_rng(seed)
    if how == "one":                             # a single expert takes all
        return np.full((tokens, top_k), experts - 1, np.int32)
    if how == "none":                            # a batch of padding
        return np.full((tokens, top_k), -1, np.int32)
    ids = r.integers(0, experts, (tokens, top_k)).astype(np.int32)
    if how == "mixed":                           # padding and other values that name none
        bad = np.array([-1, experts, 2 ** 31 - 1, -2 ** 31], np.int32)
        at = r.random(ids.shape) < 0.1
        ids[at] = bad[r.integers(0, 4, int(at.sum()))]
    return ids


def _plan(ids, experts, capacity=0):
    plan = dsl.ExpertPlan.empty(*ids.shape, experts, capacity)
    plan.buf.fill_(0x5A)                         # its contents on entry do not matter
    dsl.fp8_expert_plan(torch.from_numpy(ids).to(DEV), plan)
    return plan


def _check_plan(plan, want):
    offsets, counts, slots, sources = want
    np.testing.assert_array_equal(plan.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(plan.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(plan.slots.cpu().numpy(), slots)
    np.testing.assert_array_equal(plan.sources.cpu().numpy(), sources)


@pytest.mark.parametrize("how", ["mixed", "one", "none", "all"])
@pytest.mark.parametrize("tokens, top_k, experts, capacity", [
    (1, 1, 1, 0), (1, 8, 8, 0), (7, 3, 5, 16), (63, 1, 2, 0), (64, 2, 1024, 0), (65, 5, 3, 32),
    (1000, 8, 64, 144), (1024, 8, 16, 0), (1025, 8, 16, 0), (4099, 3, 13, 1168),
    (20000, 4, 128, 0), (9000, 2, 1024, 16), (300, 64, 100, 0), (40000, 1, 7, 0)])
def test_plan(tokens, top_k, experts, capacity, how):
    """One workgroup (to 8192 pairs) and several; a token may name an expert twice."""
    ids = _ids(tokens, top_k, experts, 1, how)
    _check_plan(_plan(ids, experts, capacity), ref.plan(ids, experts, capacity))


@pytest.mark.parametrize("capacity", [0, 48])
def test_plan_of_no_tokens(capacity):
    ids = np.zeros((0, 4), np.int32)
    plan = _plan(ids, 5, capacity)
    _check_plan(plan, ref.plan(ids, 5, capacity))
    y = torch.full((plan.rows, 32), 3.0, dtype=BF16, device=DEV)
    x = torch.empty(0, 32, dtype=BF16, device=DEV)
    dsl.fp8_expert_gather(plan, x, y)
    assert (y == 0).all()                        # every row belongs to a segment
    dsl.fp8_expert_combine(plan, y, x)
    dsl.fp8_expert_combine_backward(plan, x, y, torch.empty(0, 4, device=DEV))


def test_plan_of_the_most_pairs():
    """2^23 pairs, checked by what a plan is: slots and sources are each other's
    inverse, experts' pairs are in order, counts are the ids'."""
    tokens, top_k, experts = 1 << 20, 8, 1024
    ids = torch.randint(0, experts, (tokens, top_k), dtype=torch.int32, device=DEV,
                        generator=torch.Generator(DEV).manual_seed(2))
    plan = dsl.ExpertPlan.empty(tokens, top_k, experts)
    dsl.fp8_expert_plan(ids, plan)
    counts = torch.bincount(ids.view(-1), minlength=experts)
    assert torch.equal(plan.counts.long(), counts)
    lengths = (counts + 15) // 16 * 16
    assert torch.equal(plan.offsets[1:].long(), lengths.cumsum(0))
    slots, sources = plan.slots.view(-1).long(), plan.sources.long()
    assert torch.equal(sources[slots], torch.arange(tokens * top_k, device=DEV))
    assert int((sources >= 0).sum()) == tokens * top_k
    order = torch.sort(ids.view(-1), stable=True).indices
    assert torch.equal(sources[sources >= 0], order)


SHAPES = [  # tokens, top_k, experts, capacity, cols
    (1, 1, 1, 0, 16), (1, 8, 8, 0, 2048), (3, 2, 5, 16, 48), (17, 3, 4, 0, 528),
    (130, 6, 3, 0, 144), (257, 2, 9, 64, 2064), (64, 8, 64, 0, 1040), (1000, 4, 37, 112, 112),
    (9, 64, 7, 0, 256)]


@pytest.mark.parametrize("tokens, top_k, experts, capacity, cols", SHAPES + [
    (5, 2, 3, 0, 8), (33, 3, 4, 0, 24), (12, 9, 4, 0, 4104)])
@pytest.mark.parametrize("how", ["mixed", "none", "one"])
def test_gather(tokens, top_k, experts, capacity, cols, how):
    ids = _ids(tokens, top_k, experts, 3, how)
    plan, (offsets, _, _, sources) = _plan(ids, experts, capacity), ref.plan(ids, experts, capacity)
    x = _rand((tokens, cols), 4)
    x[-1, 3], x[0, 2] = float("nan"), float("-inf")
    y = torch.full((plan.rows, cols), -7.0, dtype=BF16, device=DEV)
    dsl.fp8_expert_gather(plan, x.to(DEV), y)
    end = int(offsets[-1])
    np.testing.assert_array_equal(bits16(y[:end]), ref.gather(bits16(x), sources, top_k, end))
    assert (y[end:] == -7.0).all()               # behind the last segment


@pytest.mark.parametrize("tokens, top_k, experts, capacity, cols", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("fmt", [dsl.E4M3, dsl.E5M2])
def test_gather_cast(tokens, top_k, experts, capacity, cols, weighted, fmt):
    ids = _ids(tokens, top_k, experts, 5)
    plan, (offsets, _, _, sources) = _plan(ids, experts, capacity), ref.plan(ids, experts, capacity)
    x = _rand((tokens, cols), 6)
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(7))
    w[ids < 0] = float("nan")                    # of pairs without an expert: not read
    scale, amax = torch.tensor([37.5], device=DEV), torch.zeros(1, device=DEV)
    q = dsl.Float8Tensor.empty(plan.rows, cols, fmt)
    q.data.fill_(0xAA)
    q.data_t.fill_(0xAA)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x.to(DEV), scale, q, amax,
                                              weights=w.to(DEV) if weighted else None)
    end = int(offsets[-1])
    y = ref.gather(bits16(x), sources, top_k, end, w.numpy() if weighted else None)
    codes, _, top, sinv = oracle.cast_transpose_amax(y, 37.5, fmt)
    np.testing.assert_array_equal(bits8(q.data[:end]), codes)
    assert (q.data[end:] == 0xAA).all()
    for part, a, b in zip(plan.segments(q, offsets), offsets, offsets[1:]):
        np.testing.assert_array_equal(bits8(part.data), codes[a:b])
        np.testing.assert_array_equal(bits8(part.data_t), codes[a:b].T)
    assert (q.data_t.view(-1)[end * cols:] == 0xAA).all()
    assert f32(amax)[0] == top and f32(q.scale_inv)[0] == sinv
    # One output alone gives the same codes; a larger amax stays.
    amax.fill_(1e30)
    for want_data in (True, False):
        one = dsl.Float8Tensor.empty(plan.rows, cols, fmt, data=want_data, transpose=not want_data)
        for t in (one.data, one.data_t):
            if t is not None:
                t.fill_(0xAA)
        dsl.fp8_expert_gather_cast_transpose_amax(plan, x.to(DEV), scale, one, amax,
                                                  weights=w.to(DEV) if weighted else None)
        got, want = (one.data, q.data) if want_data else (one.data_t, q.data_t)
        assert torch.equal(got, want) and float(amax) == float(F32(1e30))


@pytest.mark.parametrize("how", ["none", "nan"])
def test_gather_cast_specials(how):
    """A batch of padding (zero codes, an untouched amax) and NaN, infinite and
    overflowing rows; a weight of 0 on an infinity is a NaN."""
    tokens, top_k, experts, cols = 40, 2, 3, 144
    ids = _ids(tokens, top_k, experts, 8, "none" if how == "none" else "all")
    plan, want = _plan(ids, experts, 48), ref.plan(ids, experts, 48)
    x = _rand((tokens, cols), 9)
    x[1, 5], x[2, 7], x[3, 9], x[4, 11] = float("nan"), float("inf"), float("-inf"), 3e38
    w = torch.full((tokens, top_k), 2.0)
    w[2, 0] = 0.0
    scale, amax = torch.tensor([1.0], device=DEV), torch.zeros(1, device=DEV)
    q = dsl.Float8Tensor.empty(plan.rows, cols, dsl.E4M3)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x.to(DEV), scale, q, amax, weights=w.to(DEV))
    y = ref.gather(bits16(x), want[3], top_k, plan.rows, w.numpy())
    codes, _, top, _ = oracle.cast_transpose_amax(y, 1.0, dsl.E4M3)
    np.testing.assert_array_equal(bits8(q.data), codes)
    assert np.array_equal(f32(amax)[0], top, equal_nan=True)
    if how == "none":
        assert not codes.any() and float(amax) == 0.0


@pytest.mark.parametrize("cols", [16, 144, 256])
def test_gather_cast_infinite_weights(cols):
    """An infinite weight makes its row infinite and nothing else, also where a tile
    reaches past the columns."""
    ids = _ids(40, 2, 3, 12, "all")
    plan, want = _plan(ids, 3, 48), ref.plan(ids, 3, 48)
    x = _rand((40, cols), 13).abs() + 1.0
    w = torch.full((40, 2), 0.5)
    w[7, 1], w[9, 0] = float("inf"), float("-inf")
    amax, q = torch.zeros(1, device=DEV), dsl.Float8Tensor.empty(plan.rows, cols, dsl.E5M2)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x.to(DEV), torch.ones(1, device=DEV), q, amax,
                                              weights=w.to(DEV))
    y = ref.gather(bits16(x), want[3], 2, plan.rows, w.numpy())
    codes, _, top, _ = oracle.cast_transpose_amax(y, 1.0, dsl.E5M2)
    np.testing.assert_array_equal(bits8(q.data), codes)
    assert float(amax) == float(top) == float("inf")


def test_gather_cast_without_a_kept_pair():
    """Segments without rows: no tile, an untouched buffer and amax, the scale-inverse."""
    plan, x = _plan(np.full((40, 2), -1, np.int32), 3), _rand((40, 64), 11).to(DEV)
    q, amax = dsl.Float8Tensor.empty(plan.rows, 64, dsl.E4M3), torch.full((1,), 2.0, device=DEV)
    q.data.fill_(7)
    q.data_t.fill_(7)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x, torch.tensor([4.0], device=DEV), q, amax)
    assert (q.data == 7).all() and (q.data_t == 7).all()
    assert float(amax) == 2.0 and float(q.scale_inv) == 0.25


def test_gather_cast_noop_and_empty():
    ids = _ids(40, 2, 3, 10, "all")
    plan, x = _plan(ids, 3, 32), _rand((40, 64), 11).to(DEV)
    scale, amax, flag = torch.tensor([2.0], device=DEV), torch.zeros(1, device=DEV), \
        torch.ones(1, dtype=torch.int32, device=DEV)
    q = dsl.Float8Tensor.empty(plan.rows, 64, dsl.E4M3)
    q.data.fill_(1)
    q.data_t.fill_(1)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x, scale, q, amax, noop_flag=flag)
    assert (q.data == 1).all() and (q.data_t == 1).all() and float(amax) == 0
    assert float(q.scale_inv) == 1.0
    empty = dsl.ExpertPlan.empty(0, 2, 3)
    dsl.fp8_expert_plan(torch.empty(0, 2, dtype=torch.int32, device=DEV), empty)
    none = dsl.Float8Tensor.empty(0, 64, dsl.E4M3)
    dsl.fp8_expert_gather_cast_transpose_amax(empty, x[:0], scale, none, amax)
    assert float(none.scale_inv) == 0.5


def _check_y(y, want, size, top_k):
    y = bf16_values(bits16(y))
    bound = (top_k + 1) * 2.0 ** -24 * size
    assert (np.abs(y - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound) + 2.0 ** -134).all()


@pytest.mark.parametrize("tokens, top_k, experts, capacity, cols", SHAPES + [
    (5, 2, 3, 0, 8), (33, 3, 4, 0, 24), (12, 9, 4, 0, 4104)])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("based", [False, True])
def test_combine(tokens, top_k, experts, capacity, cols, weighted, based):
    ids = _ids(tokens, top_k, experts, 12)
    plan, (_, _, slots, sources) = _plan(ids, experts, capacity), ref.plan(ids, experts, capacity)
    x, base = _rand((plan.rows, cols), 13), _rand((tokens, cols), 14)
    x[torch.from_numpy(sources < 0)] = float("nan")          # rows without a pair: not read
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(15)) - 0.3
    w[torch.from_numpy(slots < 0)] = float("nan")
    y = torch.full((tokens, cols), -7.0, dtype=BF16, device=DEV)
    dsl.fp8_expert_combine(plan, x.to(DEV), y, weights=w.to(DEV) if weighted else None,
                           base=base.to(DEV) if based else None)
    want, size = ref.combine(np.nan_to_num(bf16_values(bits16(x))), slots,
                             np.nan_to_num(w.numpy()) if weighted else None,
                             bf16_values(bits16(base)) if based else None)
    _check_y(y, want, size, top_k)
    if based:                                    # into base itself
        z = base.to(DEV)
        dsl.fp8_expert_combine(plan, x.to(DEV), z, weights=w.to(DEV) if weighted else None, base=z)
        assert torch.equal(z.view(torch.int16), y.view(torch.int16))


def test_combine_specials():
    """Infinities and NaNs of rows that are read, and a token without experts."""
    ids = np.array([[0, 1], [1, 0], [-1, -1], [0, -1]], np.int32)
    plan, (_, _, slots, _) = _plan(ids, 2), ref.plan(ids, 2)
    x = _rand((plan.rows, 16), 16)
    x[slots[0, 0], 0], x[slots[0, 1], 0] = float("inf"), float("-inf")
    x[slots[1, 0], 1], x[slots[3, 0], 2] = float("nan"), float("inf")
    y = torch.full((4, 16), -7.0, dtype=BF16, device=DEV)
    dsl.fp8_expert_combine(plan, x.to(DEV), y)
    got = y.float().cpu()
    assert got[0, 0].isnan() and got[1, 1].isnan() and got[3, 2] == float("inf")
    assert (got[2] == 0).all() and got.isfinite().sum() == 4 * 16 - 3


@pytest.mark.parametrize("tokens, top_k, experts, capacity, cols", SHAPES + [
    (5, 2, 3, 0, 8), (33, 3, 4, 0, 24), (12, 9, 4, 0, 4104)])
@pytest.mark.parametrize("with_dx", [False, True])
def test_combine_backward(tokens, top_k, experts, capacity, cols, with_dx):
    ids = _ids(tokens, top_k, experts, 17)
    plan = _plan(ids, experts, capacity)
    offsets, _, slots, sources = ref.plan(ids, experts, capacity)
    x, dy = _rand((plan.rows, cols), 18), _rand((tokens, cols), 19)
    x[torch.from_numpy(sources < 0)] = float("nan")
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(20)) - 0.3
    w[torch.from_numpy(slots < 0)] = float("nan")
    dw = torch.full((tokens, top_k), -7.0, device=DEV)
    dx = torch.full((plan.rows, cols), -7.0, dtype=BF16, device=DEV) if with_dx else None
    xd = x.to(DEV)
    dsl.fp8_expert_combine_backward(plan, dy.to(DEV), xd, dw, weights=w.to(DEV), dx=dx)
    want, size = ref.combine_weight_gradient(bf16_values(bits16(dy)),
                                             np.nan_to_num(bf16_values(bits16(x))), slots)
    assert (np.abs(f32(dw) - want) <= (cols + 1) * 2.0 ** -24 * size).all()
    again = torch.empty_like(dw)
    dsl.fp8_expert_combine_backward(plan, dy.to(DEV), xd, again, weights=w.to(DEV),
                                    dx=xd if with_dx else None)
    assert torch.equal(again, dw)                # the same bits, also with dx in x's place
    if with_dx:
        end = int(offsets[-1])
        np.testing.assert_array_equal(bits16(dx[:end]),
                                      ref.gather(bits16(dy), sources, top_k, end, w.numpy()))
        assert (dx[end:] == -7.0).all()
        assert torch.equal(xd[:end].view(torch.int16), dx[:end].view(torch.int16))
        np.testing.assert_array_equal(bits16(xd[end:]), bits16(x[end:]))


def test_gradients_are_adjoint():
    """sum(dy * combine(x, w)) changes with w by dw and with gathered rows by dx:
    differences of the calls themselves, in bf16's resolution of y."""
    tokens, top_k, experts, cols = 50, 3, 6, 256
    ids = _ids(tokens, top_k, experts, 21)
    plan = _plan(ids, experts)
    x, dy = _rand((plan.rows, cols), 22).to(DEV), _rand((tokens, cols), 23).to(DEV)
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(24)).to(DEV)
    dw, y0, y1 = torch.empty_like(w), torch.empty_like(dy), torch.empty_like(dy)
    dsl.fp8_expert_combine_backward(plan, dy, x, dw, weights=w)
    step = torch.randn(tokens, top_k, generator=torch.Generator().manual_seed(25)).to(DEV)
    dsl.fp8_expert_combine(plan, x, y0, weights=w - step)
    dsl.fp8_expert_combine(plan, x, y1, weights=w + step)
    live = plan.slots >= 0
    for t in range(tokens):
        up = (dy[t].double() * y1[t].double()).sum()
        down = (dy[t].double() * y0[t].double()).sum()
        got = float((dw[t].double() * step[t].double())[live[t]].sum())
        # Each y is within 2^-8 of itself; fp32 sums are far below that.
        slack = 2.0 ** -8 * float((dy[t].double().abs() * (y1[t].abs() + y0[t].abs()).double()).sum())
        assert abs(float(up - down) / 2 - got) <= 0.51 * slack + 1e-6


def test_strides():
    """Column slices of wider tensors on every side."""
    tokens, top_k, experts, cols = 70, 2, 5, 48
    ids = _ids(tokens, top_k, experts, 26)
    plan, (offsets, _, slots, sources) = _plan(ids, experts), ref.plan(ids, experts)
    end = int(offsets[-1])
    wide = _rand((tokens, 3 * cols + 16), 27).to(DEV)
    x = wide[:, 16:16 + cols]
    rows = torch.full((plan.rows, 2 * cols), -7.0, dtype=BF16, device=DEV)
    dsl.fp8_expert_gather(plan, x, rows[:, cols:])
    np.testing.assert_array_equal(bits16(rows[:end, cols:]),
                                  ref.gather(bits16(x), sources, top_k, end))
    assert (rows[:, :cols] == -7.0).all() and (rows[end:] == -7.0).all()
    q = dsl.Float8Tensor.empty(plan.rows, cols, dsl.E4M3)
    scale = torch.tensor([3.0], device=DEV)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x, scale, q)
    np.testing.assert_array_equal(
        bits8(q.data[:end]),
        oracle.cast_transpose_amax(ref.gather(bits16(x), sources, top_k, end), 3.0, dsl.E4M3)[0])
    # y and base side by side in one tensor.
    base, y = wide[:, 16:16 + cols], wide[:, 16 + cols:16 + 2 * cols]
    keep = wide.clone()
    dsl.fp8_expert_combine(plan, rows[:, cols:], y, base=base)
    want, size = ref.combine(bf16_values(bits16(rows[:, cols:])), slots, None,
                             bf16_values(bits16(base)))
    _check_y(y, want, size, top_k)
    assert torch.equal(wide[:, :16 + cols], keep[:, :16 + cols])
    assert torch.equal(wide[:, 16 + 2 * cols:], keep[:, 16 + 2 * cols:])
    dw = torch.empty(tokens, top_k, device=DEV)
    dx = torch.full((plan.rows, 2 * cols), -7.0, dtype=BF16, device=DEV)
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(28))
    dsl.fp8_expert_combine_backward(plan, base, rows[:, cols:], dw, weights=w.to(DEV),
                                    dx=dx[:, :cols])
    np.testing.assert_array_equal(bits16(dx[:end, :cols]),
                                  ref.gather(bits16(base), sources, top_k, end, w.numpy()))
    assert (dx[:, cols:] == -7.0).all()


def test_refusals_on_the_device():
    plan = _plan(_ids(20, 2, 3, 29), 3)
    x = torch.zeros(20, 32, dtype=BF16, device=DEV)
    y = torch.zeros(plan.rows, 32, dtype=BF16, device=DEV)
    fresh = dsl.ExpertPlan.empty(20, 2, 3)
    with pytest.raises(ValueError, match="built"):
        dsl.fp8_expert_gather(fresh, x, y)
    both = torch.zeros(plan.rows + 20, 32, dtype=BF16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        dsl.fp8_expert_gather(plan, both[plan.rows - 1:plan.rows + 19], both[:plan.rows])
    with pytest.raises(ValueError, match="overlap"):
        dsl.fp8_expert_combine(plan, both[:plan.rows], both[plan.rows - 1:plan.rows + 19])
    with pytest.raises(ValueError, match="overlap"):
        dsl.fp8_expert_combine_backward(plan, both[plan.rows - 1:plan.rows + 19], y,
                                        torch.zeros(20, 2, device=DEV),
                                        weights=torch.zeros(20, 2, device=DEV),
                                        dx=both[:plan.rows])
    with pytest.raises(ValueError):
        dsl.fp8_expert_gather(plan, x.cpu(), y)
    with pytest.raises(ValueError):
        dsl.fp8_expert_combine(plan, y, x, weights=torch.zeros(20, 3, device=DEV))
    with pytest.raises(TypeError):
        dsl.fp8_expert_combine(plan, y, x, weights=torch.zeros(20, 2, dtype=BF16, device=DEV))
    with pytest.raises(dsl.Fp8Error):                       # 8 columns past a multiple of 16
        dsl.fp8_expert_gather_cast_transpose_amax(plan, x[:, :24], torch.ones(1, device=DEV),
                                                  dsl.Float8Tensor.empty(plan.rows, 24, dsl.E4M3))


def test_a_buffer_without_a_plan():
    """Calls on a buffer that holds no plan of these sizes write nothing."""
    plan = _plan(_ids(20, 2, 3, 30), 3, 16)
    wide = torch.zeros(dsl.fp8_expert_plan_bytes(20, 2, 3, 32), dtype=torch.uint8, device=DEV)
    wide[:plan.buf.numel()] = plan.buf
    for buf in (wide, torch.zeros_like(wide)):
        other = dsl.ExpertPlan(buf, 20, 2, 3, 32, built=True)
        x = torch.ones(20, 32, dtype=BF16, device=DEV)
        y = torch.full((other.rows, 32), 5.0, dtype=BF16, device=DEV)
        z, dw = torch.full((20, 32), 5.0, dtype=BF16, device=DEV), torch.full((20, 2), 5.0, device=DEV)
        q = dsl.Float8Tensor.empty(other.rows, 32, dsl.E4M3)
        q.data.fill_(5)
        dsl.fp8_expert_gather(other, x, y)
        dsl.fp8_expert_combine(other, y, z)
        dsl.fp8_expert_combine_backward(other, x, y, dw)
        dsl.fp8_expert_gather_cast_transpose_amax(other, x, torch.ones(1, device=DEV), q)
        for t in (y, z, dw, q.data):
            assert (t == 5).all()


def test_past_32_bits_of_elements():
    """Tensors of 2^32 elements and more in expert order (8.6 GB)."""
    tokens, top_k, experts, cols = 1 << 17, 4, 16, 8192
    g = torch.Generator(DEV).manual_seed(31)
    ids = torch.randint(0, experts, (tokens, top_k), dtype=torch.int32, device=DEV, generator=g)
    plan = dsl.ExpertPlan.empty(tokens, top_k, experts)
    dsl.fp8_expert_plan(ids, plan)
    # A row's values tell its token.
    x = (torch.arange(tokens, device=DEV) % 251).to(BF16)[:, None].repeat(1, cols)
    y = torch.empty(plan.rows, cols, dtype=BF16, device=DEV)
    assert y.numel() > 1 << 32
    dsl.fp8_expert_gather(plan, x, y)
    end, sources = int(plan.offsets[-1]), plan.sources.long()
    want = torch.where(sources >= 0, (sources // top_k) % 251, 0).to(BF16)
    for a in range(0, end, 1 << 16):
        b = min(end, a + (1 << 16))
        assert (y[a:b] == want[a:b, None]).all()
    z, w = torch.empty_like(x), torch.full((tokens, top_k), 0.5, device=DEV)
    dsl.fp8_expert_combine(plan, y, z, weights=w)
    assert (z == (2 * x)).all()                             # small integers: exact
    dw = torch.empty(tokens, top_k, device=DEV)
    dsl.fp8_expert_combine_backward(plan, torch.ones_like(x), y, dw, weights=w, dx=y)
    assert (dw == x[:, :1].float() * cols).all()
    for a in range(0, end, 1 << 16):
        b = min(end, a + (1 << 16))
        assert (y[a:b] == torch.where(sources[a:b] >= 0, 0.5, 0.0).to(BF16)[:, None]).all()
    del y, z
    q = dsl.Float8Tensor.empty(plan.rows, cols, dsl.E4M3)
    x.clamp_(max=16.0)                                      # E4M3 holds them
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x, torch.ones(1, device=DEV), q)
    want = torch.where(sources >= 0, x[sources // top_k, 0], 0).to(torch.float8_e4m3fn) \
        .view(torch.uint8)
    offsets = plan.offsets.tolist()
    for part, a in zip(plan.segments(q, offsets), offsets):
        mine = want[a:a + part.rows]
        assert (part.data == mine[:, None]).all() and (part.data_t == mine).all()


def test_rows_far_apart():
    """A row stride past 2^23 elements, in every call that takes one: 4 rows of 2^24."""
    ids = _ids(4, 2, 3, 30, "all")
    plan, want = _plan(ids, 3), ref.plan(ids, 3)
    end = int(want[0][-1])
    wide = torch.empty(4, 1 << 24, dtype=BF16, device=DEV)
    x, x0 = wide[:, :64], _rand((4, 64), 31)
    x.copy_(x0)
    q, amax = dsl.Float8Tensor.empty(plan.rows, 64, dsl.E4M3), torch.zeros(1, device=DEV)
    dsl.fp8_expert_gather_cast_transpose_amax(plan, x, torch.ones(1, device=DEV), q, amax)
    y = ref.gather(bits16(x0), want[3], 2, end)
    codes, _, top, _ = oracle.cast_transpose_amax(y, 1.0, dsl.E4M3)
    np.testing.assert_array_equal(bits8(q.data[:end]), codes)
    assert float(amax) == float(top)
    rows = torch.zeros(plan.rows, 64, dtype=BF16, device=DEV)
    dsl.fp8_expert_gather(plan, x, rows)
    np.testing.assert_array_equal(bits16(rows[:end]), y)
    back = torch.empty(4, 64, dtype=BF16, device=DEV)
    dsl.fp8_expert_combine(plan, rows, back, base=x)
    assert torch.equal(back.cpu(), (3 * x0.float()).to(BF16))
    dw, dx = torch.zeros(4, 2, device=DEV), torch.zeros_like(rows)
    dsl.fp8_expert_combine_backward(plan, x, rows, dw, weights=torch.ones(4, 2, device=DEV), dx=dx)
    np.testing.assert_array_equal(bits16(dx[:end]), y)
    dot = (x0.double() ** 2).sum(1, keepdim=True)
    assert ((dw.cpu().double() - dot).abs() <= 65 * 2.0 ** -24 * dot).all()


@pytest.mark.parametrize("tokens, top_k, experts, cols", [
    (17, 3, 4, 528), (130, 6, 3, 1024), (257, 2, 9, 1032), (33, 9, 5, 4104)])
def test_weight_gradient_with_and_without_dx(tokens, top_k, experts, cols):
    """The same bits: the sums' order follows from the sizes alone."""
    ids = _ids(tokens, top_k, experts, 40)
    plan = _plan(ids, experts)
    dy, x = _rand((tokens, cols), 41).to(DEV), _rand((plan.rows, cols), 42).to(DEV)
    a, b = (torch.empty(tokens, top_k, device=DEV) for _ in range(2))
    dsl.fp8_expert_combine_backward(plan, dy, x, a)
    dsl.fp8_expert_combine_backward(plan, dy, x, b, weights=torch.rand(tokens, top_k, device=DEV),
                                    dx=torch.empty_like(x))
    assert torch.equal(a, b)
