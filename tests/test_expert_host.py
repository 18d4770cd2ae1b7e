"""Expert routing on the CPU: the reference against differences, sizes of plans
and buffers, and every refusal (nothing reaches a device)."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import expert_reference as ref


def test_reference_gradients_against_differences():
    """sum(dy * combine(...)) is linear in x and in w: a central difference has no
    truncation error, 1e-9 covers float64 rounding of sums of about 1e3 terms."""
    r = np.random.default_rng(0)
    tokens, top_k, experts, cols = 7, 3, 4, 16
    ids = r.integers(-1, experts + 1, (tokens, top_k))
    for capacity in (0, 16):
        _, _, slots, sources = ref.plan(ids, experts, capacity)
        x, dy = r.standard_normal((sources.size, cols)), r.standard_normal((tokens, cols))
        w, base = r.standard_normal((tokens, top_k)), r.standard_normal((tokens, cols))
        loss = lambda x, w: float((dy * ref.combine(x, slots, w, base)[0]).sum())
        dw = ref.combine_weight_gradient(dy, x, slots)[0]
        dx = np.zeros_like(x)
        for s, pair in enumerate(sources):
            if pair >= 0:
                dx[s] = w.reshape(-1)[pair] * dy[pair // top_k]
        for which, grad in ((0, dx), (1, dw)):
            for at in r.integers(0, grad.size, 30):
                step = np.zeros(grad.size)
                step[at] = 1.0
                step = step.reshape(grad.shape)
                up = loss(x + step, w) if which == 0 else loss(x, w + step)
                down = loss(x - step, w) if which == 0 else loss(x, w - step)
                assert abs((up - down) / 2 - grad.ravel()[at]) < 1e-9
        # The gather's gradient is the combine without weights.
        gathered = np.where((sources >= 0)[:, None], dy[np.maximum(sources, 0) // top_k], 0.0)
        assert abs((gathered * x).sum() - (dy * ref.combine(x, slots)[0]).sum()) < 1e-9


def test_rows_and_plan_sizes():
    for tokens, top_k, experts, capacity in ((0, 1, 1, 0), (0, 8, 64, 32), (1, 1, 1024, 0),
                                             (64, 8, 64, 0), (8192, 2, 8, 2560),
                                             (1 << 23, 1, 1, 0), (1 << 17, 64, 1024, 16384)):
        rows = ref.rows_of(tokens, top_k, experts, capacity)
        assert dsl.fp8_expert_rows(tokens, top_k, experts, capacity) == rows
        n = dsl.fp8_expert_plan_bytes(tokens, top_k, experts, capacity)
        assert n >= 4 * (tokens * top_k + rows + 2 * experts + 1)
        p = dsl.ExpertPlan.empty(tokens, top_k, experts, capacity, device="meta")
        assert p.rows == rows and p.buf.numel() == n
        ends = [(v.storage_offset() * v.element_size() + v.numel() * 4)
                for v in (p.offsets, p.counts, p.slots, p.sources)]
        assert max(ends) <= n
    for bad in ((-1, 1, 1, 0), (1, 0, 1, 0), (1, 65, 1, 0), (1, 1, 0, 0), (1, 1, 1025, 0),
                ((1 << 23) + 1, 1, 1, 0), (1 << 22, 3, 1, 0), (1, 1, 1, -16), (1, 1, 1, 8),
                (1, 1, 1, (1 << 24) + 16), (1, 1, 1024, (1 << 14) + 16)):
        with pytest.raises(dsl.Fp8Error):
            dsl.fp8_expert_rows(*bad)
        with pytest.raises(dsl.Fp8Error):
            dsl.fp8_expert_plan_bytes(*bad)


def test_every_batch_fits_its_rows():
    """The rows that the sizes fix hold the segments of any ids: those of many
    random batches, and the worst one (every expert one pair past a multiple of 16)."""
    r = np.random.default_rng(1)
    for _ in range(200):
        tokens, top_k, experts = (int(r.integers(1, n)) for n in (60, 5, 40))
        ids = r.integers(0, experts, (tokens, top_k))
        assert ref.plan(ids, experts)[0][-1] <= ref.rows_of(tokens, top_k, experts, 0)
    ids = np.repeat(np.arange(20), 17).reshape(-1, 1)
    assert ref.plan(ids, 20)[0][-1] == 20 * 32 == ref.rows_of(340, 1, 20, 0)


SIZES = (64, 2, 8, 0)


def _sizes(tokens=64, top_k=2, experts=8, capacity=0):
    return ctypes.byref(dsl._ExpertSizes(tokens, capacity, top_k, experts))


NEED = dsl.fp8_expert_plan_bytes(*SIZES)
ROWS = dsl.fp8_expert_rows(*SIZES)
PLAN, X, Y, W, B = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def test_plan_refusals():
    L = dsl.lib()
    call = lambda s=_sizes(), ids=X, plan=PLAN, size=NEED: L.fp8_expert_plan(s, ids, plan, size, None)
    assert call(s=None) == -1 and call(ids=None) == -1 and call(plan=None) == -1
    assert call(s=_sizes(tokens=-1)) == -2 and call(s=_sizes(top_k=65)) == -2
    assert call(s=_sizes(experts=1025)) == -2 and call(s=_sizes(capacity=24)) == -2
    assert call(ids=X + 2) == -3 and call(plan=PLAN + 8) == -3
    assert call(size=NEED - 1) == -2
    assert L.fp8_expert_plan_layout(_sizes(), None) == -1
    assert L.fp8_expert_rows(None) == -1 and L.fp8_expert_plan_bytes(None) == -1


def _common(call):
    """What every call with a plan refuses."""
    assert call(s=None) == -1 and call(plan=None) == -1
    assert call(plan=PLAN + 4) == -3 and call(size=NEED - 1) == -2
    assert call(s=_sizes(experts=0)) == -2
    for cols in (-8, 12, (1 << 22) + 8):
        assert call(cols=cols) == -2
    assert call(ldx=56) == -2 and call(ldx=68) == -2 and call(ldx=1 << 30) == -2
    assert call(x=None) == -1 and call(x=X + 8) == -3


def test_gather_refusals():
    L = dsl.lib()
    call = lambda s=_sizes(), plan=PLAN, size=NEED, x=X, ldx=64, y=Y, ldy=64, cols=64: \
        L.fp8_expert_gather(s, plan, size, x, ldx, y, ldy, cols, None)
    _common(call)
    assert call(y=None) == -1 and call(y=Y + 8) == -3 and call(ldy=56) == -2 and call(ldy=68) == -2
    # Nothing to do.
    assert call(cols=0, x=None, y=None) == 0
    none = _sizes(tokens=0)
    assert call(s=none, size=1 << 20, x=None, y=None) == 0


def test_gather_cast_refusals():
    L = dsl.lib()

    def desc(rows=ROWS, cols=64, fmt=0, data=0x60000, data_t=0x70000, sinv=0x80000):
        return ctypes.byref(dsl._Desc(data, data_t, sinv, fmt, 0, rows, cols))

    call = lambda s=_sizes(), plan=PLAN, size=NEED, x=X, ldx=64, cols=64, w=W, scale=0x90000, \
        out=desc(): L.fp8_expert_gather_cast_transpose_amax(s, plan, size, x, ldx, cols, w, scale,
                                                            out, None, None, None)
    assert call(s=None) == -1 and call(plan=None) == -1 and call(size=NEED - 1) == -2
    assert call(plan=PLAN + 4) == -3
    assert call(x=None) == -1 and call(x=X + 8) == -3 and call(w=W + 2) == -3
    assert call(scale=None) == -1 and call(out=None) == -1
    assert call(out=desc(rows=ROWS - 16)) == -2 and call(out=desc(cols=80)) == -2
    assert call(out=desc(fmt=2)) == -4 and call(out=desc(data=0, data_t=0)) == -1
    assert call(out=desc(data=0x60008)) == -3 and call(out=desc(data_t=0x70008)) == -3
    assert call(cols=72, ldx=72, out=desc(cols=72)) == -2          # not a multiple of 16
    assert call(ldx=48) == -2 and call(ldx=1 << 30) == -2
    # 2^24 tiles over all segments.
    big = dict(tokens=1 << 20, top_k=8, experts=8)
    rows = dsl.fp8_expert_rows(1 << 20, 8, 8)
    assert call(s=_sizes(**big), size=1 << 40, cols=1 << 15, ldx=1 << 15,
                out=desc(rows=rows, cols=1 << 15)) == -2


def test_combine_refusals():
    L = dsl.lib()
    call = lambda s=_sizes(), plan=PLAN, size=NEED, x=X, ldx=64, w=W, base=B, ldbase=64, y=Y, \
        ldy=64, cols=64: L.fp8_expert_combine(s, plan, size, x, ldx, w, base, ldbase, y, ldy, cols,
                                              None)
    _common(call)
    assert call(y=None) == -1 and call(y=Y + 8) == -3 and call(ldy=56) == -2
    assert call(base=B + 8) == -3 and call(ldbase=56) == -2 and call(w=W + 2) == -3
    assert call(cols=0, x=None, y=None) == 0
    assert call(s=_sizes(tokens=0), size=1 << 20, x=None, y=None) == 0


def test_combine_backward_refusals():
    L = dsl.lib()
    call = lambda s=_sizes(), plan=PLAN, size=NEED, dy=B, lddy=64, x=X, ldx=64, w=W, dw=0x60000, \
        dx=Y, lddx=64, cols=64: L.fp8_expert_combine_backward(s, plan, size, dy, lddy, x, ldx, w,
                                                              dw, dx, lddx, cols, None)
    _common(call)
    assert call(dy=None) == -1 and call(dy=B + 8) == -3 and call(lddy=56) == -2
    assert call(dw=None) == -1 and call(dw=0x60002) == -3
    assert call(w=None) == -1 and call(w=W + 2) == -3
    assert call(dx=Y + 8) == -3 and call(lddx=56) == -2
    assert call(s=_sizes(tokens=0), size=1 << 20, dy=None, x=None, dw=None, dx=None) == 0


def test_python_refusals():
    plan = dsl.ExpertPlan.empty(4, 2, 3, device="cpu")
    x, y = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(plan.rows, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                     # shape of the ids
        dsl.fp8_expert_plan(torch.zeros(4, 3, dtype=torch.int32), plan)
    with pytest.raises(ValueError):                     # not on a device
        dsl.fp8_expert_plan(torch.zeros(4, 2, dtype=torch.int32), plan)
    with pytest.raises(ValueError):                     # 1-D
        dsl.fp8_expert_gather(plan, x[0], y)
    with pytest.raises(ValueError):                     # rows of y
        dsl.fp8_expert_gather(plan, x, y[:-1])
    with pytest.raises(TypeError):
        dsl.fp8_expert_gather(plan, x.float(), y)
    with pytest.raises(ValueError):                     # dx without weights
        dsl.fp8_expert_combine_backward(plan, x.to("meta"), y.to("meta"), None, dx=y.to("meta"))


def test_a_plan_keeps_its_sizes():
    """The shapes that the calls check and the sizes that the kernels use are the same."""
    plan = dsl.ExpertPlan.empty(4, 2, 3, device="cpu")
    for name, value in (("tokens", 5), ("top_k", 3), ("experts", 4), ("capacity", 16), ("rows", 8)):
        with pytest.raises(ValueError, match="sizes"):
            setattr(plan, name, value)
    plan.built = True
    assert dsl.ExpertPlan(plan.buf, 4, 2, 3).rows == plan.rows
    with pytest.raises(ValueError, match="built"):
        dsl._expert_call(dsl.ExpertPlan.empty(4, 2, 3, device="cpu"))


def test_segments():
    """Each expert's part of a tensor in expert order."""
    plan = dsl.ExpertPlan.empty(40, 1, 3, device="cpu")
    assert plan.rows == 80
    q = dsl.Float8Tensor(torch.arange(80 * 16).to(torch.uint8).view(80, 16),
                         torch.arange(80 * 16).to(torch.uint8).view(16, 80), torch.ones(1), 0, 80,
                         16)
    with pytest.raises(ValueError):
        plan.segments(q)
    parts = plan.segments(q, [0, 32, 32, 48])
    assert [(p.rows, p.cols) for p in parts] == [(32, 16), (0, 16), (16, 16)]
    for p, first in zip(parts, (0, 32, 32)):
        assert p.data.shape == (p.rows, 16) and p.data_t.shape == (16, p.rows)
        assert torch.equal(p.data, q.data[first:first + p.rows])
        assert torch.equal(p.data_t.reshape(-1), q.data_t.view(-1)[first * 16:(first + p.rows) * 16])
        assert p.data_t.is_contiguous() and p.scale_inv is q.scale_inv
    fixed = dsl.ExpertPlan.empty(40, 1, 3, 32, device="cpu")
    assert [p.rows for p in fixed.segments(dsl.Float8Tensor(None, None, torch.ones(1), 0, 96, 16))] \
        == [32, 32, 32]
    with pytest.raises(ValueError):
        fixed.segments(q)


@pytest.mark.parametrize("capacity", [0, 32])
def test_a_plan_is_copied_and_pickled(capacity):
    """As part of a module it is: a copy has the sizes and a buffer and views of its own."""
    plan = dsl.ExpertPlan.empty(40, 2, 3, capacity, device="cpu")
    plan.buf.copy_((torch.arange(plan.buf.numel()) % 251).to(torch.uint8))
    plan.built = True
    offsets = plan.offsets
    for other in (copy.deepcopy(plan), pickle.loads(pickle.dumps(plan)), copy.copy(plan)):
        assert (other.tokens, other.top_k, other.experts, other.capacity, other.rows, other.built) \
            == (40, 2, 3, capacity, plan.rows, True)
        assert torch.equal(other.buf, plan.buf) and torch.equal(other.offsets, offsets)
        sizes = other._sizes._obj
        assert (sizes.tokens, sizes.top_k, sizes.experts, sizes.capacity) == (40, 2, 3, capacity)
        with pytest.raises(ValueError, match="sizes"):
            other.tokens = 41
    deep = copy.deepcopy({"plan": plan, "buf": plan.buf})
    assert deep["plan"].buf is deep["buf"] and deep["buf"].data_ptr() != plan.buf.data_ptr()
    deep["buf"].zero_()
    assert not deep["plan"].offsets.any() and torch.equal(plan.offsets, offsets)


def test_views_follow_the_buffer():
    """A buffer given other memory in place, or replaced, is the one that is seen."""
    plan = dsl.ExpertPlan.empty(40, 2, 3, device="cpu")
    plan.buf.zero_()
    assert plan.offsets.tolist() == [0, 0, 0, 0] and plan.offsets is plan.offsets
    for change in (lambda b: setattr(plan.buf, "data", b), lambda b: plan.buf.set_(b),
                   lambda b: setattr(plan, "buf", b)):
        new = plan.buf + 1
        change(new)
        assert plan.offsets.data_ptr() - plan.buf.data_ptr() == plan._layout.offsets
        assert torch.equal(plan.slots.view(torch.uint8).unique(), new.unique())


def test_gather_cast_takes_the_gathers_strides():
    """Every stride that fp8_expert_gather takes.  (The weights' misalignment, looked at
    last, ends the call before anything reaches a device.)"""
    L = dsl.lib()
    out = ctypes.byref(dsl._Desc(0x60000, 0x70000, 0x80000, 0, 0, ROWS, 64))
    for ldx, want in ((64, -3), ((1 << 23) - 8, -3), (1 << 23, -3), (1 << 24, -3),
                      ((1 << 30) - 8, -3), (1 << 30, -2), (56, -2), (68, -2)):
        assert L.fp8_expert_gather_cast_transpose_amax(
            _sizes(), PLAN, NEED, X, ldx, 64, W + 2, 0x90000, out, None, None, None) == want, ldx
