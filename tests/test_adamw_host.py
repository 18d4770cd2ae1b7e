"""The optimizer on the CPU: the reference against torch's AdamW in float64, the
stochastic rounding's mean over all its numbers, and every refusal (nothing
reaches a device)."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import adamw_reference as ref

F = np.float32


def test_reference_against_torch():
    """Ten steps with weight decay.  The reference rounds m, v and the gradient's
    scaling to fp32: 8 roundings of 2^-24 a step in m or v, relative to their largest
    terms, and an update is a few of them away; 1e-5 of the update's size (lr per
    step) covers ten steps of it."""
    r = np.random.default_rng(0)
    n, lr, wd, b1, b2, eps = 500, 1e-2, 0.1, 0.9, 0.99, 1e-8
    p = r.standard_normal(n)
    t = torch.tensor(p, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)
    m, v = np.zeros(n, F), np.zeros(n, F)
    for step in range(1, 11):
        g = r.standard_normal(n).astype(F)
        t.grad = torch.tensor(g, dtype=torch.float64)
        opt.step()
        m, v, p, _ = ref.step(p, g, m, v, step, lr, wd, b1, b2, eps)
        assert np.abs(p - t.detach().numpy()).max() <= 1e-5 * lr * step


def test_mean_of_the_rounding():
    """Over all 65536 numbers the codes' mean is the value: the lower neighbour
    plus ceil or floor of place * 65536 of its 65536 parts, so within 2^-16 of the
    neighbours' distance."""
    r = np.random.default_rng(1)
    u = np.arange(65536)
    for y in np.concatenate([r.uniform(0, 448, 12), 2.0 ** r.uniform(-12, 8, 12), [448.0, 0.0]]):
        y = float(F(y))
        got = ref.VALUES[ref.place(np.full(u.size, y), u)]
        step = 2.0 ** (np.floor(np.log2(max(y, 2.0 ** -6))) - 3)
        assert abs(got.mean() - y) <= step * 2.0 ** -16 * 1.001
        assert got.max() - got.min() <= step * 1.001 and got.max() <= 448.0


def test_scales():
    x = np.zeros(4 * 256, F)
    x[0], x[256], x[512], x[768] = 448.0, 448.0000305, 1e-45, 3.4e38
    assert ref.scales_of(x).tolist() == [1.0, 2.0, 2.0 ** -126, 2.0 ** 120]
    assert (ref.VALUES[[0x7E, 0x01, 0x08]] == [448.0, 2.0 ** -9, 2.0 ** -6]).all()


def _tensor(param=0x10000, grad=0x20000, m=0x30000, v=0x40000, ms=None, vs=None, copy=None, n=100,
            wd=0.0, pd=1, gd=1, reserved=0):
    return dsl._AdamWTensorDesc(param, grad, m, v, ms, vs, copy, n, wd, pd, gd, reserved)


def _opt(lr=0x50000, steps=0x60000, b1=0.9, b2=0.999, eps=1e-8):
    return dsl._AdamWDesc(lr, steps, b1, b2, eps, 7)


def test_step_refusals():
    L = dsl.lib()

    def call(t=_tensor(), opt=_opt(), count=1, scale=None, flag=None, tensors=True):
        array = (dsl._AdamWTensorDesc * 2)(_tensor(), t) if tensors else None
        return L.fp8_adamw_step(None if opt is None else ctypes.byref(opt), array,
                                2 if count == 1 else count, scale, flag, None)

    assert call(opt=None) == -1 and call(tensors=False) == -1
    assert call(opt=_opt(lr=None)) == -1 and call(opt=_opt(steps=None)) == -1
    assert call(opt=_opt(lr=0x50002)) == -3 and call(opt=_opt(steps=0x60008)) == -3
    assert call(scale=0x70001) == -3 and call(flag=0x70002) == -3
    assert call(count=-1) == -5
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b1=float("nan")), dict(b2=1.0), dict(b2=-1e-9),
                dict(eps=0.0), dict(eps=-1e-8), dict(eps=1e-60), dict(eps=float("inf")),
                dict(eps=float("nan")), dict(eps=1e39), dict(eps=1.3e30), dict(eps=1.1e-38)):
        assert call(opt=_opt(**bad)) == -5, bad
    for bad in (dict(pd=2), dict(gd=-1), dict(reserved=1), dict(wd=-0.1), dict(wd=float("inf")),
                dict(wd=float("nan")), dict(copy=0x80000, pd=0), dict(ms=0x80000),
                dict(vs=0x80000)):
        assert call(t=_tensor(**bad)) == -5, bad
    assert call(t=_tensor(n=-1)) == -2 and call(t=_tensor(n=(1 << 34) + 1)) == -2
    for name in ("param", "grad", "m", "v"):
        assert call(t=_tensor(**{name: None})) == -1
        assert call(t=_tensor(**{name: 0x10008})) == -3
    assert call(t=_tensor(copy=0x80008)) == -3
    assert call(t=_tensor(ms=0x80002, vs=0x90000)) == -3
    assert call(t=_tensor(ms=0x80000, vs=0x90002)) == -3


def test_norm_refusals():
    L = dsl.lib()
    need = dsl.fp8_grad_norm_workspace_bytes()

    def call(g=0x10000, n=100, dtype=1, reserved=0, count=1, most=1.0, norm=0x20000, factor=None,
             flag=None, ws=0x30000, size=need, grads=True):
        array = (dsl._GradDesc * 1)((g, n, dtype, reserved)) if grads else None
        return L.fp8_grad_norm(array, count, most, norm, factor, flag, ws, size, None)

    for most in (0.0, -1.0, float("nan")):
        assert call(most=most) == -5
    assert call(count=-1) == -5 and call(dtype=2) == -5 and call(reserved=1) == -5
    assert call(norm=None) == -1 and call(ws=None) == -1 and call(grads=False) == -1
    assert call(g=None) == -1
    assert call(g=0x10008) == -3 and call(norm=0x20002) == -3 and call(factor=0x20002) == -3
    assert call(flag=0x20001) == -3 and call(ws=0x30008) == -3
    assert call(size=need - 1) == -2 and call(n=-1) == -2 and call(n=(1 << 34) + 1) == -2


def test_python_refusals():
    p, g = torch.zeros(300), torch.zeros(300)
    with pytest.raises(ValueError):
        dsl.AdamWTensor.zeros(p, g, bits=16)
    t = dsl.AdamWTensor.zeros(p, g, bits=8)
    assert t.m.dtype == torch.uint8 and t.m_scale.shape == (2,) and t.m_scale.sum() == 0
    with pytest.raises(ValueError):                     # not on a device
        t.desc()
    for change, error in ((dict(grad=None), ValueError), (dict(v=None), ValueError),
                          (dict(grad=g.double()), TypeError), (dict(param=p.half()), TypeError),
                          (dict(v_scale=None), ValueError),
                          (dict(param=p.bfloat16(), copy=p.bfloat16()), TypeError)):
        fields = dict(param=p, grad=g, m=t.m, v=t.v, m_scale=t.m_scale, v_scale=t.v_scale)
        with pytest.raises(error):
            dsl.AdamWTensor(**{**fields, **change}).desc()
    with pytest.raises(TypeError):
        dsl.fp8_grad_norm([g.half()], torch.zeros(1), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dsl.fp8_grad_norm([g], torch.zeros(0), torch.zeros(8, dtype=torch.uint8))


def test_assigned_steps_are_the_state():
    """A resumed run sets the count that the kernels read, and reads the one of a state
    that it puts in place."""
    opt = dsl.AdamW([], device="cpu")
    assert opt.steps.tolist() == [0] and opt.state.tolist() == [0] * (dsl.ADAMW_STATE_BYTES // 8)
    state = opt.state
    for taken in (500, torch.tensor([2 ** 33]), torch.tensor(7.0), torch.zeros(1, 1).int()):
        opt.steps = taken
        assert opt.state is state                       # what a captured step reads
        assert int(state[0]) == int(opt.steps) == int(taken) and not state[1:].any()
    opt.steps += 3
    assert int(state[0]) == 3
    for bad in (torch.zeros(2), torch.zeros(0)):
        with pytest.raises(ValueError, match="single"):
            opt.steps = bad
    opt.state = torch.arange(9, 9 + state.numel())
    assert opt.steps.tolist() == [9] and opt.steps.dtype == torch.int64
    opt.steps.fill_(4)
    assert int(opt.state[0]) == 4


def test_an_optimizer_is_copied_and_pickled(monkeypatch):
    """As a checkpoint does: a copy holds the state in tensors of its own, which are the
    same ones wherever the program has them, and descriptors of these."""
    monkeypatch.setattr(dsl, "_ptr", lambda t, dtype=None, what="": None if t is None else t.data_ptr())
    monkeypatch.setattr(dsl, "_on_current_device", lambda *tensors: None)
    monkeypatch.setattr(dsl, "_device", lambda: -1)
    param, grad = torch.randn(300), torch.randn(300)
    opt = dsl.AdamW([dsl.AdamWTensor.zeros(param, grad, 8, weight_decay=0.5)], lr=0.25,
                    betas=(0.5, 0.75), eps=1e-3, seed=9, device="cpu")
    opt.steps = 41
    opt.tensors[0].m[0] = 7
    array, count = opt._tensor_array()                  # as after a step
    assert count == 1 and array[0].param == param.data_ptr()
    deep = copy.deepcopy({"opt": opt, "param": param})
    for other in (deep["opt"], pickle.loads(pickle.dumps(opt))):
        assert (int(other.steps), float(other.lr), other.betas, other.eps, other.seed) \
            == (41, 0.25, (0.5, 0.75), 1e-3, 9)
        mine, its = opt.tensors[0], other.tensors[0]
        array, count = other._tensor_array()
        assert count == 1 and array[0].n == 300 and array[0].weight_decay == 0.5
        for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
            a, b = getattr(mine, name), getattr(its, name)
            assert torch.equal(a, b) and a.data_ptr() != b.data_ptr()
            assert getattr(array[0], name) == b.data_ptr()
        other.steps += 1
        assert int(other.state[0]) == 42 and int(opt.state[0]) == 41
    assert deep["opt"].tensors[0].param is deep["param"]
    assert copy.copy(opt.tensors[0]).param is param
    assert opt._tensor_array()[0][0].param == param.data_ptr()
    empty = copy.deepcopy(dsl.AdamW([], device="cpu"))
    assert empty._tensor_array()[1] == 0 and len(empty._tensor_array()[0]) == 0


def test_tensors_share_nothing_that_is_written(monkeypatch):
    """A parameter listed twice (tied weights), moments in each other's place and a
    gradient within a parameter race on the device and are refused; pieces of one
    buffer, a shared gradient and a gradient that its own copy replaces are not."""
    monkeypatch.setattr(dsl, "_ptr", lambda t, dtype=None, what="": None if t is None else t.data_ptr())
    monkeypatch.setattr(dsl, "_on_current_device", lambda *tensors: None)
    monkeypatch.setattr(dsl, "_device", lambda: -1)
    flat, grads = torch.zeros(4 * 512), torch.zeros(4 * 512)
    make = lambda i, **kw: dsl.AdamWTensor.zeros(flat[512 * i:][:512], grads[512 * i:][:512], **kw)
    opt = dsl.AdamW([make(0), make(1, bits=8), make(2), make(3, bits=8)], device="cpu")
    assert opt._tensor_array()[1] == 4
    opt.tensors[2].grad = opt.tensors[0].grad           # read only
    b16 = torch.zeros(512, dtype=torch.bfloat16)
    opt.tensors[3].grad = opt.tensors[3].copy = b16     # read before it is written
    assert opt._tensor_array()[1] == 4

    def refused(what):
        for _ in range(2):                              # the second call looks again
            with pytest.raises(ValueError, match=what):
                opt._tensor_array()

    a, b, c, d = opt.tensors
    opt.tensors = [a, b, c, d, a]
    refused("share")
    for t, name, bad, what in (
            (c, "param", a.param, "share"), (c, "v", c.m, "share"), (c, "m", a.m, "share"),
            (b, "v_scale", d.m_scale, "share"), (c, "param", flat[768:][:512], "share"),
            (a, "copy", b16, "share"), (c, "grad", b.param, "grad"),
            (c, "grad", flat[4:][:512], "grad"), (b, "grad", b16, "grad"),
            (a, "param", grads[512:][:512], "grad"),    # another tensor's gradient
            (d, "copy", torch.zeros(516, dtype=torch.bfloat16)[4:], None)):
        opt.tensors, old = [a, b, c, d], getattr(t, name)
        assert opt._tensor_array()[1] == 4
        setattr(t, name, bad)
        refused(what) if what else opt._tensor_array()
        setattr(t, name, old)
    half = torch.zeros(1024, dtype=torch.bfloat16)
    d.grad, d.copy = half[:512], half[8:][:512]
    refused("grad")
    opt.tensors = [dsl.AdamWTensor.zeros(flat[:0], flat[:0])] * 2
    assert opt._tensor_array()[1] == 2                  # nothing is written


def test_assigned_learning_rate():
    """A number goes where captured steps read it, a tensor takes its place."""
    opt = dsl.AdamW([], lr=0.5, device="cpu")
    lr = opt.lr
    opt.lr = 0.25
    assert opt.lr is lr and lr.tolist() == [0.25] and lr.dtype == torch.float32
    opt.lr *= 0.5
    assert opt.lr is lr and lr.tolist() == [0.125]
    schedule = torch.tensor([2.0])
    opt.lr = schedule
    assert opt.lr is schedule
    opt.lr = 3
    assert schedule.tolist() == [3.0] and lr.tolist() == [0.125]


def test_a_new_gradient_is_checked(monkeypatch):
    """Between steps a gradient may be another tensor, of the other type too; one that
    the step does not take is refused as at the first step, and the rest is not stale."""
    monkeypatch.setattr(dsl.torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(dsl, "_on_current_device", lambda *tensors: None)
    monkeypatch.setattr(dsl, "_device", lambda: -1)
    param = torch.zeros(4, 75)
    t = dsl.AdamWTensor.zeros(param, torch.zeros(4, 75), 8, weight_decay=0.5)
    first = t.desc()
    assert t.desc() is first and first.grad_dtype == 1
    for dtype, code in ((torch.bfloat16, 0), (torch.float32, 1)):
        t.grad = torch.zeros(4, 75, dtype=dtype)
        d = t.desc()
        assert d is not first and t.desc() is d
        assert (d.grad, d.grad_dtype) == (t.grad.data_ptr(), code)
        for name, _ in d._fields_:
            if name not in ("grad", "grad_dtype"):
                assert getattr(d, name) == getattr(first, name), name
    good = t.grad
    for bad, error in ((None, ValueError), (torch.zeros(4, 76), ValueError),
                       (torch.zeros(4, 75, dtype=torch.float64), TypeError),
                       (torch.zeros(75, 4).t(), ValueError), (torch.zeros(75 * 4), ValueError)):
        t.grad = bad
        with pytest.raises(error, match="grad"):
            t.desc()
        t.grad = good
        assert t.desc().grad == good.data_ptr()
    t.grad, t.weight_decay = torch.zeros(4, 75), 0.25
    assert (t.desc().grad, t.desc().weight_decay) == (t.grad.data_ptr(), 0.25)
    t.grad, t.v = torch.zeros(4, 75), torch.zeros(4, 75, dtype=torch.uint8)
    assert (t.desc().grad, t.desc().v) == (t.grad.data_ptr(), t.v.data_ptr())


def test_shared_spans_by_brute_force():
    """Every pair of spans, over small random layouts: half of them overlap."""
    r = np.random.default_rng(2)
    overlap = lambda a, b: max(a[0], b[0]) < min(a[1], b[1])
    refused, layouts = 0, 4000
    for _ in range(layouts):
        opt, mine = dsl.AdamW([], device="cpu"), []
        for _ in range(r.integers(1, 5)):
            t = dsl.AdamWTensor(None, None, None, None)
            starts = r.integers(0, 60, r.integers(0, 3)).tolist()
            spans = [(a, a + int(r.integers(1, 9))) for a in starts]
            a = int(r.integers(0, 60))
            grad = spans[0] if spans and r.random() < 0.2 else (a, a + int(r.integers(0, 9)))
            t._seen = (0.0, 0, (), (), None, tuple(x for s in spans for x in s), grad)
            opt.tensors.append(t)
            mine.append((spans, grad))
        every = [(i, s) for i, (spans, _) in enumerate(mine) for s in spans]
        bad = any(overlap(s, t) for k, (_, s) in enumerate(every) for _, t in every[:k]) or \
            any(overlap(g, s) and not (i == j and s == g)
                for j, (_, g) in enumerate(mine) for i, s in every)
        refused += bad
        for _ in range(2):                              # a refused call is looked at again
            try:
                opt._need_separate(range(len(mine)))
                assert not bad
            except ValueError:
                assert bad
    assert 0.3 < refused / layouts < 0.7
