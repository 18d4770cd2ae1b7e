"""The adapters on the CPU: the reference's gradients against differences,
sizes of plans and workspaces, and every refusal (nothing reaches a device)."""
import ctypes

import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import op_reference as ref


def test_reference_gradients_against_differences():
    """sum(dy * y) is linear in each of x, A and B, so a central difference
    has no truncation error: 1e-9 covers float64 rounding of sums of about
    1e3 terms over a step of 1."""
    r = np.random.default_rng(0)
    rows, k, n, rank, count = 11, 16, 24, 8, 3
    x, dy = r.standard_normal((rows, k)), r.standard_normal((rows, n))
    a, b = r.standard_normal((count, rank, k)), r.standard_normal((count, n, rank))
    alpha, ids = r.standard_normal(count), np.array([0, 2, -1, 0, 2, 2, 7, 0, 0, -1, 2])
    mask, f = ref.keep_mask(rows, k, 0.3, 5, 6), float(ref.factor(0.3))
    loss = lambda x, a, b: float((dy * ref.adapter_forward(x, a, b, alpha, ids, None, mask, f)[0]).sum())
    h = ref.adapter_forward(x, a, b, alpha, ids, None, mask, f)[1]
    dx, da, db, _ = ref.adapter_backward(x, a, b, alpha, ids, dy, h, None, mask, f)
    for which, grad in ((0, dx), (1, da), (2, db)):
        args = [x, a, b]
        for at in r.integers(0, grad.size, 40):
            step = np.zeros(grad.size)
            step[at] = 1.0
            step = step.reshape(grad.shape)
            up = loss(*[v + step if i == which else v for i, v in enumerate(args)])
            down = loss(*[v - step if i == which else v for i, v in enumerate(args)])
            assert abs((up - down) / 2 - grad.ravel()[at]) < 1e-9
    assert (da[1] == 0).all() and (db[1] == 0).all()               # no row of its own


def test_sizes():
    assert dsl.fp8_adapter_plan_bytes(0, 1) >= 0
    for rows, adapters in ((1, 1), (1, 4096), (33, 2), (8192, 9), (1 << 20, 64)):
        groups = min(adapters + 1, rows)
        # every row of its own group's last tile: the most tiles there can be
        tiles = (rows + 31 * groups) // 32
        assert dsl.fp8_adapter_plan_bytes(rows, adapters) >= 4 * (33 * tiles + 2 * adapters)
        assert dsl.fp8_adapter_workspace_bytes(rows, adapters, 16, 2048, 2048) >= rows * 16 * 4
    # more rows or ranks never ask for less
    w = dsl.fp8_adapter_workspace_bytes
    assert w(64, 8, 16, 256, 256) <= w(64, 8, 128, 256, 256)
    for bad in ((-1, 1, 16, 64, 64), ((1 << 26) + 1, 1, 16, 64, 64), (8, 0, 16, 64, 64),
                (8, 4097, 16, 64, 64), (8, 1, 0, 64, 64), (8, 1, 12, 64, 64), (8, 1, 136, 64, 64),
                (8, 1, 16, 0, 64), (8, 1, 16, 60, 64), (8, 1, 16, 64, 4), (8, 1, 16, 64, 1 << 23)):
        with pytest.raises(dsl.Fp8Error):
            w(*bad)
    for bad in ((-1, 1), ((1 << 26) + 1, 1), (1, 0), (1, 5000)):
        with pytest.raises(dsl.Fp8Error):
            dsl.fp8_adapter_plan_bytes(*bad)


def test_plan_refusals():
    L = dsl.lib()
    need = dsl.fp8_adapter_plan_bytes(16, 4)
    call = lambda ids=0x1000, rows=16, adapters=4, plan=0x2000, size=need: L.fp8_adapter_plan(
        ids, rows, adapters, plan, size, None)
    assert call(rows=-1) == -2 and call(adapters=0) == -2 and call(adapters=4097) == -2
    assert call(ids=None) == -1 and call(plan=None) == -1
    assert call(ids=0x1002) == -3 and call(plan=0x2008) == -3
    assert call(size=need - 1) == -2
    assert call(rows=0) == 0 and call(rows=0, ids=None, plan=None, size=0) == 0


def _w(a=0x10000, b=0x20000, alpha=0x30000, count=4, rank=16, n_in=64, n_out=128):
    return dsl._AdaptersDesc(a, b, alpha, count, rank, n_in, n_out)


def _drop(p=0.1, rng=0x8000, reserved=0):
    return ctypes.byref(dsl._DropoutDesc(rng, p, reserved))


PLAN = 0x40000
WS = 0x50000


def test_forward_refusals():
    L = dsl.lib()
    size = dsl.fp8_adapter_plan_bytes(16, 4)
    ws_size = dsl.fp8_adapter_workspace_bytes(16, 4, 16, 64, 128)

    def call(w=None, plan=PLAN, plan_size=size, drop=None, x=0x1000, ldx=64, base=0x2000, ldb=128,
             y=0x3000, ldy=128, rows=16, h=None, ws=WS, ws_bytes=ws_size):
        return L.fp8_adapter_fwd(ctypes.byref(w or _w()), plan, plan_size, drop, x, ldx, base, ldb,
                                 y, ldy, rows, h, ws, ws_bytes, None)

    assert L.fp8_adapter_fwd(None, PLAN, size, None, 0x1000, 64, None, 0, 0x3000, 128, 16, None, WS,
                             ws_size, None) == -1
    for w in (_w(count=0), _w(count=4097), _w(rank=4), _w(rank=20), _w(rank=136), _w(n_in=60),
              _w(n_in=0), _w(n_out=4), _w(n_out=1 << 23)):
        assert call(w) == -2
    assert call(rows=-1) == -2
    for w in (_w(a=0), _w(b=0), _w(alpha=0)):
        assert call(w) == -1
    assert call(plan=None) == -1 and call(ws=None) == -1
    assert call(_w(a=0x10008)) == -3 and call(_w(alpha=0x30002)) == -3
    assert call(plan=PLAN + 8) == -3 and call(ws=WS + 4) == -3
    assert call(plan_size=size - 1) == -2 and call(ws_bytes=ws_size - 1) == -2
    assert call(drop=_drop(p=1.0)) == -5 and call(drop=_drop(rng=0)) == -1
    assert call(drop=_drop(rng=0x8001)) == -3
    assert call(ldx=56) == -2 and call(ldx=68) == -2 and call(ldb=120) == -2 and call(ldy=132) == -2
    assert call(ldx=1 << 62) == -2
    assert call(x=None) == -1 and call(y=None) == -1
    assert call(x=0x1008) == -3 and call(base=0x2002) == -3 and call(y=0x3008) == -3
    assert call(h=0x6004) == -3
    assert call(rows=0) == 0 and call(rows=0, x=None, y=None, plan=None, ws=None) == 0


def test_backward_refusals():
    L = dsl.lib()
    size = dsl.fp8_adapter_plan_bytes(16, 4)
    ws_size = dsl.fp8_adapter_workspace_bytes(16, 4, 16, 64, 128)

    def call(w=None, plan=PLAN, plan_size=size, drop=None, x=0x1000, ldx=64, dy=0x2000, lddy=128,
             h=0x3000, base=0x4000, ldb=64, dx=0x5000, lddx=64, rows=16, da=0x6000, db=0x7000,
             dtype=1, ws=WS, ws_bytes=ws_size):
        return L.fp8_adapter_backward(ctypes.byref(w or _w()), plan, plan_size, drop, x, ldx, dy,
                                      lddy, h, base, ldb, dx, lddx, rows, da, db, dtype, ws,
                                      ws_bytes, None)

    assert call(_w(rank=12)) == -2 and call(_w(a=0)) == -1
    assert call(plan_size=size - 1) == -2 and call(ws_bytes=ws_size - 1) == -2
    assert call(dtype=2) == -5
    assert call(da=None) == -5 and call(db=None) == -5
    assert call(lddy=120) == -2 and call(ldx=60) == -2 and call(lddx=60) == -2 and call(ldb=56) == -2
    assert call(dy=None) == -1 and call(x=None) == -1 and call(h=None) == -1
    assert call(dy=0x2008) == -3 and call(x=0x1008) == -3 and call(h=0x3004) == -3
    assert call(dx=0x5008) == -3 and call(base=0x4008) == -3
    assert call(da=0x6008) == -3 and call(db=0x7004) == -3
    assert call(drop=_drop(p=float("nan"))) == -5
    # nothing asked for, or no rows and no gradients to clear
    assert call(dx=None, da=None, db=None, x=None, h=None, ldx=0) == 0
    assert call(rows=0, da=None, db=None) == 0


def test_binding_refusals():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    w = dsl.Adapters(bf(2, 16, 64), bf(2, 128, 16), torch.ones(2))
    plan = dsl.AdapterPlan(torch.zeros(4, dtype=torch.uint8), 8, 2)
    with pytest.raises(ValueError, match="3-D"):
        dsl.Adapters(bf(16, 64), bf(2, 128, 16), torch.ones(2)).desc()
    with pytest.raises(ValueError, match="Adapters.b"):
        dsl.Adapters(bf(2, 16, 64), bf(2, 128, 8), torch.ones(2)).desc()
    with pytest.raises(ValueError, match="alpha"):
        dsl.Adapters(bf(2, 16, 64), bf(2, 128, 16), torch.ones(3)).desc()
    with pytest.raises(ValueError, match="row_adapter"):
        dsl.fp8_adapter_plan(torch.zeros(7, dtype=torch.int32), plan)
    with pytest.raises(ValueError, match="not been built"):
        dsl._adapter_call(w, plan, None, None)
    plan.built = True
    with pytest.raises(ValueError, match="2 adapters, the call has 3"):
        dsl._adapter_call(dsl.Adapters(bf(3, 16, 64), bf(3, 128, 16), torch.ones(3)), plan, None,
                          None)
    with pytest.raises(ValueError, match="workspace is required"):
        dsl._adapter_call(w, plan, None, None)
    with pytest.raises(ValueError, match="x must have shape"):          # the plan's rows
        dsl.fp8_adapter_fwd(w, plan, bf(9, 64), None, bf(9, 128))
    with pytest.raises(Exception, match="cannot assign"):               # handles do not change
        w.a = bf(2, 16, 64)
    with pytest.raises(ValueError, match="device tensor"):
        dsl.fp8_adapter_fwd(w, plan, bf(8, 64), None, bf(8, 128))
    with pytest.raises(ValueError, match="x must have shape"):
        dsl.fp8_adapter_fwd(w, plan, bf(8, 72), None, bf(8, 128))
    with pytest.raises(ValueError, match="dy must have shape"):
        dsl.fp8_adapter_backward(w, plan, bf(8, 64), bf(8, 120))
    with pytest.raises(ValueError, match="overlap"):       # not even the input itself
        dsl._need_apart((0x1000, 64), (0x1000, 64), 8, 64, 64, 2, "y")
