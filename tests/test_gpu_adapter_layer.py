"""The operators as a fine-tuning and a serving step use them together: a
frozen FP8 linear with its adapters beside it, dropout on the adapters' input
and on the branch that joins the residual stream, the next linear's input cast
in the same pass, and the way back.

Every stage is checked against its reference on the inputs that it really had
(the stage before it on the GPU), so no error adds up; the chain captured in a
graph equals the chain run eagerly, bit for bit."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
import oracle
import workloads
from tests import op_reference as ref
from tests.gpu_util import DEV, assert_gemm_close, bf16_values, bits8, bits16, f32

pytestmark = pytest.mark.gpu

ROWS, HIDDEN, RANK, COUNT = 208, 256, 16, 3
P_IN, P_OUT = 0.1, 0.2


class Layer:
    """One linear [HIDDEN, HIDDEN] with adapters, its inputs and every buffer of a step."""

    def __init__(self):
        bf = lambda shape, std, seed: workloads.normal_bf16(shape, std, seed).to(DEV)
        self.x, self.residual = bf((ROWS, HIDDEN), 1.0, 900), bf((ROWS, HIDDEN), 1.0, 901)
        self.weight, self.bias = bf((HIDDEN, HIDDEN), 0.05, 902), bf((HIDDEN,), 0.05, 903)
        self.w = dsl.Adapters(bf((COUNT, RANK, HIDDEN), 0.06, 904),
                              bf((COUNT, HIDDEN, RANK), 0.06, 905),
                              torch.tensor([1.0, 0.5, 2.0], device=DEV))
        ids = np.random.default_rng(1).integers(-1, COUNT, ROWS)
        self.ids = torch.tensor(ids, dtype=torch.int32, device=DEV)
        self.plan = dsl.AdapterPlan.empty(ROWS, COUNT)
        self.ws = torch.empty(dsl.fp8_adapter_workspace_bytes(ROWS, COUNT, RANK, HIDDEN, HIDDEN),
                              dtype=torch.uint8, device=DEV)
        self.rng = torch.tensor([[11, 0], [12, 0]], device=DEV)       # two dropout sites
        self.drop_in = dsl.Dropout(P_IN, self.rng[0])
        self.drop_out = dsl.Dropout(P_OUT, self.rng[1])
        self.state = dsl.DelayedScalingState([dsl.E4M3, dsl.E4M3, dsl.E4M3, dsl.E5M2], device=DEV)
        self.state.scale.copy_(torch.tensor([60.0, 2000.0, 60.0, 4.0e4]))
        q = lambda fmt: dsl.Float8Tensor.empty(ROWS, HIDDEN, fmt)
        self.qx, self.qz, self.qdy = q(dsl.E4M3), q(dsl.E4M3), q(dsl.E5M2)
        self.qw = dsl.Float8Tensor.empty(HIDDEN, HIDDEN, dsl.E4M3)
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=DEV)
        self.y0, self.y, self.z, self.dx0, self.dx = (e(ROWS, HIDDEN) for _ in range(5))
        self.h = e(ROWS, RANK, dtype=torch.float32)
        self.da, self.db = e(COUNT, RANK, HIDDEN, dtype=torch.float32), \
            e(COUNT, HIDDEN, RANK, dtype=torch.float32)
        self.dz = bf((ROWS, HIDDEN), 1e-3, 906)
        self.dy = e(ROWS, HIDDEN)
        self.dbias = e(HIDDEN, dtype=torch.float32)
        self.dws = e(dsl.fp8_cast_dbias_workspace_bytes(ROWS, HIDDEN), dtype=torch.uint8)

    def step(self):
        s = self.state
        part = lambda t, i: t[i:i + 1]
        dsl.fp8_adapter_plan(self.ids, self.plan)
        dsl.fp8_cast_transpose_amax(self.x, part(s.scale, 0), self.qx, part(s.amax_cur, 0))
        dsl.fp8_cast_transpose_amax(self.weight, part(s.scale, 1), self.qw, part(s.amax_cur, 1))
        dsl.fp8_linear_fwd(self.qx, self.qw, self.bias, self.y0)
        dsl.fp8_adapter_fwd(self.w, self.plan, self.x, self.y0, self.y, h=self.h, drop=self.drop_in,
                            workspace=self.ws)
        dsl.fp8_dropout_cast_transpose_amax(self.y, self.drop_out, part(s.scale, 2), self.qz,
                                            part(s.amax_cur, 2), residual=self.residual, y=self.z)
        # the way back from the gradient of z
        dsl.fp8_dropout_cast_transpose_amax(self.dz, self.drop_out, part(s.scale, 3), self.qdy,
                                            part(s.amax_cur, 3), y=self.dy, dbias=self.dbias,
                                            workspace=self.dws)
        dsl.fp8_linear_dgrad(self.qdy, self.qw, self.dx0)
        dsl.fp8_adapter_backward(self.w, self.plan, self.x, self.dy, self.h, dx_base=self.dx0,
                                 dx=self.dx, da=self.da, db=self.db, drop=self.drop_in,
                                 workspace=self.ws)

    def outputs(self):
        return [self.y0, self.y, self.h, self.z, self.qz.data, self.qz.data_t, self.qdy.data,
                self.dbias, self.dx0, self.dx, self.da, self.db, self.state.amax_cur]


def test_every_stage_against_its_reference():
    L = Layer()
    L.step()
    torch.cuda.synchronize()
    v = lambda t: bf16_values(bits16(t))
    a, b, alpha, ids = v(L.w.a), v(L.w.b), f32(L.w.alpha).astype(np.float64), L.ids.cpu().numpy()
    keep = ref.keep_mask(ROWS, HIDDEN, P_IN, 11, 0)
    f = float(ref.factor(P_IN))
    # the shared product
    ox, _, _, sx = oracle.cast_transpose_amax(bits16(L.x), 60.0, dsl.E4M3)
    ow, owt, _, sw = oracle.cast_transpose_amax(bits16(L.weight), 2000.0, dsl.E4M3)
    assert_gemm_close(v(L.y0), bf16_values(oracle.gemm_nt(ox, 0, ow, 0, sx, sw, bias=bits16(L.bias))))
    # its adapters: sums of 256 terms of about 0.06, a rank of 16, one bf16 rounding
    wy, wh = ref.adapter_forward(v(L.x), a, b, alpha, ids, v(L.y0), keep, f)
    terms = np.einsum("rk,rjk->rj", np.abs(v(L.x)) * keep * f, np.abs(a)[np.maximum(ids, 0)]) * 2.0
    assert (np.abs(f32(L.h) - wh) <= (HIDDEN + 4) * 2.0 ** -23 * terms).all()
    err = np.abs(wh).max() * np.abs(b).max() * RANK * (2.0 ** -16 + (HIDDEN + 40) * 2.0 ** -23)
    assert (np.abs(v(L.y) - wy) <= 2.0 ** -8 * np.abs(wy) + 2 * err).all()
    # dropout onto the residual, cast for the next linear: bit for bit
    m = ref.keep_mask(ROWS, HIDDEN, P_OUT, 12, 0)
    z = ref.bf16_round(ref.dropout(L.y.float().cpu().numpy(), m, ref.factor(P_OUT),
                                   L.residual.float().cpu().numpy()))
    np.testing.assert_array_equal(bits16(L.z), z)
    q, qt, amax, _ = oracle.cast_transpose_amax(z, 60.0, dsl.E4M3)
    np.testing.assert_array_equal(bits8(L.qz.data), q)
    np.testing.assert_array_equal(bits8(L.qz.data_t), qt)
    assert float(L.state.amax_cur[2]) == amax
    # the way back
    dy = ref.bf16_round(ref.dropout(L.dz.float().cpu().numpy(), m, ref.factor(P_OUT)))
    np.testing.assert_array_equal(bits16(L.dy), dy)
    qd, _, _, sd = oracle.cast_transpose_amax(dy, 4.0e4, dsl.E5M2)
    np.testing.assert_array_equal(bits8(L.qdy.data), qd)
    d = bf16_values(dy)
    assert (np.abs(f32(L.dbias) - d.sum(0)) <= (2 + 12) * 2.0 ** -24 * np.abs(d).sum(0)).all()
    assert_gemm_close(v(L.dx0), bf16_values(oracle.gemm_nt(qd, 1, owt, 0, sd, sw)))
    wdx, wda, wdb, wg = ref.adapter_backward(v(L.x), a, b, alpha, ids, v(L.dy),
                                             f32(L.h).astype(np.float64), v(L.dx0), keep, f)
    err = np.abs(wg).max() * np.abs(a).max() * RANK * f * (2.0 ** -16 + (HIDDEN + 40) * 2.0 ** -23)
    assert (np.abs(v(L.dx) - wdx) <= 2.0 ** -8 * np.abs(wdx) + 2 * err).all()
    n = (ids >= 0).sum()
    sum_g = np.einsum("rn,rnj->rj", np.abs(d), np.abs(b)[np.maximum(ids, 0)]) * 2.0
    e = ((HIDDEN + 4) + 3 * n + 4) * 2.0 ** -23 * sum_g.max() * f * np.abs(v(L.x)).sum(0).max()
    assert (np.abs(f32(L.da) - wda) <= e).all()
    e = (3 * n + 4) * 2.0 ** -23 * np.abs(wh).max() * np.abs(d).sum(0).max()
    assert (np.abs(f32(L.db) - wdb) <= e).all()


def test_the_captured_step_equals_the_eager_one():
    """Two graphs with buffers of their own, replayed in turn with new masks
    (the offsets move between replays), new rows per adapter and the scale
    update between them; each replay equals the eager step on a third set."""
    a, b, eager = Layer(), Layer(), Layer()
    graphs = []
    for L in (a, b):
        L.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            L.step()
        graphs.append(graph)
    for L in (a, b, eager):
        L.state.amax_cur.zero_()
    for replay in range(4):
        for L in (a, b, eager):
            L.rng[:, 1] = replay
            L.ids.copy_(torch.roll(L.ids, 7))
        for graph in graphs:
            graph.replay()
        eager.step()
        torch.cuda.synchronize()
        for got in (a, b):
            for x, y in zip(got.outputs(), eager.outputs()):
                assert torch.equal(x, y)
        for L in (a, b, eager):
            L.state.update()


def test_serving_batch_beside_a_cached_weight():
    """Decode steps of changing requests beside one cached FP8 weight: rows of
    the base model alone come out as the shared product left them."""
    L = Layer()
    L.step()
    base = L.y0.clone()
    for ids in ([-1] * ROWS, [2] * ROWS, list(np.arange(ROWS) % (COUNT + 1) - 1)):
        L.ids.copy_(torch.tensor(ids, dtype=torch.int32))
        dsl.fp8_adapter_plan(L.ids, L.plan)
        L.y.copy_(base)
        dsl.fp8_adapter_fwd(L.w, L.plan, L.x, L.y, L.y, workspace=L.ws)
        alone = L.ids < 0
        assert torch.equal(L.y[alone], base[alone])
        wy, _ = ref.adapter_forward(bf16_values(bits16(L.x)), bf16_values(bits16(L.w.a)),
                                    bf16_values(bits16(L.w.b)), f32(L.w.alpha).astype(np.float64),
                                    np.array(ids), bf16_values(bits16(base)))
        assert (np.abs(bf16_values(bits16(L.y)) - wy) <= 2.0 ** -8 * np.abs(wy) + 1e-3).all()
