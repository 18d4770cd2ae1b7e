"""A layer of FP8 experts from its tokens to its weights' update: every expert's
operands and products against the same calls on rows gathered by torch (bit for
bit), an expert without tokens, dropped tokens, and the whole step captured."""
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TOKENS, TOP_K, EXPERTS, HIDDEN, INNER = 300, 2, 5, 256, 512
SCALES = dict(x=40.0, w1=2000.0, w2=2000.0, a=30.0, do=3e4, du=3e4)


class Layer:
    """y = x + combine(relu(x W1^T) W2^T) with fp32 master weights."""

    def __init__(self, capacity, bits, seed=0):
        g = torch.Generator(DEV).manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
        self.w1 = [rand(INNER, HIDDEN, std=0.05) for _ in range(EXPERTS)]
        self.w2 = [rand(HIDDEN, INNER, std=0.05) for _ in range(EXPERTS)]
        self.g1, self.g2 = ([torch.zeros_like(w) for w in ws] for ws in (self.w1, self.w2))
        self.plan = dsl.ExpertPlan.empty(TOKENS, TOP_K, EXPERTS, capacity)
        rows = self.plan.rows
        f8 = dsl.Float8Tensor.empty
        self.qw1 = [f8(INNER, HIDDEN, dsl.E4M3) for _ in range(EXPERTS)]
        self.qw2 = [f8(HIDDEN, INNER, dsl.E4M3) for _ in range(EXPERTS)]
        self.qx, self.qdo = f8(rows, HIDDEN, dsl.E4M3), f8(rows, HIDDEN, dsl.E5M2)
        self.qa, self.qdu = f8(rows, INNER, dsl.E4M3), f8(rows, INNER, dsl.E5M2)
        z = lambda n: torch.zeros(rows, n, dtype=BF16, device=DEV)
        self.u, self.o, self.da, self.dr = z(INNER), z(HIDDEN), z(INNER), z(HIDDEN)
        self.y, self.dx = (torch.empty(TOKENS, HIDDEN, dtype=BF16, device=DEV) for _ in range(2))
        self.dweights = torch.empty(TOKENS, TOP_K, device=DEV)
        self.scale = {k: torch.tensor([v], device=DEV) for k, v in SCALES.items()}
        self.amax = {k: torch.zeros(1, device=DEV) for k in SCALES}
        self.opt = dsl.AdamW([dsl.AdamWTensor.zeros(w, d, bits, weight_decay=0.1) for w, d in
                              zip(self.w1 + self.w2, self.g1 + self.g2)], lr=1e-3, seed=5)
        self.norm, self.factor = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        self.flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(dsl.fp8_grad_norm_workspace_bytes(), dtype=torch.uint8, device=DEV)

    def cast(self, name, x, out):
        dsl.fp8_cast_transpose_amax(x, self.scale[name], out, self.amax[name])

    def run(self, ids, x, weights, dy, offsets=None):
        plan, s, am = self.plan, self.scale, self.amax
        if plan.capacity:
            dsl.fp8_expert_plan(ids, plan)
            offsets = [e * plan.capacity for e in range(EXPERTS + 1)]
        for e in range(EXPERTS):
            self.cast("w1", self.w1[e], self.qw1[e])
            self.cast("w2", self.w2[e], self.qw2[e])
        # Forward.
        dsl.fp8_expert_gather_cast_transpose_amax(plan, x, s["x"], self.qx, am["x"])
        parts = lambda q: plan.segments(q, offsets)
        qx, qa = parts(self.qx), parts(self.qa)
        for e in range(EXPERTS):
            a, b = offsets[e], offsets[e + 1]
            dsl.fp8_linear_fwd(qx[e], self.qw1[e], None, self.u[a:b])
            self.cast("a", torch.relu(self.u[a:b]), qa[e])
            dsl.fp8_linear_fwd(qa[e], self.qw2[e], None, self.o[a:b])
        dsl.fp8_expert_combine(plan, self.o, self.y, weights=weights, base=x)
        # Backward.
        dsl.fp8_expert_combine_backward(plan, dy, self.o, self.dweights)
        dsl.fp8_expert_gather_cast_transpose_amax(plan, dy, s["do"], self.qdo, am["do"],
                                                  weights=weights)
        qdo, qdu = parts(self.qdo), parts(self.qdu)
        for e in range(EXPERTS):
            a, b = offsets[e], offsets[e + 1]
            dsl.fp8_linear_dgrad(qdo[e], self.qw2[e], self.da[a:b])
            dsl.fp8_linear_wgrad(qdo[e], qa[e], self.g2[e])
            self.cast("du", self.da[a:b] * (self.u[a:b] > 0), qdu[e])
            dsl.fp8_linear_dgrad(qdu[e], self.qw1[e], self.dr[a:b])
            dsl.fp8_linear_wgrad(qdu[e], qx[e], self.g1[e])
        dsl.fp8_expert_combine(plan, self.dr, self.dx, base=dy)
        # Update.
        dsl.fp8_grad_norm(self.opt.grads, self.norm, self.ws, 0.05, factor=self.factor,
                          noop_flag=self.flag)
        self.opt.step(grad_scale=self.factor, noop_flag=self.flag)


def _batch(seed, unused=None):
    g = torch.Generator(DEV).manual_seed(seed)
    score = torch.randn(TOKENS, EXPERTS, generator=g, device=DEV)
    if unused is not None:
        score[:, unused] = -100.0
    best = score.topk(TOP_K, 1)
    ids = best.indices.to(torch.int32)
    ids[::17] = -1                                          # padding tokens
    x = torch.randn(TOKENS, HIDDEN, generator=g, device=DEV).to(BF16)
    dy = (torch.randn(TOKENS, HIDDEN, generator=g, device=DEV) * 1e-3).to(BF16)
    return ids.contiguous(), x, best.values.softmax(1).contiguous(), dy


@pytest.mark.parametrize("capacity", [0, 112])
def test_layer_against_rows_gathered_by_torch(capacity):
    layer = Layer(capacity, 32)
    ids, x, weights, dy = _batch(1, unused=3)
    dsl.fp8_expert_plan(ids, layer.plan)
    offsets = layer.plan.offsets.tolist()
    w1, w2 = [w.clone() for w in layer.w1], [w.clone() for w in layer.w2]
    layer.run(ids, x, weights, dy, offsets)
    assert capacity == 0 or int(layer.plan.counts.max()) == capacity     # some are dropped
    s = layer.scale
    y_want, dx_want = x.double(), dy.double()
    y_size, dx_size = y_want.abs(), dx_want.abs()
    for e in range(EXPERTS):
        a, b = offsets[e], offsets[e + 1]
        pairs = torch.nonzero(ids.reshape(-1) == e)[:, 0]
        if capacity:
            pairs = pairs[:capacity]
        t, n = pairs // TOP_K, pairs.numel()
        w = weights.reshape(-1)[pairs][:, None]
        assert layer.plan.counts[e] == n
        if e == 3:
            assert n == 0 and (layer.g1[e] == 0).all() and (layer.g2[e] == 0).all()
            if b == a:
                continue

        def padded(v, cols):
            out = torch.zeros(b - a, cols, dtype=BF16, device=DEV)
            out[:n] = v
            return out

        def cast(v, name, fmt):
            q = dsl.Float8Tensor.empty(v.shape[0], v.shape[1], fmt)
            dsl.fp8_cast_transpose_amax(v.contiguous(), s[name], q)
            return q

        new = lambda rows, cols, dtype=BF16: torch.empty(rows, cols, dtype=dtype, device=DEV)
        qx, qw1, qw2 = cast(padded(x[t], HIDDEN), "x", 0), cast(w1[e], "w1", 0), cast(w2[e], "w2", 0)
        u, o = new(b - a, INNER), new(b - a, HIDDEN)
        dsl.fp8_linear_fwd(qx, qw1, None, u)
        qa = cast(torch.relu(u), "a", 0)
        dsl.fp8_linear_fwd(qa, qw2, None, o)
        # The fp32 product rounded to bf16, as the definition has it.
        qdo = cast(padded((w * dy[t].float()).to(BF16), HIDDEN), "do", 1)
        da, dr = new(b - a, INNER), new(b - a, HIDDEN)
        g1, g2 = new(INNER, HIDDEN, torch.float32), new(HIDDEN, INNER, torch.float32)
        dsl.fp8_linear_dgrad(qdo, qw2, da)
        dsl.fp8_linear_wgrad(qdo, qa, g2)
        qdu = cast(da * (u > 0), "du", 1)
        dsl.fp8_linear_dgrad(qdu, qw1, dr)
        dsl.fp8_linear_wgrad(qdu, qx, g1)
        for got, want in ((layer.u[a:b], u), (layer.o[a:b], o), (layer.g1[e], g1),
                          (layer.g2[e], g2), (layer.dr[a:b], dr)):
            assert torch.equal(got, want)
        for got, want in ((layer.qx, qx), (layer.qdo, qdo)):
            part = layer.plan.segments(got, offsets)[e]
            assert torch.equal(part.data, want.data) and torch.equal(part.data_t, want.data_t)
        y_want.index_add_(0, t, w.double() * o[:n].double())
        y_size.index_add_(0, t, (w.double() * o[:n].double()).abs())
        dx_want.index_add_(0, t, dr[:n].double())
        dx_size.index_add_(0, t, dr[:n].double().abs())
        dw = (dy[t].double() * o[:n].double()).sum(1)
        dw_size = (dy[t].double() * o[:n].double()).abs().sum(1)
        got = layer.dweights.reshape(-1)[pairs].double()
        assert ((got - dw).abs() <= (HIDDEN + 1) * 2.0 ** -24 * dw_size).all()
    # top_k + 1 fp32 operations, then half a bf16 step.
    for got, want, size in ((layer.y, y_want, y_size), (layer.dx, dx_want, dx_size)):
        bound = (TOP_K + 1) * 2.0 ** -24 * size
        assert ((got.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all()
    grads = torch.cat([g.reshape(-1) for g in layer.g1 + layer.g2]).double()
    assert abs(float(layer.norm) - float(grads.norm())) <= 2.0 ** -23 * float(grads.norm())
    assert float(layer.factor) < 1.0 and int(layer.flag) == 0
    assert all(not torch.equal(a, b) for a, b in zip(layer.w1 + layer.w2, w1 + w2))


@pytest.mark.parametrize("bits", [32, 8])
def test_whole_step_captured(bits):
    """Replays with other tokens, routes and weights between eager steps of a copy, which
    they must equal in every bit; each begins with the plan."""
    ids, x, weights, dy = _batch(2)
    captured, eager = Layer(112, bits), Layer(112, bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.run(ids, x, weights, dy)
    torch.cuda.current_stream().wait_stream(side)
    eager.run(ids, x, weights, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        captured.run(ids, x, weights, dy)
    for step in range(4):
        for old, new in zip((ids, x, weights, dy), _batch(10 + step)):
            old.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        eager.run(ids, x, weights, dy)
        torch.cuda.synchronize()
        for a, b in ((captured.y, eager.y), (captured.dx, eager.dx),
                     (captured.dweights, eager.dweights), (captured.norm, eager.norm),
                     *zip(captured.w1 + captured.w2, eager.w1 + eager.w2),
                     *zip([t.m for t in captured.opt.tensors], [t.m for t in eager.opt.tensors])):
            assert torch.equal(a, b)
        assert captured.opt.steps.tolist() == [step + 2]


def test_two_graphs_share_a_plan_and_run_on_another_stream():
    """Two captured layers' calls read one plan, built eagerly between their replays on
    a side stream."""
    ids, x, weights, dy = _batch(3)
    plan = dsl.ExpertPlan.empty(TOKENS, TOP_K, EXPERTS, 128)
    dsl.fp8_expert_plan(ids, plan)
    rows = torch.zeros(plan.rows, HIDDEN, dtype=BF16, device=DEV)
    y, dw = torch.zeros_like(x), torch.zeros(TOKENS, TOP_K, device=DEV)
    calls = (lambda: dsl.fp8_expert_gather(plan, x, rows),
             lambda: (dsl.fp8_expert_combine(plan, rows, y, weights=weights, base=x),
                      dsl.fp8_expert_combine_backward(plan, dy, rows, dw)))
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            c()
        graphs.append(g)
    side = torch.cuda.Stream()
    for seed in (4, 5, 6):
        new, _, _, _ = _batch(seed)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            dsl.fp8_expert_plan(new, plan, stream=side)
            for g in graphs:
                g.replay()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        live = plan.slots >= 0
        # A token's own row, once for each slot: y = x (1 + the weights of its slots).
        want = x.double() * (1 + (weights * live).sum(1, keepdim=True).double())
        assert ((y.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-30).all()
        dot = (dy.double() * x.double()).sum(1, keepdim=True) * live
        size = (dy.double() * x.double()).abs().sum(1, keepdim=True)
        assert ((dw.double() - dot).abs() <= (HIDDEN + 1) * 2.0 ** -24 * size).all()
