"""GPU parity of the low-rank adapters (fp8_adapter_plan, fp8_adapter_fwd,
fp8_adapter_backward) against a float64 reference.

Two kinds of inputs:
* small integers (and alpha, dropout factor powers of two): every product and
  sum is an integer below 2^16 that fp32 and two bf16 parts hold exactly, so h,
  y before its rounding, dx, dA and dB are exact and compared bit for bit;
* normal values, within bounds counted from the operator's roundings: an fp32
  sum of n products in any order is off by at most n 2^-23 sum |terms| (one
  step per addition, the matrix core's additions rounded or truncated), a
  split h or g by 2^-16 of it (two bf16 parts; 2^-23 for three), a bf16
  result by 2^-8 of it."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import op_reference as ref
from tests.gpu_util import DEV, bits16, f32

pytestmark = pytest.mark.gpu

SEED, OFFSET = 77, 3
U = 2.0 ** -23


class Case:
    """Inputs on the CPU (float64 numpy and device tensors) of one call."""

    def __init__(self, rows, k, n, rank, count, ids, p=0.0, ints=True, seed=0, base=True):
        g = torch.Generator().manual_seed(seed)
        if ints:
            draw = lambda *s, m=2: torch.randint(-m, m + 1, s, generator=g).to(torch.bfloat16)
        else:
            draw = lambda *s, m=1: torch.randn(*s, generator=g).to(torch.bfloat16)
        self.rows, self.rank, self.count, self.p = rows, rank, count, p
        self.x, self.dy, self.a, self.b = draw(rows, k), draw(rows, n), draw(count, rank, k, m=1), \
            draw(count, n, rank, m=1)
        self.base = draw(rows, n, m=9) if base else None
        self.dx_base = draw(rows, k, m=9) if base else None
        self.alpha = torch.tensor([2.0 ** (i % 3 - 1) * (-1) ** i for i in range(count)]) if ints \
            else torch.randn(count, generator=g)
        self.h = draw(rows, rank, m=30).float() if ints else torch.randn(rows, rank, generator=g)
        self.ids = torch.as_tensor(ids, dtype=torch.int32)
        self.mask = ref.keep_mask(rows, k, p, SEED, OFFSET) if p else None
        self.f = float(ref.factor(p)) if p else 1.0
        self.d64 = lambda t: None if t is None else t.double().numpy()
        self.dev = lambda t: None if t is None else t.to(DEV)
        self.w = dsl.Adapters(self.dev(self.a), self.dev(self.b), self.dev(self.alpha))
        self.plan = dsl.AdapterPlan.empty(rows, count)
        self.plan.buf.fill_(0xA5)
        dsl.fp8_adapter_plan(self.dev(self.ids), self.plan)
        self.drop = dsl.Dropout(p, torch.tensor([SEED, OFFSET], device=DEV)) if p else None
        # the workspace's contents on entry do not matter: NaNs
        self.ws = torch.full((dsl.fp8_adapter_workspace_bytes(rows, count, rank, k, n),), 0xFF,
                             dtype=torch.uint8, device=DEV)

    def forward(self, keep_h=True):
        y = torch.full((self.rows, self.b.shape[1]), -7.0, dtype=torch.bfloat16, device=DEV)
        h = torch.full((self.rows, self.rank), -7.0, device=DEV) if keep_h else None
        dsl.fp8_adapter_fwd(self.w, self.plan, self.dev(self.x), self.dev(self.base), y, h=h,
                            drop=self.drop, workspace=self.ws)
        return y, h

    def backward(self, dtype=torch.float32):
        dx = torch.full(self.x.shape, -7.0, dtype=torch.bfloat16, device=DEV)
        da = torch.full(self.a.shape, -7.0, dtype=dtype, device=DEV)
        db = torch.full(self.b.shape, -7.0, dtype=dtype, device=DEV)
        dsl.fp8_adapter_backward(self.w, self.plan, self.dev(self.x), self.dev(self.dy),
                                 self.dev(self.h), dx_base=self.dev(self.dx_base), dx=dx, da=da,
                                 db=db, drop=self.drop, workspace=self.ws)
        return dx, da, db

    def want_forward(self):
        return ref.adapter_forward(self.d64(self.x), self.d64(self.a), self.d64(self.b),
                                   self.d64(self.alpha), self.ids.numpy(), self.d64(self.base),
                                   self.mask, self.f)

    def want_backward(self):
        return ref.adapter_backward(self.d64(self.x), self.d64(self.a), self.d64(self.b),
                                    self.d64(self.alpha), self.ids.numpy(), self.d64(self.dy),
                                    self.d64(self.h), self.d64(self.dx_base), self.mask, self.f)


def _same_bf16(got, want64):
    np.testing.assert_array_equal(bits16(got + 0.0), ref.bf16_round((want64 + 0.0).astype(np.float32)))


def _exact(case, dtype=torch.float32):
    y, h = case.forward()
    wy, wh = case.want_forward()
    np.testing.assert_array_equal(f32(h), wh)
    _same_bf16(y, wy)
    dx, da, db = case.backward(dtype)
    wdx, wda, wdb, _ = case.want_backward()
    _same_bf16(dx, wdx)
    for got, want in ((da, wda), (db, wdb)):
        if dtype == torch.float32:
            np.testing.assert_array_equal(f32(got), want)
        else:
            _same_bf16(got, want)


def _ids(rows, count, seed=0, none=0.2):
    g = np.random.default_rng(seed)
    ids = g.integers(0, count, rows)
    ids[g.random(rows) < none] = -1
    return ids


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 65, 200])
def test_rows(rows):
    _exact(Case(rows, 72, 136, 16, 3, _ids(rows, 3)))


@pytest.mark.parametrize("rank", list(range(8, 129, 8)))
def test_ranks(rank):
    _exact(Case(37, 104, 88, rank, 2, _ids(37, 2)))


@pytest.mark.parametrize("k, n", [(8, 8), (8, 520), (520, 8), (24, 40), (256, 512), (264, 776),
                                  (1048, 1032), (40, 2056)])
@pytest.mark.parametrize("rank", [8, 24, 64])
def test_features(k, n, rank):
    _exact(Case(33, k, n, rank, 2, _ids(33, 2)))


@pytest.mark.parametrize("p", [0.5, 0.75])
@pytest.mark.parametrize("rank", [8, 24, 40, 128])
def test_dropout_on_the_input(rank, p):
    _exact(Case(50, 264, 72, rank, 3, _ids(50, 3), p=p))


@pytest.mark.parametrize("rank", [16, 32, 64, 128])
def test_bf16_gradients(rank):
    _exact(Case(70, 136, 264, rank, 2, _ids(70, 2), p=0.5), torch.bfloat16)


@pytest.mark.parametrize("rows, count", [(300, 3), (900, 40), (2000, 1)])
def test_long_batches_span_chunks(rows, count):
    """Adapters that begin and end inside a weight-gradient chunk; one that spans many."""
    _exact(Case(rows, 16, 24, 8, count, _ids(rows, count, none=0.05)))


def test_a_long_contraction_in_parts():
    """Few rows: the contraction runs in several parts whose sums meet in order."""
    _exact(Case(3, 8192, 8200, 16, 2, [1, -1, 0]))


@pytest.mark.parametrize("ids", [[-1] * 40, [2] * 40, [0, 99, -7, 2 ** 31 - 1] * 10,
                                 [5] * 39 + [0], list(range(4)) * 10])
def test_groups(ids):
    """No row with an adapter; one adapter for all; values outside the range;
    adapters without rows (zero gradients)."""
    _exact(Case(40, 40, 48, 16, 6, ids))


def test_more_adapters_than_rows():
    _exact(Case(3, 16, 16, 8, 4096, [4095, 0, 4095]))


def test_plan_keeps_the_batch_order_and_reuses_its_buffer():
    """Building again in one buffer: the second batch's results, for batches
    of which the second leaves tiles unused."""
    c = Case(300, 16, 24, 8, 7, _ids(300, 7))
    _exact(c)
    c.ids = torch.as_tensor(np.where(np.arange(300) < 290, 3, -1), dtype=torch.int32)
    dsl.fp8_adapter_plan(c.ids.to(DEV), c.plan)
    _exact(c)


def test_without_base_and_without_h():
    c = Case(40, 72, 88, 16, 3, _ids(40, 3), base=False)
    _exact(c)
    y, _ = c.forward(keep_h=False)
    _same_bf16(y, c.want_forward()[0])


def test_single_gradients():
    c = Case(40, 72, 88, 16, 3, _ids(40, 3), p=0.5)
    dx, da, db = c.backward()
    only = torch.zeros_like(dx)
    dsl.fp8_adapter_backward(c.w, c.plan, None, c.dev(c.dy), dx_base=c.dev(c.dx_base), dx=only,
                             drop=c.drop, workspace=c.ws)
    assert torch.equal(only, dx)
    da2, db2 = torch.zeros_like(da), torch.zeros_like(db)
    dsl.fp8_adapter_backward(c.w, c.plan, c.dev(c.x), c.dev(c.dy), c.dev(c.h), da=da2, db=db2,
                             drop=c.drop, workspace=c.ws)
    assert torch.equal(da2, da) and torch.equal(db2, db)


def test_no_rows_clear_the_gradients():
    c = Case(8, 72, 88, 16, 3, _ids(8, 3))
    plan = dsl.AdapterPlan.empty(0, 3)
    dsl.fp8_adapter_plan(torch.zeros(0, dtype=torch.int32, device=DEV), plan)
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        da = torch.full(c.a.shape, 3.0, dtype=dtype, device=DEV)
        db = torch.full(c.b.shape, 3.0, dtype=dtype, device=DEV)
        dsl.fp8_adapter_backward(c.w, plan, e(72), e(88), torch.empty(0, 16, device=DEV), dx=e(72),
                                 da=da, db=db, workspace=c.ws)
        assert float(da.abs().sum()) == 0.0 and float(db.abs().sum()) == 0.0
    dsl.fp8_adapter_fwd(c.w, plan, e(72), e(88), e(88), workspace=c.ws)


def test_strides_in_place_and_untouched_surroundings():
    c = Case(50, 72, 88, 24, 3, _ids(50, 3))
    wide = torch.full((50, 304), -3.0, dtype=torch.bfloat16, device=DEV)
    x, base = wide[:, 8:80], wide[:, 104:192]
    x.copy_(c.x)
    base.copy_(c.base)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, base, base, workspace=c.ws)      # y is base
    _same_bf16(base, c.want_forward()[0])
    assert torch.equal(x.cpu(), c.x)
    for lo, hi in ((0, 8), (80, 104), (192, 304)):
        assert (wide[:, lo:hi] == -3.0).all()
    y = wide[:, 200:288]                                                 # another slice
    base.copy_(c.base)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y, workspace=c.ws)
    _same_bf16(y, c.want_forward()[0])
    assert torch.equal(base.cpu(), c.base)
    dy, dx = torch.zeros(50, 96, dtype=torch.bfloat16, device=DEV)[:, 8:], wide[:, 200:272]
    dy.copy_(c.dy)
    dx.copy_(c.dx_base)
    dsl.fp8_adapter_backward(c.w, c.plan, None, dy, dx_base=dx, dx=dx, workspace=c.ws)
    _same_bf16(dx, c.want_backward()[0])


def test_a_bad_row_stays_alone():
    """NaN and infinite rows reach their own outputs only; a row without an
    adapter passes its base through whatever it holds; dropped NaNs leave no
    trace."""
    c = Case(40, 72, 88, 16, 2, [0, 1] * 20)
    c.ids[7] = -1
    dsl.fp8_adapter_plan(c.ids.to(DEV), c.plan)
    clean, hc = c.forward()
    c.x[4] = float("nan")
    c.x[5] = float("inf")
    c.x[7] = float("nan")
    c.base[9, 3] = float("inf")
    y, h = c.forward()
    others = [r for r in range(40) if r not in (4, 5, 9)]
    assert torch.equal(y[others], clean[others]) and torch.equal(h[others], hc[others])
    assert torch.isnan(y[4]).all() and torch.isnan(h[4]).all()
    assert not torch.isfinite(h[5]).any() or bool((c.a[1] == 0).any())
    assert float(y[9, 3]) == float("inf") and torch.isfinite(y[9, 4:]).all()
    assert torch.isfinite(y[7]).all()
    # a NaN everywhere that the dropout drops
    d = Case(40, 72, 88, 16, 2, [0, 1] * 20, p=0.5)
    want = d.forward()
    d.x[torch.from_numpy(~d.mask)] = float("nan")
    got = d.forward()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _, da, _ = d.backward()
    assert torch.isfinite(da).all()


def test_infinite_h_and_g():
    """An infinity in h meets its zero low part as an infinity, not a NaN."""
    c = Case(8, 16, 24, 8, 1, [0] * 8)
    c.h[:] = 0.0
    c.h[3, 2] = float("inf")
    c.dy[:] = 1.0
    _, _, db = c.backward()
    assert (db[0, :, 2] == float("inf")).all() and torch.isfinite(db[0, :, [0, 1, 3, 4]]).all()


@pytest.mark.parametrize("rank", [8, 16, 40, 128])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_normal_values_within_counted_bounds(rank, p):
    rows, k, n, count = 201, 1048, 776, 3
    c = Case(rows, k, n, rank, count, _ids(rows, count), p=p, ints=False)
    y, h = c.forward()
    wy, wh = c.want_forward()
    ids = c.ids.numpy()
    live = (ids >= 0) & (ids < count)
    at = np.where(live, ids, 0)
    A, B, al = (np.abs(c.d64(t))[at] * live.reshape(-1, *[1] * (t.dim() - 1))
                for t in (c.a, c.b, c.alpha))
    X = np.abs(c.d64(c.x)) * (1.0 if c.mask is None else c.mask) * c.f
    # + 4: the two factors, their product and the product with the sum
    sum_h = np.einsum("rk,rjk->rj", X, A) * al[:, None]
    err_h = (k + 4) * U * sum_h
    assert (np.abs(f32(h) - wh) <= err_h).all()
    e32 = np.einsum("rj,rnj->rn", err_h + (2.0 ** -16 + (2 * rank + 1) * U) * np.abs(wh), B) \
        + U * np.abs(wy)
    assert (np.abs(y.double().cpu().numpy() - wy) <= 2.0 ** -8 * (np.abs(wy) + e32) + e32).all()

    dx, da, db = c.backward()
    wdx, wda, wdb, wg = c.want_backward()
    DY = np.abs(c.d64(c.dy))
    err_g = (n + 3) * U * np.einsum("rn,rnj->rj", DY, B) * al[:, None]
    keep = c.f * (np.ones_like(X) if c.mask is None else c.mask)
    e32 = keep * np.einsum("rj,rjk->rk", err_g + (2.0 ** -16 + (2 * rank + 2) * U) * np.abs(wg), A) \
        + U * np.abs(wdx)
    assert (np.abs(dx.double().cpu().numpy() - wdx) <= 2.0 ** -8 * (np.abs(wdx) + e32) + e32).all()
    for i in range(count):
        mine = np.nonzero(ids == i)[0]
        terms = 3 * mine.size + 3
        e = (err_g[mine] + (2.0 ** -23 + terms * U) * np.abs(wg[mine])).T @ X[mine]
        assert (np.abs(f32(da[i]) - wda[i]) <= e).all()
        e = (2.0 ** -23 + terms * U) * (DY[mine].T @ np.abs(c.d64(c.h))[mine])
        assert (np.abs(f32(db[i]) - wdb[i]) <= e).all()


def test_repeated_calls_give_the_same_bits():
    c = Case(700, 264, 520, 40, 5, _ids(700, 5), p=0.1, ints=False)
    first = c.forward() + c.backward()
    c.ws.fill_(0x5A)
    for a, b in zip(first, c.forward() + c.backward()):
        assert torch.equal(a, b)


def test_two_streams_with_workspaces_of_their_own():
    c = Case(500, 520, 264, 16, 4, _ids(500, 4), ints=False)
    want = c.forward()[0]
    x, base = c.dev(c.x), c.dev(c.base)
    ys = [torch.empty_like(want) for _ in range(2)]
    wss = [torch.empty_like(c.ws) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for y, ws, s in zip(ys, wss, streams):
            dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want) and torch.equal(ys[1], want)


def test_captured_plan_forward_and_backward_follow_their_inputs():
    """Plan, forward and backward in one graph: each replay sees the row ids,
    activations and dropout offset that the program wrote before it."""
    c = Case(90, 136, 200, 24, 4, _ids(90, 4), p=0.5)
    ids, x, base, dy = (c.dev(t) for t in (c.ids, c.x, c.base, c.dy))
    rng = torch.tensor([SEED, OFFSET], device=DEV)
    drop = dsl.Dropout(0.5, rng)
    y, h = torch.empty_like(base), torch.empty(90, 24, device=DEV)
    dx, da, db = torch.empty_like(x), torch.empty(c.a.shape, device=DEV), \
        torch.empty(c.b.shape, device=DEV)

    def step():
        dsl.fp8_adapter_plan(ids, c.plan)
        dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y, h=h, drop=drop, workspace=c.ws)
        dsl.fp8_adapter_backward(c.w, c.plan, x, dy, h, dx=dx, da=da, db=db, drop=drop,
                                 workspace=c.ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for replay in range(4):
        ids.copy_(torch.as_tensor(_ids(90, 4, seed=replay, none=0.3 * replay)))
        x.copy_(x.flip(0))
        rng[1] = replay
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, h, dx, da, db)]
        for t in (y, h, dx, da, db):
            t.fill_(-1.0)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, h, dx, da, db)):
            assert torch.equal(a, b)


def test_binding_refuses_what_the_kernels_cannot_see():
    c = Case(16, 64, 128, 16, 4, _ids(16, 4))
    x, y = c.dev(c.x), torch.empty(16, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(dsl.Fp8Error):
        dsl.fp8_adapter_fwd(c.w, c.plan, x, None, y, workspace=c.ws[:16])
    with pytest.raises(ValueError, match="overlap"):
        wide = torch.empty(16, 256, dtype=torch.bfloat16, device=DEV)
        dsl.fp8_adapter_fwd(c.w, c.plan, x, wide[:, 8:136], wide[:, :128], workspace=c.ws)
    with pytest.raises(ValueError, match="not been built"):
        dsl.fp8_adapter_fwd(c.w, dsl.AdapterPlan.empty(16, 4), x, None, y, workspace=c.ws)


@pytest.mark.parametrize("rank, k", [(16, 72), (24, 136), (40, 200), (128, 40), (16, 1048), (64, 2056)])
@pytest.mark.parametrize("rows", [3, 40])
def test_infinite_weights_stay_in_their_rank(rank, k, rows):
    """An infinite weight meets its own column of x only: h is infinite in its
    rank (x is positive) and finite elsewhere, whatever the padding of the
    contraction does; the same for g, whose padded rows are B's."""
    c = Case(rows, k, k, rank, 1, [0] * rows)
    c.x.fill_(1.0)
    c.dy.fill_(1.0)
    c.alpha.fill_(1.0)
    c.h.zero_()
    for at in (0, k - 8, k - 1):
        a, b = torch.ones_like(c.a), torch.ones_like(c.b)
        a[0, 3, at] = b[0, at, 3] = float("inf")
        c.w = dsl.Adapters(a.to(DEV), b.to(DEV), c.dev(c.alpha))
        _, h = c.forward()
        want = torch.full((rows, rank), float(k), device=DEV)
        want[:, 3] = float("inf")
        assert torch.equal(h, want)
        _, da, _ = c.backward()                       # dA = g^T x, g = the same sums
        want = torch.full_like(da, float(k * rows))
        want[:, 3] = float("inf")
        assert torch.equal(da, want)


def test_byte_offsets_past_32_bits():
    """Rows 2 MiB apart: the last ones lie 4.4 GB behind the first."""
    rows, ld = 2100, 1 << 20
    c = Case(rows, 72, 88, 16, 3, _ids(rows, 3))
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)
    view = lambda at, n: torch.as_strided(big, (rows, n), (ld, 1), at)
    x, base, y, dy, dx = view(0, 72), view(96, 88), view(192, 88), view(288, 88), view(384, 72)
    x.copy_(c.x)
    base.copy_(c.base)
    dy.copy_(c.dy)
    dx.copy_(c.dx_base)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y, workspace=c.ws)
    _same_bf16(y, c.want_forward()[0])
    da, db = torch.empty(c.a.shape, device=DEV), torch.empty(c.b.shape, device=DEV)
    dsl.fp8_adapter_backward(c.w, c.plan, x, dy, c.dev(c.h), dx_base=dx, dx=dx, da=da, db=db,
                             workspace=c.ws)
    wdx, wda, wdb, _ = c.want_backward()
    _same_bf16(dx, wdx)
    np.testing.assert_array_equal(f32(da), wda)
    np.testing.assert_array_equal(f32(db), wdb)


@pytest.mark.parametrize("rows, count, k, n", [(16, 1, 4096, 1032), (17, 1, 4096, 1032),
                                               (64, 32, 2048, 8192), (64, 32, 2056, 8200),
                                               (8, 8, 4096, 512), (8, 8, 4104, 512)])
def test_both_sides_of_the_one_launch_rule(rows, count, k, n):
    """Batches just inside and just outside of the rule that puts the forward
    into one launch, with and without h."""
    c = Case(rows, k, n, 16, count, _ids(rows, count, none=0.1))
    y, h = c.forward()
    wy, wh = c.want_forward()
    np.testing.assert_array_equal(f32(h), wh)
    _same_bf16(y, wy)
    assert torch.equal(c.forward(keep_h=False)[0], y)


def test_a_plan_that_was_never_built_writes_nothing():
    """Through the C ABI a buffer without a plan of these sizes: no work."""
    import ctypes
    c = Case(40, 72, 88, 16, 3, _ids(40, 3))
    x, base = c.dev(c.x), c.dev(c.base)
    y = torch.full((40, 88), -7.0, dtype=torch.bfloat16, device=DEV)
    for buf in (torch.full_like(c.plan.buf, 0xA5), torch.zeros_like(c.plan.buf)):
        rc = dsl.lib().fp8_adapter_fwd(ctypes.byref(c.w.desc()), buf.data_ptr(), buf.numel(), None,
                                       x.data_ptr(), 72, base.data_ptr(), 88, y.data_ptr(), 88, 40,
                                       None, c.ws.data_ptr(), c.ws.numel(),
                                       torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert (y == -7.0).all()


def test_handles_reshaped_in_place():
    """The descriptors that Adapters and Dropout keep follow their tensors."""
    wide = Case(40, 64, 48, 16, 3, [r % 4 - 1 for r in range(40)], seed=5)
    _same_bf16(wide.forward()[0], wide.want_forward()[0])
    narrow = Case(40, 64, 48, 8, 3, wide.ids.tolist(), seed=6)
    # the same memory, now of rank 8
    w = wide.w
    w.a.resize_(3, 8, 64).copy_(narrow.a)
    w.b.resize_(3, 48, 8).copy_(narrow.b)
    w.alpha.copy_(narrow.alpha)
    narrow.w = w
    _same_bf16(narrow.forward()[0], narrow.want_forward()[0])
    drop = dsl.Dropout(0.5, torch.tensor([1, 2], device=DEV))
    x = torch.ones(8, 16, device=DEV)
    dsl.fp8_dropout(x, drop, torch.empty_like(x))
    drop.rng.resize_(1)
    with pytest.raises(ValueError):
        dsl.fp8_dropout(x, drop, torch.empty_like(x))


@pytest.mark.parametrize("tiles", [[1, 1, 1], [1, 2, 0, 1], [0, 3, 2, 3], [2, 2], [1, 0, 0, 1], [3]])
@pytest.mark.parametrize("rank", [72, 128])
def test_pairs_of_tiles(rank, tiles):
    """Adapters that begin in the second tile of a pair, with and without rows."""
    ids = [a for a, t in enumerate(tiles) for _ in range(32 * t - 5 if t else 0)] + [-1] * 40
    _exact(Case(len(ids), 72, 264, rank, len(tiles), ids, seed=sum(tiles)))
