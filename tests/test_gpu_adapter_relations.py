"""Relations between calls of the adapters that hold bit for bit, on normal
values, where the order of sums and every rounding show."""
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests.gpu_util import DEV, bits16
from tests.test_gpu_adapter import Case, _exact, _ids, _same_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows, k, n, rank, p", [(201, 1048, 776, 24, 0.1), (90, 264, 136, 8, 0.0),
                                                 (300, 520, 264, 64, 0.0), (70, 136, 1032, 128, 0.5)])
def test_bf16_gradients_are_the_fp32_ones_rounded_once(rows, k, n, rank, p):
    c = Case(rows, k, n, rank, 3, _ids(rows, 3), p=p, ints=False)
    dx, da, db = c.backward()
    dx16, da16, db16 = c.backward(torch.bfloat16)
    assert torch.equal(dx16, dx)
    for got, exact in ((da16, da), (db16, db)):
        assert (bits16(got) == bits16(exact.to(torch.bfloat16))).all()


@pytest.mark.parametrize("rows, k, n, rank, p", [(4200, 2048, 1048, 16, 0.0), (4200, 1048, 2048, 8, 0.1),
                                                 (4200, 2056, 2048, 32, 0.5), (2100, 1032, 2056, 64, 0.0),
                                                 (2100, 2048, 2048, 128, 0.0), (48, 1048, 776, 16, 0.1)])
def test_a_rows_results_do_not_depend_on_the_other_rows(rows, k, n, rank, p):
    """Batches of one size that share their last rows: those rows' h, y and dx
    have the same bits wherever the plan puts them."""
    same, count = 30, 3
    c = Case(rows, k, n, rank, count, _ids(rows, count), p=p, ints=False)
    first = None
    for seed in range(4):
        ids = _ids(rows, count, seed=seed, none=0.3 * seed)
        ids[-same:] = [r % (count + 1) - 1 for r in range(same)]
        dsl.fp8_adapter_plan(c.dev(torch.as_tensor(ids, dtype=torch.int32)), c.plan)
        got = [t[-same:] for t in (*c.forward(), c.backward()[0])]
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b)


def test_handles_refuse_a_type_changed_in_place():
    """Memory that now holds another type at the same address and in the same
    shape (a module converted after its first call) is not read as the old one."""
    c = Case(40, 72, 88, 16, 3, _ids(40, 3), p=0.5)
    c.forward()
    for t, other in ((c.w.a, torch.float16), (c.w.b, torch.float16), (c.w.alpha, torch.int32),
                     (c.drop.rng, torch.float64)):
        was = t.dtype
        t.data = t.data.view(other)
        with pytest.raises(TypeError, match=str(was)):
            c.forward()
        t.data = t.data.view(was)
    c.forward()


@pytest.mark.parametrize("rank, n", [(16, 264), (64, 2056), (128, 520)])
def test_the_largest_batchs_workspace_serves_every_smaller_one(rank, n):
    """Rows that the plan of K parts treats differently: one part, a few, many."""
    whole = Case(2050, 1048, n, rank, 3, _ids(2050, 3))
    for rows in (2018, 994, 482, 129, 33, 1):
        c = Case(rows, 1048, n, rank, 3, _ids(rows, 3))
        c.ws = whole.ws
        _exact(c)


@pytest.mark.parametrize("rows, count, rank, k, n", [(512, 512, 64, 1048, 1032), (300, 3, 128, 2056, 264),
                                                     (2050, 4, 40, 136, 2048), (20, 2, 8, 4096, 72)])
def test_the_forwards_own_workspace_is_all_that_it_writes(rows, count, rank, k, n):
    """Forward and data gradient in their own workspace, its surroundings watched."""
    c = Case(rows, k, n, rank, count, _ids(rows, count), p=0.5)
    y, h = c.forward()
    dx = c.backward()[0]
    size = dsl.fp8_adapter_fwd_workspace_bytes(rows, count, rank, k, n)
    room = torch.full((size + 8192,), 0xFF, dtype=torch.uint8, device=DEV)
    ws = room[4096:4096 + size]
    y2, y3, h2, dx2 = (torch.empty_like(t) for t in (y, y, h, dx))
    x, base, dy, dx_base = (c.dev(t) for t in (c.x, c.base, c.dy, c.dx_base))
    dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y2, h=h2, drop=c.drop, workspace=ws)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y3, drop=c.drop, workspace=ws)
    dsl.fp8_adapter_backward(c.w, c.plan, None, dy, dx_base=dx_base, dx=dx2, drop=c.drop, workspace=ws)
    for got, want in ((y2, y), (y3, y), (h2, h), (dx2, dx)):
        assert torch.equal(got, want)
    assert (room[:4096] == 0xFF).all() and (room[4096 + size:] == 0xFF).all()
    da, db = torch.empty(c.a.shape, device=DEV), torch.empty(c.b.shape, device=DEV)
    if size < dsl.fp8_adapter_workspace_bytes(rows, count, rank, k, n):
        with pytest.raises(dsl.Fp8Error):
            dsl.fp8_adapter_backward(c.w, c.plan, x, dy, h, da=da, db=db, drop=c.drop, workspace=ws)


@pytest.mark.parametrize("rows, rank", [(40, 16), (200, 40)])
def test_an_infinite_row_is_infinite_or_nan_everywhere_and_alone(rows, rank):
    """One launch and two: x = inf meets weights of -1, 0 and 1, so every h and
    y of its row is lost, and no other row's."""
    c = Case(rows, 72, 88, rank, 2, [0, 1] * (rows // 2))
    y, h = c.forward()
    c.x[5] = float("inf")
    yi, hi = c.forward()
    assert not torch.isfinite(hi[5]).any() and not torch.isfinite(yi[5]).any()
    others = [r for r in range(rows) if r != 5]
    assert torch.equal(hi[others], h[others]) and torch.equal(yi[others], y[others])


@pytest.mark.parametrize("rows", [20, 300])
def test_lower_ranks_padded_with_zeros(rows):
    """Adapters of rank 4, 12 and 16 in one call of rank 16: the results of their
    own ranks, and zero gradients for the padding."""
    c = Case(rows, 136, 264, 16, 3, _ids(rows, 3), p=0.5)
    for i, rank in enumerate((4, 12, 16)):
        c.a[i, rank:] = 0
        c.b[i, :, rank:] = 0
        c.h[c.ids == i, rank:] = 0
    c.w = dsl.Adapters(c.dev(c.a), c.dev(c.b), c.dev(c.alpha))
    _exact(c)
    _, h = c.forward()
    _, da, db = c.backward()
    for i, rank in enumerate((4, 12, 16)):
        assert (h.cpu()[c.ids == i, rank:] == 0).all()
        assert (da[i, rank:] == 0).all() and (db[i, :, rank:] == 0).all()


def test_a_rank_above_the_most_in_two_calls():
    """Rank 160 as 128 and 32, the second onto what the first wrote."""
    first, second = (Case(90, 136, 264, rank, 3, _ids(90, 3), seed=rank) for rank in (128, 32))
    x, y = first.dev(first.x), torch.empty(90, 264, dtype=torch.bfloat16, device=DEV)
    dsl.fp8_adapter_fwd(first.w, first.plan, x, first.dev(first.base), y, workspace=first.ws)
    _same_bf16(y, first.want_forward()[0])
    second.x, second.base = first.x, y.cpu()
    dsl.fp8_adapter_fwd(second.w, second.plan, x, y, y, workspace=second.ws)
    _same_bf16(y, second.want_forward()[0])
