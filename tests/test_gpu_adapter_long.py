"""The loops that long batches of the adapters run: several tiles in a
workgroup of the expand and of the weight gradients, and more than one part of
the contraction beside more tiles than compute units.

Integer inputs (see test_gpu_adapter.py), so results are exact.  Each case says
which split it reaches and checks that it does."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import adapter_splits as splits
from tests.gpu_util import DEV, f32
from tests.test_gpu_adapter import Case, _exact, _ids, _same_bf16

pytestmark = pytest.mark.gpu


def _batch(order, rows, count):
    """Row ids, a tenth of them -1: any order, or runs of uneven lengths."""
    if order == "scatter":
        return _ids(rows, count, none=0.1)
    cuts = np.sort(np.random.default_rng(3).integers(0, rows, count))
    ids = np.searchsorted(cuts, np.arange(rows), side="right") % (count + 1)
    return np.where(ids == count, -1, ids)


# 3 adapters of many chunks each; 9 that begin and end inside chunks; 40, of
# which several lie in one chunk.
@pytest.mark.parametrize("count, order", [(3, "scatter"), (9, "scatter"), (9, "runs"), (40, "scatter")])
@pytest.mark.parametrize("rank, k, n, p, dtype", [(8, 8200, 8200, 0.0, torch.float32),
                                                  (24, 8200, 4104, 0.5, torch.bfloat16),
                                                  (64, 4104, 8200, 0.0, torch.float32),
                                                  (72, 4104, 4104, 0.5, torch.float32),
                                                  (128, 6152, 4104, 0.0, torch.bfloat16)])
def test_weight_gradients_over_several_tiles_a_workgroup(rank, k, n, p, dtype, count, order):
    rows = 1500
    assert splits.gradient_chunk(splits.tiles(rows, count), rank, k, n) >= 3
    c = Case(rows, k, n, rank, count, _batch(order, rows, count), p=p)
    dx, da, db = c.backward(dtype)
    wdx, wda, wdb, _ = c.want_backward()
    _same_bf16(dx, wdx)
    for got, want in ((da, wda), (db, wdb)):
        if dtype is torch.float32:
            np.testing.assert_array_equal(f32(got), want)
        else:
            _same_bf16(got, want)


@pytest.mark.parametrize("count, order", [(3, "scatter"), (30, "scatter"), (7, "runs")])
@pytest.mark.parametrize("rank", [40, 64, 72, 128])
def test_expand_over_several_tiles_a_workgroup(rank, count, order):
    """Forward, in place and not, with and without a base, adapters changing
    inside a chunk and ending before the rows of none do."""
    rows, k, n = 4200, 136, 8200
    assert splits.expand_chunk(splits.tiles(rows, count), n, rank) >= 3
    c = Case(rows, k, n, rank, count, _batch(order, rows, count))
    y, h = c.forward()
    wy, wh = c.want_forward()
    np.testing.assert_array_equal(f32(h), wh)
    _same_bf16(y, wy)
    x, both = c.dev(c.x), c.dev(c.base)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, both, both, workspace=c.ws)
    assert torch.equal(both, y)
    dsl.fp8_adapter_fwd(c.w, c.plan, x, None, both, h=h, workspace=c.ws)
    _same_bf16(both, wy - c.d64(c.base))
    np.testing.assert_array_equal(f32(h), wh)


@pytest.mark.parametrize("count, order", [(3, "scatter"), (7, "runs")])
@pytest.mark.parametrize("rank, p", [(40, 0.5), (64, 0.0), (128, 0.5)])
def test_data_gradient_over_several_tiles_a_workgroup(rank, p, count, order):
    """With and without the packing of the weight gradients before it."""
    rows, k, n = 4200, 8200, 136
    assert splits.expand_chunk(splits.tiles(rows, count), k, rank) >= 3
    c = Case(rows, k, n, rank, count, _batch(order, rows, count), p=p)
    dx, da, db = c.backward()
    wdx, wda, wdb, _ = c.want_backward()
    _same_bf16(dx, wdx)
    np.testing.assert_array_equal(f32(da), wda)
    np.testing.assert_array_equal(f32(db), wdb)
    both = c.dev(c.dx_base)
    dsl.fp8_adapter_backward(c.w, c.plan, None, c.dev(c.dy), dx_base=both, dx=both, drop=c.drop,
                             workspace=c.ws)
    assert torch.equal(both, dx)


@pytest.mark.parametrize("rows, count, rank, C", [(8192, 3, 32, 4104), (8300, 3, 64, 4104),
                                                  (8300, 3, 40, 6152), (8300, 3, 128, 6152),
                                                  (12200, 3, 72, 4104)])
def test_parts_of_the_contraction_beside_more_tiles_than_units(rows, count, rank, C):
    tiles = splits.tiles(rows, count)
    assert tiles > 256 and splits.parts(tiles, C, rank) >= 2
    # the forward's contraction, h kept and not
    c = Case(rows, C, 72, rank, count, _ids(rows, count, none=0.05))
    y, h = c.forward()
    wy, wh = c.want_forward()
    np.testing.assert_array_equal(f32(h), wh)
    _same_bf16(y, wy)
    assert torch.equal(c.forward(keep_h=False)[0], y)
    # the backward's: g in parts for dx and for the packed operands
    _exact(Case(rows, 72, C, rank, count, _ids(rows, count, none=0.05)))


def test_a_long_batch_in_a_graph_follows_its_inputs():
    """Several tiles a workgroup in every kernel, captured and replayed."""
    rows, k, n, rank, count = 1500, 4104, 8200, 64, 9
    assert splits.gradient_chunk(splits.tiles(rows, count), rank, k, n) >= 3
    c = Case(rows, k, n, rank, count, _ids(rows, count), p=0.5)
    ids, x, base, dy = (c.dev(t) for t in (c.ids, c.x, c.base, c.dy))
    y, h, dx = torch.empty_like(base), torch.empty(rows, rank, device=DEV), torch.empty_like(x)
    da, db = torch.empty(c.a.shape, device=DEV), torch.empty(c.b.shape, device=DEV)

    def step():
        dsl.fp8_adapter_plan(ids, c.plan)
        dsl.fp8_adapter_fwd(c.w, c.plan, x, base, y, h=h, drop=c.drop, workspace=c.ws)
        dsl.fp8_adapter_backward(c.w, c.plan, x, dy, h, dx=dx, da=da, db=db, drop=c.drop,
                                 workspace=c.ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for replay in range(3):
        ids.copy_(torch.as_tensor(_ids(rows, count, seed=replay, none=0.3 * replay)))
        x.copy_(x.flip(0))
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
