"""The adapters and the dropout's cast at sizes whose indexes or grids leave
what 32 bits and one grid dimension hold."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests.gpu_util import DEV
from tests.test_gpu_adapter import Case, _exact, _ids

pytestmark = pytest.mark.gpu


def test_more_chunks_than_a_grid_dimension():
    """A million rows: the chunks of tiles run over two grid dimensions, and the
    packing's rows of workgroups before them."""
    rows, count = 1_060_000, 5
    _exact(Case(rows, 16, 8, 8, count, _ids(rows, count)))


def test_h_past_32_bits_of_elements():
    """17 million rows of rank 128: h has more than 2^31 elements.  Integers, so
    that torch's fp32 products over 8 terms and 128 are exact as well."""
    rows, k, n, rank = 17_000_000, 8, 8, 128
    g = torch.Generator(device=DEV).manual_seed(0)
    draw = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    x, base, a, b = draw(rows, k), draw(rows, n), draw(1, rank, k), draw(1, n, rank)
    ids = torch.zeros(rows, dtype=torch.int32, device=DEV)
    ids[rows // 2] = -1
    w = dsl.Adapters(a, b, torch.full((1,), 2.0, device=DEV))
    plan = dsl.AdapterPlan.empty(rows, 1)
    dsl.fp8_adapter_plan(ids, plan)
    ws = torch.empty(dsl.fp8_adapter_workspace_bytes(rows, 1, rank, k, n), dtype=torch.uint8, device=DEV)
    h, y, dx = torch.empty(rows, rank, device=DEV), torch.empty_like(base), torch.empty_like(x)
    da, db = torch.empty(1, rank, k, device=DEV), torch.empty(1, n, rank, device=DEV)
    dsl.fp8_adapter_fwd(w, plan, x, base, y, h=h, workspace=ws)
    dsl.fp8_adapter_backward(w, plan, x, base, h, dx=dx, da=da, db=db, workspace=ws)
    wda, wdb = torch.zeros(rank, k, device=DEV, dtype=torch.float64), \
        torch.zeros(n, rank, device=DEV, dtype=torch.float64)
    A, B = a[0].float(), b[0].float()
    for at in range(0, rows, 1 << 20):
        s = slice(at, at + (1 << 20))
        live = (ids[s] >= 0)[:, None]
        wh = torch.where(live, 2.0 * (x[s].float() @ A.t()), 0.0)
        wg = torch.where(live, 2.0 * (base[s].float() @ B), 0.0)
        assert torch.equal(h[s], wh)
        assert torch.equal(y[s], (base[s].float() + wh @ B.t()).to(torch.bfloat16))
        assert torch.equal(dx[s], (wg @ A).to(torch.bfloat16))
        wda += wg.double().t() @ x[s].double()
        wdb += base[s].double().t() @ wh.double()
    # Terms of both signs, at most 16: the running sums stay below 2^24, so fp32
    # adds them exactly.
    for got, want in ((da[0], wda), (db[0], wdb)):
        assert want.abs().max() < 2 ** 22 and torch.equal(got.double(), want)


def test_dropout_cast_past_32_bits_of_elements():
    """Codes and transpose of more than 2^31 elements, against the dropout and
    the cast called one after the other."""
    rows, cols = 32784, 65552
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(
        generator=torch.Generator(device=DEV).manual_seed(0))
    drop = dsl.Dropout(0.1, torch.tensor([7, 8], device=DEV))
    scale, amax, amax2 = torch.tensor([64.0], device=DEV), *(torch.zeros(1, device=DEV) for _ in range(2))
    one = dsl.Float8Tensor.empty(rows, cols, dsl.E4M3, device=DEV)
    y = torch.empty_like(x)
    dsl.fp8_dropout_cast_transpose_amax(x, drop, scale, one, amax, y=y)
    dsl.fp8_dropout(x, drop, x)
    assert torch.equal(y, x)
    two = dsl.Float8Tensor.empty(rows, cols, dsl.E4M3, device=DEV)
    dsl.fp8_cast_transpose_amax(x, scale, two, amax2)
    assert torch.equal(one.data, two.data) and torch.equal(one.data_t, two.data_t)
    assert torch.equal(amax, amax2) and np.isfinite(float(amax))
