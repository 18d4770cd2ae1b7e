"""Relations between calls of the adapters that hold bit for bit, on normal
values, where the order of sums and every rounding show."""
import pytest
import torch

from tests.gpu_util import bits16
from tests.test_gpu_adapter import Case, _ids

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
