"""A captured dropout beside eager work between its replays."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import op_reference as ref
from tests.gpu_util import DEV, bf16_values, bits16

pytestmark = pytest.mark.gpu


def test_replays_and_eager_calls_in_turn():
    """Each replay gives its offset's mask, and what the program does with the
    result, or on other tensors, between the replays is right as well."""
    rows, cols, p, seed = 64, 128, 0.4, 5
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x32 = x.float().numpy()
    xd, y, z = x.to(DEV), torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), \
        torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    rng, rng2 = (torch.tensor([seed, v], device=DEV) for v in (0, 1000))
    captured, eager = dsl.Dropout(p, rng), dsl.Dropout(p, rng2)
    dsl.fp8_dropout(xd, captured, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        dsl.fp8_dropout(xd, captured, y)
    want = lambda offset: ref.bf16_round(ref.dropout(x32, ref.keep_mask(rows, cols, p, seed, offset),
                                                     ref.factor(p)))
    for offset in range(4):
        rng[1], rng2[1] = offset, 1000 + offset
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits16(y), want(offset))
        # Sums of bf16 values of about one are exact in 64 bits, in any order.
        assert float(y.double().sum()) == bf16_values(want(offset)).sum()
        dsl.fp8_dropout(xd, eager, z)
        np.testing.assert_array_equal(bits16(z), want(1000 + offset))
        np.testing.assert_array_equal(bits16(y), want(offset))
