"""Plans at the edges of their forms (one workgroup to 4096 pairs, pieces beyond), with
and without a capacity, and the plan of rows that are in expert order already."""
import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import expert_reference as ref
from tests.gpu_util import DEV, bits8

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _ids(tokens, top_k, experts, how, seed=0):
    r = np.random.default_rng(seed)
    if how == "one":                             # the last expert takes all, the others are empty
        return np.full((tokens, top_k), experts - 1, np.int32)
    if how == "runs":                            # long runs of one expert, in falling order
        pair = np.arange(tokens * top_k, dtype=np.int64)
        return (experts - 1 - pair * experts // pair.size).astype(np.int32).reshape(tokens, top_k)
    ids = r.integers(0, experts, (tokens, top_k)).astype(np.int32)
    ids[r.random(ids.shape) < 0.1] = -1
    return ids


def _build(ids, experts, capacity):
    plan = dsl.ExpertPlan.empty(*ids.shape, experts, capacity)
    plan.buf.fill_(0x5A)                         # its contents on entry do not matter
    dsl.fp8_expert_plan(torch.from_numpy(ids).to(DEV), plan)
    return plan


@pytest.mark.parametrize("how", ["mixed", "one", "runs"])
@pytest.mark.parametrize("experts, capacity", [(1, 0), (8, 0), (8, 512), (8, 10240), (100, 48),
                                               (1024, 0)])
@pytest.mark.parametrize("tokens, top_k", [
    (1000, 3),                                   # 375 pairs a wave: more than its first 256
    (1365, 3), (512, 8), (241, 17),              # 4095, 4096, 4097 pairs
    (6143, 1), (2048, 3)])                       # two pieces, three
def test_edges(tokens, top_k, experts, capacity, how):
    ids = _ids(tokens, top_k, experts, how)
    plan, want = _build(ids, experts, capacity), ref.plan(ids, experts, capacity)
    for got, array in zip((plan.offsets, plan.counts, plan.slots, plan.sources), want):
        np.testing.assert_array_equal(got.cpu().numpy(), array)


@pytest.mark.parametrize("capacity", [0, 112])
@pytest.mark.parametrize("fmt", [dsl.E4M3, dsl.E5M2])
def test_rows_in_expert_order(capacity, fmt):
    """The activations between an expert's linears, cast for all experts in one call:
    each expert's part is what the plain cast writes for its rows, with zeros for those
    that hold no pair."""
    experts, cols = 5, 208
    ids = _ids(300, 2, experts, "mixed", 1)
    ids[ids == 3] = 4                            # one has no pairs
    plan = _build(ids, experts, capacity)
    sources = plan.sources.long()
    expert = torch.from_numpy(ids).to(DEV).view(-1)
    again = dsl.ExpertPlan.empty(plan.rows, 1, experts, capacity)
    dsl.fp8_expert_plan(torch.where(sources >= 0, expert[sources.clamp(min=0)], -1)
                        .to(torch.int32).view(-1, 1), again)
    assert torch.equal(again.offsets, plan.offsets) and torch.equal(again.counts, plan.counts)
    assert again.rows >= plan.rows and (again.rows == plan.rows or capacity == 0)
    live = sources >= 0
    assert torch.equal(again.slots.view(-1)[live].long(), torch.nonzero(live)[:, 0])
    u = torch.randn(plan.rows, cols, generator=torch.Generator(DEV).manual_seed(2), device=DEV).to(BF16)
    u[~live] = float("nan")                      # not read
    scale, amax = torch.tensor([30.0], device=DEV), torch.zeros(1, device=DEV)
    q = dsl.Float8Tensor.empty(again.rows, cols, fmt)
    dsl.fp8_expert_gather_cast_transpose_amax(again, u, scale, q, amax)
    zeroed = torch.where(live[:, None], u, 0).to(BF16)
    offsets, top = plan.offsets.tolist(), torch.zeros(1, device=DEV)
    for part, a, b in zip(again.segments(q, offsets), offsets, offsets[1:]):
        if a == b:
            continue
        one = dsl.Float8Tensor.empty(b - a, cols, fmt)
        dsl.fp8_cast_transpose_amax(zeroed[a:b], scale, one, top)
        np.testing.assert_array_equal(bits8(part.data), bits8(one.data))
        np.testing.assert_array_equal(bits8(part.data_t), bits8(one.data_t))
    assert float(amax) == float(top) > 0.0
