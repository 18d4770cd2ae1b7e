"""The optimizer's state in a program: counts and learning rates assigned between
captured steps, and copies that go on as the original does."""
import copy
import pickle

import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def _opt(bits, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda n: torch.randn(n, generator=g, device=DEV)
    return dsl.AdamW([dsl.AdamWTensor.zeros(rand(n), rand(n), bits, weight_decay=0.1)
                      for n in (300, 5000)], lr=1e-2, seed=3)


def _equal(a, b):
    return torch.equal(a.state, b.state) and all(
        torch.equal(getattr(x, n), getattr(y, n)) for x, y in zip(a.tensors, b.tensors)
        for n in ("param", "grad", "m", "v", "m_scale", "v_scale") if getattr(x, n) is not None)


@pytest.mark.parametrize("bits", [32, 8])
def test_copies_go_on_alike(bits):
    opt = _opt(bits)
    opt.step()
    others = [copy.deepcopy(opt), pickle.loads(pickle.dumps(opt))]
    kept = copy.deepcopy(opt)
    for _ in range(3):
        opt.step()
    assert not _equal(opt, kept)
    for other in others:
        assert _equal(other, kept)                      # not written by the original's steps
        for _ in range(3):
            other.step()
        assert _equal(other, opt) and other.steps.tolist() == [4]


@pytest.mark.parametrize("bits", [32, 8])
def test_resumed_counts_and_rates_in_a_captured_step(bits):
    """Assigned numbers reach the captured step's replays, which equal eager steps."""
    captured, eager = _opt(bits), _opt(bits)
    captured.step()
    eager.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        captured.step()
    for taken, lr in ((500, 1e-3), (torch.tensor(7.0), 0.5), (2 ** 33, 1e-2)):
        for opt in (captured, eager):
            opt.steps, opt.lr = taken, lr
        for _ in range(2):
            graph.replay()
            eager.step()
            torch.cuda.synchronize()
            assert _equal(captured, eager)
        assert captured.steps.tolist() == [int(taken) + 2]
