"""The library's AdamW in the toy stack's training step: against torch's from the
same gradients, and captured."""
import pytest
import torch

import delayed_scaling_linear_amd as dsl
import workloads
from bench import ToyStack, _adamw, _library_adamw, _stack_params, capture_train_step
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def _make():
    stack = ToyStack(dsl, workloads, 2, train=True, modulate="finite")
    x = workloads.uniform_bf16((workloads.TOKENS, workloads.HIDDEN), workloads.SEED_X).to(DEV)
    target = workloads.uniform_bf16((workloads.TOKENS, workloads.HIDDEN),
                                    workloads.SEED_X + 1).to(DEV)
    return stack, x, target


def test_steps_against_torch():
    """One step from zero moments with the same gradients.  Either side's parameter is
    within 4 roundings of 2^-24 of itself and 2^-20 of an update, which is at most lr
    there (m / sqrt(v) is the gradient's sign); so they differ by twice that."""
    stack, x, target = _make()
    own = _library_adamw(dsl, stack)
    with torch.no_grad():
        stack.train_step(x, target)
        start = [t.param.clone() for t in own.tensors]
        grads = [t.grad.clone() for t in own.tensors]
        own.step()
        ours = [t.param.clone() for t in own.tensors]
        for l in range(2):
            for b32, b16 in zip(stack.b32[l], stack.b16[l]):
                assert b32 is None or torch.equal(b32.to(torch.bfloat16), b16)
        params = _stack_params(stack)
        for p, g, s in zip(params, grads, start):
            p.copy_(s)
            assert torch.equal(p.grad, g)
        _adamw(params).step()
    for p, o in zip(params, ours):
        slack = 2 * (4 * 2.0 ** -24 * o.abs().double() + 2.0 ** -20 * 1e-3)
        assert bool(((p.detach().double() - o.double()).abs() <= slack).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step(bits):
    """Replays of the captured step equal eager steps of a copy in every bit."""
    (a, x, target), (b, _, _) = _make(), _make()
    opt_a, opt_b = _library_adamw(dsl, a, bits), _library_adamw(dsl, b, bits)
    with torch.no_grad():
        for _ in range(2):
            a.train_step(x, target, opt_a)
        graph = capture_train_step(b, x, target, opt_b, warmup=2)
        for step in range(3):
            a.train_step(x, target, opt_a)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for s, t in zip(opt_a.tensors, opt_b.tensors):
                for name in ("param", "m", "v", "copy"):
                    u, w = getattr(s, name), getattr(t, name)
                    assert u is None or torch.equal(u.view(torch.uint8), w.view(torch.uint8))
            assert opt_a.steps.tolist() == opt_b.steps.tolist() == [3 + step]
