"""Handles that keep a C descriptor between calls, copied and pickled after a call
has made it: a copy's descriptor is its own tensors'."""
import copy
import pickle

import pytest
import torch

import delayed_scaling_linear_amd as dsl


def _bf(*shape):
    return torch.randn(*shape).to(torch.bfloat16)


@pytest.mark.parametrize("make, names", [
    (lambda: dsl.Dropout(0.25, torch.tensor([3, 5])), ("rng",)),
    (lambda: dsl.Adapters(_bf(2, 16, 64), _bf(2, 128, 16), torch.ones(2)), ("a", "b", "alpha"))])
def test_copied_and_pickled(monkeypatch, make, names):
    monkeypatch.setattr(dsl, "_ptr", lambda t, dtype=None, what="": t.data_ptr())
    handle = make()
    used = handle.desc()
    assert handle.desc() is used
    for other in (copy.deepcopy(handle), pickle.loads(pickle.dumps(handle))):
        d = other.desc()
        for name in names:
            mine, its = getattr(handle, name), getattr(other, name)
            assert torch.equal(mine, its) and mine.data_ptr() != its.data_ptr()
            assert getattr(d, name) == its.data_ptr()
        with pytest.raises(Exception, match="cannot assign"):
            setattr(other, names[0], None)
    assert handle.desc() is used
    assert copy.deepcopy(make()).desc() is not None
