"""Workspace sizes of the adapters, on the CPU."""
import pytest

import delayed_scaling_linear_amd as dsl


@pytest.mark.parametrize("n_in, n_out", [(64, 64), (2048, 2048), (2048, 8192), (8192, 8192),
                                         (1 << 17, 520)])
@pytest.mark.parametrize("adapters", [1, 8, 64, 600])
def test_a_larger_batch_never_asks_for_less(adapters, n_in, n_out):
    """The workspace of a program's largest batch serves its smaller ones."""
    size = lambda rows, count, rank: dsl.fp8_adapter_workspace_bytes(rows, count, rank, n_in, n_out)
    for rank in (8, 16, 40, 64, 72, 128):
        sizes = [size(rows, adapters, rank) for rows in range(1, 2600)]
        assert sizes == sorted(sizes)
    for rows in (1, 33, 300, 2018, 8192, 1 << 20):
        sizes = [size(rows, adapters, rank) for rank in range(8, 129, 8)]
        assert sizes == sorted(sizes)
        sizes = [size(rows, count, 64) for count in range(1, 4097, 13)]
        assert sizes == sorted(sizes)
