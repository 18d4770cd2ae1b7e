"""Workspace sizes of the adapters, on the CPU."""
import ctypes

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


def test_a_program_that_does_not_train_keeps_the_sums_alone():
    """No demand for the weight gradients' operands and partial sums: 512
    requests of 512 adapters took 2 GiB for 0.1 MiB."""
    whole, part = dsl.fp8_adapter_workspace_bytes, dsl.fp8_adapter_fwd_workspace_bytes
    for rows, adapters, rank, n_in, n_out in ((1, 1, 8, 8, 8), (16, 4, 16, 64, 128),
                                              (64, 32, 16, 2048, 8192), (8192, 9, 64, 2048, 6144),
                                              (512, 512, 64, 8192, 8192), (1 << 20, 4, 128, 64, 64)):
        sizes = rows, adapters, rank, n_in, n_out
        # one part's sums at the least, of no more than 2 MiB beside them
        assert 4 * rows * rank <= part(*sizes) <= max(min(1 << 20, whole(*sizes)),
                                                      4 * rank * max(rows, min(16 * rows, 33280)) + 256)
        assert part(*sizes) <= whole(*sizes)
    for adapters, rank in ((1, 8), (64, 64), (600, 128)):
        sizes = [part(rows, adapters, rank, 2048, 8192) for rows in range(1, 2600)]
        assert sizes == sorted(sizes)
    with pytest.raises(dsl.Fp8Error):
        part(8, 1, 12, 64, 64)


def test_calls_without_weight_gradients_ask_for_no_more():
    """Through the C ABI, up to the check that comes behind the workspace's."""
    L = dsl.lib()
    sizes = 512, 512, 64, 8192, 8192
    plan_size = dsl.fp8_adapter_plan_bytes(512, 512)
    w = ctypes.byref(dsl._AdaptersDesc(0x10000, 0x20000, 0x30000, 512, 64, 8192, 8192))
    whole, part = dsl.fp8_adapter_workspace_bytes(*sizes), dsl.fp8_adapter_fwd_workspace_bytes(*sizes)
    assert whole > 1000 * part
    fwd = lambda size, x=None: L.fp8_adapter_fwd(w, 0x40000, plan_size, None, x, 8192, None, 0, 0x3000,
                                                 8192, 512, None, 0x50000, size, None)
    assert fwd(part) == -1 and fwd(part - 1) == -2
    bwd = lambda size, dy=None, da=None: L.fp8_adapter_backward(
        w, 0x40000, plan_size, None, 0x1000, 8192, dy, 8192, 0x2000, None, 0, 0x3000, 8192, 512, da,
        da, 1, 0x50000, size, None)
    assert bwd(part) == -1 and bwd(part - 1) == -2
    assert bwd(whole, da=0x6000) == -1 and bwd(part, da=0x6000) == -2 and bwd(whole - 1, da=0x6000) == -2
