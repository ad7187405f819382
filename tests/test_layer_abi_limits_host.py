"""The C ABI of include/moe_layer.h at its limits, and what its binding and the layer refuse (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_moe_expert_scatter_amd import _lib, _steps
from quantized_moe_expert_scatter_amd import workloads as wl
from quantized_moe_expert_scatter_amd.layer import DeviceLayer
from tests.test_layer_abi_host import EINVAL, ESIZE, adapters, combine, make_set


@pytest.mark.parametrize("tokens,topk", [((1 << 26) - 3, 1), ((1 << 26) - 2, 8), ((1 << 26) - 1, 5), ((1 << 25) - 1, 9)])
def test_combine_backward_refuses_a_launch_of_2_to_32_threads(tokens, topk):
    """A wave per token and eight rows, four to a workgroup of 256: 2^24 workgroups are one too many."""
    assert combine(tokens=tokens, topk=topk) == EINVAL


@pytest.mark.parametrize("E,S", [(8, 1), (100, 5), (512, 1), (1000, 2), (2048, 3)])
def test_balance_workspace_of_a_batch_serves_every_smaller_one(E, S):
    sizes = [_steps.moe_balance_bytes(T, E, S) for T in [*range(0, 20000, 7), *range(20000, 2 ** 22, 9973), 2 ** 31 - 1]]
    assert sizes == sorted(sizes) and sizes[0] > 0
    some = [_steps.moe_balance_bytes(12345, E, s) for s in range(1, 200)]
    assert some == sorted(some)


@pytest.mark.parametrize("rank,n_in", [(8, 8), (64, 2560), (24, 1160), (256, 1 << 24)])
def test_adapter_workspace_of_a_batch_serves_every_smaller_one(rank, n_in):
    s = make_set(rank=rank, n_in=n_in)
    size = lambda T: _steps.lib().moe_adapters_bytes(ctypes.byref(s), T)
    sizes = [size(T) for T in [*range(0, 9000), *range(9000, 1 << 24, 99991), 1 << 24]]
    assert sizes == sorted(sizes) and sizes[1] > 0


def test_a_call_takes_the_workspace_of_a_larger_batch():
    """2,049 rows have two slices of the contraction and so more to hold than 4,096 with one; a call is refused
    for less than its own."""
    big = dict(rank=64, n_in=2560)
    s = make_set(**big)
    size = lambda T: _steps.lib().moe_adapters_bytes(ctypes.byref(s), T)
    assert 0 < size(2049) <= size(4096)
    assert adapters(big, tokens=2049, ldx=2560, nb=2 * 2049 * 64 * 4 - 1) == ESIZE


def test_binding_refuses_sizes_past_an_int():
    """ctypes would cut them to their low 32 bits: columns, matrix sizes, and the size queries' arguments."""
    far = (1 << 32) + 8
    bf16 = dict(dtype=torch.bfloat16, device="meta")
    with pytest.raises(_lib.MoeError, match=str(far)) as e:
        _steps._matrix(torch.empty(1, far, device="meta"), "logits")
    assert e.value.status == EINVAL
    for a, b in (((far, 8, 8), (far, 8, 8)), ((1, far, 8), (1, 8, far)), ((1, 8, far), (1, 8, 8)),
                 ((1, 8, 8), (1, far, 8))):
        with pytest.raises(_lib.MoeError, match=str(far)) as e:
            _steps.AdapterSet(torch.empty(a, **bf16), torch.empty(b, **bf16), torch.empty(a[0], device="meta"))
        assert e.value.status == EINVAL
    for args in ((far, 8, 1), (8, far, 1), (8, 8, far)):
        assert _steps.moe_balance_bytes(*args) == 0
    held = type("Set", (), {"ref": ctypes.byref(make_set())})
    assert _steps.moe_adapters_bytes(held, 8) > 0 and _steps.moe_adapters_bytes(held, far) == 0


@pytest.mark.parametrize("shape", [(4, 9), (4, 7), (5, 8), (4, 8, 1)])
def test_layer_refuses_logits_of_another_shape(shape):
    """Experts that the layer does not have would be chosen, and their rows left out of the plan."""
    L = wl.make_layer(wl.small_config("shape", 4, 128, 64, 8, 2, seed=1))
    with pytest.raises(ValueError, match="logits"):
        DeviceLayer(L.x, None, L.w_gu, L.w_down, logits=np.zeros(shape, np.float32), topk=2)
