"""The combine's gradient in the forms that few rows do not reach."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu


def test_largest_launch():
    """2^26 - 4 tokens of one row: 2^24 - 1 workgroups."""
    T, H = 2 ** 26 - 4, 4
    print("combine backward", T, H, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    dm, do = (torch.randn(T, H, device="cuda", generator=g) for _ in range(2))
    w = torch.randn(T, 1, device="cuda", generator=g)
    dw, ddm = torch.full_like(w, 3.0), torch.full_like(dm, 3.0)
    moe.moe_combine_backward(dm, w, do, dw, ddm)
    torch.cuda.synchronize()
    assert torch.equal(ddm, w * do)                       # one rounding
    terms = dm.double() * do.double()
    # four products, each rounded with its sum, and sums with zeros
    assert bool(((dw.double() - terms.sum(dim=1, keepdim=True)).abs()
                 <= terms.abs().sum(dim=1, keepdim=True) * 4 * ref.U).all())
