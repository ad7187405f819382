"""The combine's gradient in the forms that few rows do not reach."""
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


@pytest.mark.parametrize("T,K,H", [(2048, 1, 4), (2100, 10, 252), (1030, 17, 64), (4100, 8, 256), (3000, 5, 64),
                                   (2500, 10, 1280), (9001, 3, 320), (2049, 33, 132)])
def test_many_rows_against_64_bits(T, K, H):
    """From 2,048 (token, eight rows) jobs on, a wave has its own; rows over 32 MB pass the caches."""
    print("combine backward", T, K, H, T * K * H * 4 >> 20, "MB", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dm = torch.randn(T * K, H, device="cuda", generator=g)
    w, do = torch.randn(T, K, device="cuda", generator=g), torch.randn(T, H, device="cuda", generator=g)
    terms = dm.double().view(T, K, H) * do.double()[:, None, :]
    want = terms.sum(dim=2)
    # any order of H additions stays within H u of the magnitudes; each product is rounded with its sum
    tol = terms.abs().sum(dim=2) * (H + 8) * ref.U
    del terms
    want_ddm = (w[:, :, None] * do[:, None, :]).view(T * K, H)       # one rounding: exact
    for with_dw, with_ddm in ((True, True), (True, False), (False, True)):
        dw = torch.full((T + 1, K), 3.0, device="cuda")
        ddm = torch.full((T * K + 1, H), 3.0, device="cuda")
        moe.moe_combine_backward(dm, w, do, dw[:T] if with_dw else None, ddm[:T * K] if with_ddm else None)
        torch.cuda.synchronize()
        assert (dw[T:] == 3.0).all() and (ddm[T * K:] == 3.0).all()
        if with_dw:
            assert bool(((dw[:T].double() - want).abs() <= tol).all())
        if with_ddm:
            assert torch.equal(ddm[:T * K], want_ddm)
