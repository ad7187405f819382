"""The C ABI of include/moe_layer.h on the host (no GPU), at its limits."""
import pytest

from tests.test_layer_abi_host import EINVAL, combine


@pytest.mark.parametrize("tokens,topk", [((1 << 26) - 3, 1), ((1 << 26) - 2, 8), ((1 << 26) - 1, 5), ((1 << 25) - 1, 9)])
def test_combine_backward_refuses_a_launch_of_2_to_32_threads(tokens, topk):
    """A wave per token and eight rows, four to a workgroup of 256: 2^24 workgroups are one too many."""
    assert combine(tokens=tokens, topk=topk) == EINVAL
