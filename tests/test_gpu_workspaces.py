"""One workspace for many batches: that of the largest, its old contents whatever they are."""
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe

pytestmark = pytest.mark.gpu


def test_adapters_in_the_workspace_of_a_larger_batch():
    n_in, n_out, rank = 2560, 264, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g)
    s = moe.AdapterSet(rand(3, rank, n_in).bfloat16(), rand(3, n_out, rank).bfloat16(), torch.ones(3, device="cuda"))
    most = 4096
    ws = torch.empty(moe.moe_adapters_bytes(s, most), dtype=torch.uint8, device="cuda")
    ids = torch.arange(most, device="cuda", dtype=torch.int32) // 100 % 4
    x, base = rand(most, n_in), rand(most, n_out)
    for T in (most, 4080, 2049, 1023, 300, 1):
        print("adapters", T, flush=True)
        out = []
        for w in (torch.empty(moe.moe_adapters_bytes(s, T), dtype=torch.uint8, device="cuda"), ws.fill_(0xFF)):
            o = torch.empty(T, n_out, device="cuda")
            moe.moe_adapters(s, ids[:T], x[:T], base[:T], o, w)
            out.append(o)
        assert torch.equal(out[0], out[1])


def test_balance_in_the_workspace_of_a_larger_batch():
    E, K, most = 128, 4, 10000
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(most, E, device="cuda", generator=g)
    ws = torch.empty(moe.moe_balance_bytes(most, E, 3), dtype=torch.uint8, device="cuda")
    for T in (most, 8192, 8191, 16, 1, 0):
        print("balance", T, flush=True)
        off = torch.tensor([0, T // 3, T // 2], dtype=torch.int32, device="cuda")
        outs = []
        for w in (torch.empty(moe.moe_balance_bytes(T, E, 2), dtype=torch.uint8, device="cuda"), ws.fill_(0xFF)):
            o = [torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"),
                 torch.empty(2, E, dtype=torch.int32, device="cuda"), torch.empty(2, E, device="cuda"),
                 torch.empty(1, device="cuda")]
            moe.moe_route_balance(logits[:T], off, 0.2, *o, w)
            outs.append(o)
        for a, b in zip(*outs):
            assert torch.equal(a, b)
