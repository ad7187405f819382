"""The router, its statistics and its gradient at sizes that small batches do
not reach: row numbers up to 2^31 - 1, workgroups that take several rounds of
rows, loops over rows, every number of experts per lane."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from tests import layer_ref as ref
from tests.test_gpu_router import make, offsets, rtol, run_route, spread_of

pytestmark = pytest.mark.gpu


def test_balance_of_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of one expert: every row is routed once, and nothing else is."""
    T = 2 ** 31 - 1
    print("balance", T, "rows", flush=True)
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 7.0, device="cuda")
    counts = torch.empty(2, 1, dtype=torch.int32, device="cuda")
    probs, loss = torch.empty(2, 1, device="cuda"), torch.empty(1, device="cuda")
    off = torch.tensor([0, 3, T], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_balance_bytes(T, 1, 2), dtype=torch.uint8, device="cuda")
    moe.moe_route_balance(logits, off, 0.5, ids, w, counts, probs, loss, ws)
    torch.cuda.synchronize()
    assert counts.view(-1).tolist() == [3, T - 3] and probs.view(-1).tolist() == [1.0, 1.0]
    assert abs(float(loss) - 0.5) <= 0.5 * 4 * ref.U
    # piece by piece: the whole would take further buffers of this size
    for part, value in ((ids, 0), (w, 1.0)):
        for p in part.view(-1).split(1 << 28):
            assert bool((p == value).all())


def test_gradient_of_as_many_sequences_as_an_int_counts():
    """2^31 - 1 sequences, all empty but the last two, and rows behind them: each row's sequence is
    found, padding has none."""
    T, E, K, S = 40, 2, 1, 2 ** 31 - 1
    print("gradient", S, "sequences", flush=True)
    off = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    off[S - 1], off[S] = 10, 30
    counts = torch.full((S, E), 1000, dtype=torch.int32, device="cuda")      # another sequence's would show
    mine = np.array([[10, 0], [5, 15]])
    counts[S - 2:] = torch.from_numpy(mine.astype(np.int32))
    dev, l = make(T, E, "f32", seed=1)
    ids = ref.choice(l, K)
    d = torch.full((T, E), 5.0, device="cuda")
    # coef / n_seq is 1 here and in the plain form of the two sequences
    moe.moe_route_backward(dev, torch.from_numpy(ids.astype(np.int32)).cuda(), None, d, seq_off=off,
                           coef=float(2 ** 31), counts=counts)
    torch.cuda.synchronize()
    want, size = ref.route_backward(l, ids, None, True, 1.0, [0, 10, 30], 2.0, mine)
    assert np.all(np.abs(d.cpu().numpy() - want) <= size * (rtol(E, 16.0) + 32 * ref.U))
    assert not d[30:].any() and d[:30].any(dim=1).all()
