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


# experts per lane 1, 1, 2, 8, 16, 32: a workgroup takes several rounds of rows above 512 times its
# waves (16; 8 and 4 for the last two)
@pytest.mark.parametrize("T,E,K", [(20011, 40, 3), (8193, 64, 8), (17000, 100, 6), (9000, 512, 10), (9001, 509, 3),
                                   (5000, 1000, 16), (130, 1000, 16), (130, 100, 6), (3333, 2047, 12)])
@pytest.mark.parametrize("bounds,dtype,kind", [("one", "f32", "normal"), ("ragged", "bf16", "closed"),
                                               ("steps", "f32", "closed"), ("steps", "f16", "ties")])
def test_balance_in_several_rounds(T, E, K, bounds, dtype, kind):
    """Sequences that end anywhere in a workgroup's range, against the plain form."""
    print("balance", T, E, K, bounds, dtype, kind, flush=True)
    dev, l = make(T, E, dtype, seed=T, kind=kind)
    off = sorted({5, *range(5, T - 9, 37 if T < 9000 else 211), T - 9}) if bounds == "steps" else offsets(T, bounds)
    S = len(off) - 1
    ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    counts = torch.full((S + 1, E), -5, dtype=torch.int32, device="cuda")
    probs = torch.full((S + 1, E), -5.0, device="cuda")
    loss = torch.full((2,), -5.0, device="cuda")
    nb = moe.moe_balance_bytes(T, E, S)
    ws = torch.full((nb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_route_balance(dev, torch.tensor(off, dtype=torch.int32, device="cuda"), 0.3, ids, w, counts[:S],
                          probs[:S], loss[:1], ws[:nb], renorm=False, scale=1.5)
    torch.cuda.synchronize()
    assert (ws[nb:] == 0xA5).all() and (counts[S:] == -5).all() and (probs[S:] == -5.0).all() and loss[1] == -5.0
    want_ids, want_w = ref.route(l, K, False, 1.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.all(np.abs(w.cpu().numpy() - want_w)
                  <= want_w * (rtol(E) + (spread_of(l, want_ids) + K) * ref.U) + 1.5 * 2.0 ** -148)
    want_c, want_p, want_l = ref.balance(l, want_ids, off, 0.3)
    assert np.array_equal(counts[:S].cpu().numpy(), want_c)
    # a range holds at most T / 512 rows rounded up to the waves, dealt to them, and then at most 16 waves are added
    chain = max(16, (T // 512 // 16 + 1) * 16) / 4 + 16
    assert np.all(np.abs(probs[:S].cpu().numpy() - want_p) <= want_p * (rtol(E) + (chain + 2) * ref.U) + 0.5 * ref.U)
    # a probability's 0.5 u enters times coef / S * counts * E / (K n)
    share = sum(want_c[s].sum() * E / (K * max(off[s + 1] - off[s], 1)) for s in range(S))
    assert abs(float(loss[0]) - want_l) <= want_l * (rtol(E) + (chain + 16) * ref.U) + 0.3 / S * share * 0.5 * ref.U


@pytest.mark.parametrize("T,E,K", [(65537, 8, 2), (70001, 60, 3), (66000, 130, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_rows_than_waves(T, E, K, dtype):
    """Above 65,536 rows the router's and the gradient's waves take several."""
    print("route", T, E, K, dtype, flush=True)
    dev, l = make(T, E, dtype, seed=E)
    ids, w = run_route(dev, K, True, 1.0)
    want_ids, want = ref.route(l, K, True)
    assert np.array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= want * (rtol(E) + (spread_of(l, want_ids) + K) * ref.U) + 2.0 ** -148)
    rng = np.random.default_rng(T)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    off = [0, T // 2, T - 5]
    counts, _, _ = ref.balance(l, ids, off, 1.0)
    out = torch.full((T + 1, E), 9.0, dtype=dev.dtype, device="cuda")
    moe.moe_route_backward(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), out[:T], renorm=False,
                           seq_off=torch.tensor(off, dtype=torch.int32, device="cuda"), coef=0.3,
                           counts=torch.from_numpy(counts.astype(np.int32)).cuda())
    torch.cuda.synchronize()
    d, size = ref.route_backward(l, ids, dw.astype(np.float64), False, 1.0, off, 0.3, counts)
    spread = (l.max(axis=1) - l.min(axis=1)).max()
    tol = size * (rtol(E) + (K + 16 + 2 * spread) * ref.U) + np.abs(d) * ref.HALF[dtype] + 2.0 ** -133
    assert np.all(np.abs(out[:T].double().cpu().numpy() - d) <= tol)
    assert (out[T:] == 9.0).all()


@pytest.mark.parametrize("E", [60, 512, 1000])
def test_padding_that_is_not_a_number_joins_nothing(E):
    """NaN and infinities in rows outside the sequences leave the statistics and the other rows' gradient alone."""
    T, K, off = 700, 4, [9, 300, 650]
    dev, _ = make(T, E, "f32", seed=E)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[off[0]:off[-1]] = True
    inside = inside.cuda()
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        l = dev.clone()
        l[~inside] = fill
        ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        counts = torch.empty(2, E, dtype=torch.int32, device="cuda")
        probs, loss = torch.empty(2, E, device="cuda"), torch.empty(1, device="cuda")
        so = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = torch.full((moe.moe_balance_bytes(T, E, 2),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_route_balance(l, so, 0.3, ids, w, counts, probs, loss, ws)
        dw = torch.ones_like(w)
        dw[~inside] = fill
        d = torch.empty_like(l)
        moe.moe_route_backward(l, ids, dw, d, seq_off=so, coef=0.3, counts=counts)
        outs.append((counts, probs, loss, ids[inside], w[inside], d[inside]))
    for o in outs[1:]:
        for a, b in zip(o, outs[0]):
            assert torch.equal(a, b)
