"""The router, its balance statistics and its gradient on the GPU, against the
plain 64-bit forms, at the sizes and masks where they can go wrong.

Error bounds (u = 2^-24, half a step of fp32): a softmax value e^(l-m)/sum has
the exponent's argument rounded once (relative error |l - m| u in the value;
weighted by the value itself at most 0.37 u absolute), expf within 2 steps (4 u)
above and below the line, the sum's chain of J + 6 additions (J values in a
lane, 6 steps across), one division and two products: RTOL below."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [(1, 1, 1), (1, 512, 10), (3, 2, 2), (5, 8, 2), (4, 60, 6), (257, 64, 8), (9, 65, 64), (33, 188, 1),
          (130, 509, 10), (64, 512, 10), (7, 1000, 16), (6, 2048, 12), (5, 2047, 64)]


def lanes(E):
    j = 1
    while 64 * j < E:
        j *= 2
    return j


def rtol(E, spread=0.0):
    return (spread + lanes(E) + 6 + 8 + 4) * ref.U


def make(T, E, dtype, seed, pad=0, kind="normal"):
    """Device logits (a view with `pad` further columns) and their exact values."""
    rng = np.random.default_rng(seed)
    l = 2.0 * rng.standard_normal((T, E))
    if kind == "closed":
        l[rng.random((T, E)) < 0.5] = -np.inf
        l[0] = -np.inf                          # a row with nothing open
        if T > 1:
            l[1, 1:] = -np.inf                  # ... with one expert open
    elif kind == "ties":
        l = rng.integers(-1, 2, (T, E)).astype(np.float64)
        l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, -0.0, 0.0)
    elif kind == "lowest":                      # masks of the type's lowest value
        low = torch.finfo(DT[dtype]).min
        l[rng.random((T, E)) < 0.5] = low
        l[0] = low
    elif kind == "far":                         # one expert far above the rest
        l[np.arange(T), rng.integers(0, E, T)] += 80.0
    elif kind == "tiny":                        # subnormals and equal magnitudes
        l = rng.integers(-3, 4, (T, E)) * float(torch.finfo(DT[dtype]).tiny) / 4
    whole = torch.zeros(T, E + pad, dtype=DT[dtype])
    whole[:, :E] = torch.from_numpy(l).to(DT[dtype])
    dev = whole.cuda()[:, :E]
    return dev, whole[:, :E].double().numpy()


def run_route(l, K, renorm, scale):
    T = l.shape[0]
    ids = torch.full((T + 2, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, K), 7.0, device="cuda")
    moe.moe_route(l, ids[:T], w[:T], renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    assert (ids[T:] == -7).all() and (w[T:] == 7.0).all()      # rows behind are left alone
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy()


def spread_of(l, ids):
    """|l - m| of the chosen open experts."""
    v = np.take_along_axis(l, ids, 1)
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(v), np.minimum(top - v, 104.0), 0.0)


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "closed", "ties", "lowest", "far", "tiny"])
def test_route(T, E, K, dtype, kind):
    for renorm, scale, pad in ((True, 1.0, 0), (False, 2.5, 3)):
        print("route", T, E, K, dtype, kind, renorm, flush=True)
        dev, l = make(T, E, dtype, seed=T + E, pad=pad, kind=kind)
        ids, w = run_route(dev, K, renorm, scale)
        want_ids, want = ref.route(l, K, renorm, scale)
        assert np.array_equal(ids, want_ids)
        # weights below fp32's normal range keep an absolute step of 2^-149
        tol = np.abs(want) * (rtol(E) + spread_of(l, want_ids) * ref.U + K * ref.U) + scale * 2.0 ** -148
        assert np.all(np.abs(w - want) <= tol), np.max(np.abs(w - want) / (np.abs(want) + 1e-300))


@pytest.mark.parametrize("renorm", [True, False])
def test_route_rows_without_a_softmax(renorm):
    """+inf and NaN: NaN weights, ids still distinct, in range and in order; other rows untouched."""
    l = torch.randn(4, 130, generator=torch.Generator().manual_seed(1))
    l[0, 77] = float("nan")
    l[1, [5, 9]] = float("inf")
    l[2] = float("nan")
    ids, w = run_route(l.cuda(), 4, renorm, 1.0)
    assert np.array_equal(ids, ref.choice(l.double().numpy(), 4))
    assert ids[0, 0] == 77 and ids[1, :2].tolist() == [5, 9] and ids[2].tolist() == [0, 1, 2, 3]
    assert np.isnan(w[0]).all() and np.isnan(w[2]).all() and np.isnan(w[1, :2]).all()
    assert np.isfinite(w[3]).all()


def offsets(T, kind):
    if kind == "one":
        return [0, T]
    if kind == "ragged":                        # empty ones, a short and a long one, padding behind
        n = max(T - 3, 0)
        return sorted([0, 0, min(1, n), n // 3, n // 3, n, n])
    if kind == "each":
        return list(range(T + 1))
    if kind == "front":                         # padding in front too
        return [min(2, T), T]
    return [0, 0, 0]                            # nothing but padding


@pytest.mark.parametrize("T,E,K", [(0, 60, 6), (1, 512, 10), (5, 8, 2), (50, 60, 6), (257, 64, 8), (1030, 188, 3),
                                   (4099, 16, 2), (9, 2047, 64), (130, 512, 10)])
@pytest.mark.parametrize("bounds", ["one", "ragged", "each", "front", "none"])
@pytest.mark.parametrize("dtype,kind", [("f32", "normal"), ("bf16", "closed"), ("f16", "ties")])
def test_balance(T, E, K, bounds, dtype, kind):
    print("balance", T, E, K, bounds, dtype, kind, flush=True)
    dev, l = make(max(T, 1), E, dtype, seed=E, kind=kind)
    dev, l = dev[:T], l[:T]
    off = offsets(T, bounds)
    S = len(off) - 1
    if S == 0:
        off, S = [0, 0], 1
    f32, i32 = torch.float32, torch.int32
    ids = torch.empty(T, K, dtype=i32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    counts = torch.full((S + 1, E), -5, dtype=i32, device="cuda")
    probs = torch.full((S + 1, E), -5.0, device="cuda")
    loss = torch.full((2,), -5.0, device="cuda")
    nb = moe.moe_balance_bytes(T, E, S)
    ws = torch.full((nb + 64,), 0xA5, dtype=torch.uint8, device="cuda")     # old contents do not matter
    moe.moe_route_balance(dev, torch.tensor(off, dtype=i32, device="cuda"), 0.3, ids, w, counts[:S], probs[:S],
                          loss[:1], ws[:nb], renorm=True)
    torch.cuda.synchronize()
    assert (ws[nb:] == 0xA5).all() and (counts[S:] == -5).all() and (probs[S:] == -5.0).all() and loss[1] == -5.0
    if T:
        same_ids, same_w = run_route(dev, K, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), same_ids)
        assert np.array_equal(w.cpu().numpy().view(np.uint32), same_w.view(np.uint32))
        want_c, want_p, want_l = ref.balance(l, ref.choice(l, K), off, 0.3)
    else:
        want_c, want_p, want_l = np.zeros((S, E)), np.zeros((S, E)), 0.0
    assert np.array_equal(counts[:S].cpu().numpy(), want_c)
    # the longest chain of additions in fp32: a range holds at most max(16, T/512 rounded up to a
    # multiple of 16) tokens, dealt to at least 4 waves, then at most 16 waves are added (the
    # ranges are added in 64 bits)
    chain = max(16, (T // 512 // 16 + 1) * 16) / 4 + 16
    got = probs[:S].cpu().numpy()
    tol = want_p * (rtol(E) + (chain + 2) * ref.U) + 0.5 * ref.U
    assert np.all(np.abs(got - want_p) <= tol)
    # the loss is a sum of non-negative products: the same, 6 steps over the lanes, a few products;
    # the 0.5 u of the small probabilities enters times coef / S * counts * E / (K n)
    share = sum(want_c[s].sum() * E / (K * max(off[s + 1] - off[s], 1)) for s in range(S))
    tol = want_l * (rtol(E) + (chain + 16) * ref.U) + 0.3 / S * share * 0.5 * ref.U
    assert abs(float(loss[0]) - want_l) <= tol


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "closed", "lowest", "far"])
def test_route_backward(T, E, K, dtype, kind):
    dev, l = make(T, E, dtype, seed=T * 7 + E, kind=kind)
    ids = ref.choice(l, K)
    rng = np.random.default_rng(E)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    dl = np.float32(0.7)
    i_dev = torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda()
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        spread = np.where(np.isfinite(l), np.minimum(top - l, 104.0), 0.0).max()
    for renorm, bounds, with_dw, pad in ((True, "ragged", True, 0), (False, "ragged", True, 5), (True, None, True, 0),
                                         (False, "one", False, 0), (False, None, True, 0), (True, "front", True, 3),
                                         (False, "none", True, 0)):
        print("backward", T, E, K, dtype, kind, renorm, bounds, with_dw, pad, flush=True)
        off = counts = None
        if bounds:
            off = offsets(T, bounds)
            counts, _, _ = ref.balance(l, ids, off, 1.0)
        want, size = ref.route_backward(l, ids, dw.astype(np.float64) if with_dw else None, renorm, 1.5, off, 0.3,
                                        counts, float(dl))
        out = torch.full((T + 1, E + pad), 9.0, dtype=DT[dtype], device="cuda")
        moe.moe_route_backward(
            dev, i_dev, torch.from_numpy(dw).cuda() if with_dw else None, out[:T, :E], renorm=renorm, scale=1.5,
            seq_off=None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"), coef=0.3,
            counts=None if off is None else torch.from_numpy(counts.astype(np.int32)).cuda(),
            dloss=torch.tensor([dl], device="cuda"))
        torch.cuda.synchronize()
        got = out[:T, :E].double().cpu().numpy()
        # every term carries the softmax's error and the sums' K + 6 further steps; one rounding at the end.
        # Where p underflows fp32 the terms keep an absolute step; in f16 the result has one of 2^-25.
        step = {"f32": 2.0 ** -140, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}[dtype]
        tol = size * (rtol(E) + (K + 16 + 2 * spread) * ref.U) + np.abs(want) * ref.HALF[dtype] + step
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
        assert (out[T:] == 9.0).all() and (out[:, E:] == 9.0).all()


def test_route_backward_in_place_and_repeated_ids():
    """dlogits over the logits; an id named three times adds three times, one out of range nothing."""
    T, E, K = 6, 96, 5
    dev, l = make(T, E, "f32", seed=2)
    ids = np.array([[4, 4, 4, 9, 1], [95, 0, -1, 96, 2 ** 31 - 1]] * 3)
    dw = np.random.default_rng(4).standard_normal((T, K)).astype(np.float32)
    i_dev = torch.from_numpy(ids.astype(np.int32)).cuda()
    want = np.zeros((T, E))
    p = ref.softmax(l)
    for t in range(T):
        g = np.zeros(E)
        for k in range(K):
            if 0 <= ids[t, k] < E:
                g[ids[t, k]] += float(dw[t, k])
        want[t] = p[t] * (g - (p[t] * g).sum())
    moe.moe_route_backward(dev, i_dev, torch.from_numpy(dw).cuda(), dev, renorm=False)
    got = dev.cpu().numpy()
    assert np.all(np.abs(got - want) <= 3.0 * 5 * (rtol(E, 12.0) + 32 * ref.U) * p + 1e-30)


def test_long_rows_pass_32_bit_offsets():
    """Rows 2^31 bytes and more apart: the last row's logits are the ones routed."""
    ld = 1 << 28                                # fp32: 2^30 bytes a row, row 3 beyond 2^31
    whole = torch.zeros(4 * ld, device="cuda")
    view = whole.view(4, ld)[:, :40]
    view.copy_(torch.randn(4, 40, generator=torch.Generator().manual_seed(3)))
    ids, w = run_route(view, 5, True, 1.0)
    assert np.array_equal(ids, ref.choice(view.double().cpu().numpy(), 5))
    d = whole.view(4, ld)[:, 64:104]
    moe.moe_route_backward(view, torch.from_numpy(ids).cuda(), torch.ones(4, 5, device="cuda"), d, renorm=False)
    dense = torch.empty(4, 40, device="cuda")
    moe.moe_route_backward(view.contiguous(), torch.from_numpy(ids).cuda(), torch.ones(4, 5, device="cuda"), dense,
                           renorm=False)
    assert torch.equal(d, dense)


@pytest.mark.parametrize("hidden", [4, 64, 252, 2560])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 10), (130, 2), (5, 17), (64, 33)])
def test_combine_backward(hidden, T, K):
    rng = np.random.default_rng(hidden + T)
    dm = rng.standard_normal((T * K, hidden)).astype(np.float32)
    w = rng.standard_normal((T, K)).astype(np.float32)
    do = rng.standard_normal((T, hidden)).astype(np.float32)
    g = [torch.from_numpy(a).cuda() for a in (dm, w, do)]
    print("combine backward", T, K, hidden, flush=True)
    terms = dm.astype(np.float64).reshape(T, K, hidden) * do[:, None, :]
    want = terms.sum(axis=2)
    # any order of n additions stays within n u of the magnitudes; each product is rounded with its sum
    tol = np.abs(terms).sum(axis=2) * (hidden + 8) * ref.U
    want_ddm = (w[:, :, None] * do[:, None, :]).reshape(T * K, hidden)       # one rounding: exact
    for both in ((True, True), (True, False), (False, True)):
        dw = torch.full((T + 1, K), 3.0, device="cuda")
        ddm = torch.full((T * K + 1, hidden), 3.0, device="cuda")
        moe.moe_combine_backward(g[0], g[1], g[2], dw[:T] if both[0] else None, ddm[:T * K] if both[1] else None)
        torch.cuda.synchronize()
        assert (dw[T:] == 3.0).all() and (ddm[T * K:] == 3.0).all()
        if both[0]:
            assert np.all(np.abs(dw[:T].cpu().numpy() - want) <= tol)
        if both[1]:
            assert np.array_equal(ddm[:T * K].cpu().numpy(), want_ddm)


@pytest.mark.parametrize("T,K,hidden", [(1, 1, 4), (7, 10, 252), (64, 33, 2560), (2500, 10, 1280)])
def test_combine_backward_in_place(T, K, hidden):
    """ddm in dm's own buffer: few tokens, many, and rows past the caches give what separate buffers give."""
    print("combine backward in place", T, K, hidden, flush=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    dm = torch.randn(T * K, hidden, device="cuda", generator=g)
    w = torch.randn(T, K, device="cuda", generator=g)
    do = torch.randn(T, hidden, device="cuda", generator=g)
    want_dw, want = torch.empty_like(w), torch.empty_like(dm)
    moe.moe_combine_backward(dm, w, do, want_dw, want)
    dw = torch.empty_like(w)
    moe.moe_combine_backward(dm, w, do, dw, dm)
    assert torch.equal(dw, want_dw) and torch.equal(dm, want)


def test_same_bits_every_time():
    """Fixed orders of summation: a second run, and one on another stream, give the same bits."""
    T, E, K, S = 3000, 512, 10, 3
    dev, l = make(T, E, "f32", seed=5)
    off = torch.tensor([0, 7, 2000, 2990], dtype=torch.int32, device="cuda")
    dw = torch.randn(T, K, device="cuda")
    outs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None):
        o = [torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"),
             torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(S, E, device="cuda"),
             torch.empty(1, device="cuda"), torch.empty(T, E, device="cuda")]
        ws = torch.empty(moe.moe_balance_bytes(T, E, S), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        moe.moe_route_balance(dev, off, 0.1, *o[:5], ws, renorm=False, stream=stream)
        moe.moe_route_backward(dev, o[0], dw, o[5], renorm=False, seq_off=off, coef=0.1, counts=o[2], stream=stream)
        torch.cuda.synchronize()
        outs.append(o)
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_binding_refusals():
    """What only the binding can see: types, shapes, strides and places of tensors."""
    l, ids, w = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), \
        torch.zeros(4, 2, device="cuda")

    def status(f, *a, **k):
        with pytest.raises(moe.MoeError) as e:
            f(*a, **k)
        return e.value.status

    assert status(moe.moe_route, l.double(), ids, w) == -3
    assert status(moe.moe_route, l, ids.long(), w) == -3
    assert status(moe.moe_route, l, ids, w.half()) == -3
    assert status(moe.moe_route, l.cpu(), ids, w) == -1
    assert status(moe.moe_route, l, ids.cpu(), w) == -1
    assert status(moe.moe_route, l, ids, None) == -1
    assert status(moe.moe_route, l[0], ids, w) == -1
    assert status(moe.moe_route, l.t(), ids, w) == -1                        # rows not dense
    assert status(moe.moe_route, l, ids[:3], w) == -1
    assert status(moe.moe_route, l, ids, torch.zeros(2, 4, device="cuda").t()) == -1
    one = torch.zeros(1, 8, device="cuda").expand(4, 8)
    assert status(moe.moe_route_backward, l, ids, w, one) == -1              # rows written over one another
    assert status(moe.moe_route_backward, l, ids, w, l.half()) == -3
    assert status(moe.moe_combine_backward, l, w, l, w[:, :1].contiguous()) == -1
    assert status(moe.moe_route, one, ids, w) == -1                          # ld < n_expert
    a = torch.zeros(2, 16, 64, device="cuda", dtype=torch.bfloat16)
    s = moe.AdapterSet(a, torch.zeros(2, 32, 16, device="cuda", dtype=torch.bfloat16), torch.ones(2, device="cuda"))
    x, y, i = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 32, device="cuda"), ids[:, 0].contiguous()
    ws = torch.empty(moe.moe_adapters_bytes(s, 4), dtype=torch.uint8, device="cuda")
    assert status(moe.moe_adapters, s, i, x.half(), y.half(), y.half(), ws) == -3      # the set is bf16
    assert status(moe.moe_adapters, s, i, x, y.bfloat16(), y, ws) == -3
    assert status(moe.moe_adapters, s, i[:3], x, y, y, ws) == -1
    assert status(moe.moe_adapters, s, i, x, y, y.clone()[:1].expand(4, 32), ws) == -1
    assert status(moe.moe_adapters, s, i, x, y, y, ws[:-16]) == -4
    assert status(moe.AdapterSet, a, torch.zeros(2, 32, 8, device="cuda", dtype=torch.bfloat16),
                  torch.ones(2, device="cuda")) == -1


def test_no_tokens():
    """Empty batches through the binding: accepted, the statistics written as zeros."""
    e = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")
    l, ids, w = e(0, 60), e(0, 6, dtype=torch.int32), e(0, 6)
    moe.moe_route(l, ids, w)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    counts, probs, loss = torch.ones(2, 60, dtype=torch.int32, device="cuda"), e(2, 60).fill_(1), e(1).fill_(1)
    ws = e(moe.moe_balance_bytes(0, 60, 2), dtype=torch.uint8)
    moe.moe_route_balance(l, off, 0.1, ids, w, counts, probs, loss, ws)
    assert not counts.any() and not probs.any() and not loss.any()
    moe.moe_route_backward(l, ids, w, e(0, 60), seq_off=off, coef=0.1, counts=counts)
    moe.moe_combine_backward(e(0, 64), w, e(0, 64), e(0, 6), e(0, 64))
    s = moe.AdapterSet(e(2, 8, 64, dtype=torch.bfloat16), e(2, 32, 8, dtype=torch.bfloat16), e(2))
    moe.moe_adapters(s, e(0, dtype=torch.int32), e(0, 64), e(0, 32), e(0, 32), e(16, dtype=torch.uint8))
    torch.cuda.synchronize()


def test_many_sequences():
    """As many sequences as tokens and thousands more, empty: every one is written."""
    T, E, K, S = 300, 40, 3, 9000
    dev, l = make(T, E, "f32", seed=8)
    rng = np.random.default_rng(1)
    off = np.sort(np.concatenate([[0], rng.integers(0, T + 1, S - 1), [T]]))
    o = [torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"),
         torch.full((S, E), -1, dtype=torch.int32, device="cuda"), torch.full((S, E), -1.0, device="cuda"),
         torch.empty(1, device="cuda")]
    ws = torch.full((moe.moe_balance_bytes(T, E, S),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_route_balance(dev, torch.from_numpy(off.astype(np.int32)).cuda(), 0.3, *o, ws)
    want_c, want_p, want_l = ref.balance(l, ref.choice(l, K), off, 0.3)
    assert np.array_equal(o[2].cpu().numpy(), want_c)
    assert np.all(np.abs(o[3].cpu().numpy() - want_p) <= want_p * (rtol(E) + 40 * ref.U) + 0.5 * ref.U)
    # the probabilities' 0.5 u enter times coef / S * E / (K n) * K n per filled sequence
    filled = np.count_nonzero(np.diff(off))
    assert abs(float(o[4]) - want_l) <= want_l * (rtol(E) + 64 * ref.U) + 0.3 / S * filled * E * 0.5 * ref.U
    # and the gradient, with every token in a sequence of its own length
    d = torch.empty(T, E, device="cuda")
    moe.moe_route_backward(dev, o[0], None, d, seq_off=torch.from_numpy(off.astype(np.int32)).cuda(), coef=0.3,
                           counts=o[2])
    want, size = ref.route_backward(l, ref.choice(l, K), None, True, 1.0, off, 0.3, want_c)
    assert np.all(np.abs(d.cpu().numpy() - want) <= size * (rtol(E, 16.0) + 32 * ref.U) + 1e-38)
