"""Adapters: what the two-launch forms must keep, which small batches do not
reach.  Batches of 300 rows take the 16-row update, 8,200 rows the 64-row one
(ranks up to 64), rank 72 the update for any rank.

Bounds: u = 2^-24 is half a step of fp32."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TYPES = [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]
FORMS = [(300, 8), (300, 24), (300, 48), (300, 72), (8200, 24), (8200, 64), (8200, 72)]


def run(a, b, scale, ids, x, base, ranks=None):
    s = moe.AdapterSet(a, b, scale, rank=ranks)
    T = ids.numel()
    ws = torch.full((moe.moe_adapters_bytes(s, T),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(base)
    moe.moe_adapters(s, ids, x, base, out, ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,rank", FORMS)
def test_low_rank_values_of_16_bit_rows_are_fp32(T, rank, dtype):
    """base takes the update away but for its own rounding, so that the result shows the update's
    low bits.  Every factor is positive: the update's magnitudes are the update itself, and a
    sum of n_in, then rank terms, the scale and the base's addition stay within
    (n_in + rank + 8) u of it; the result is rounded once."""
    print("16-bit rows", T, rank, dtype, flush=True)
    n_in, n_out, dt = 16, 72, DT[dtype]
    rng = np.random.default_rng(T + rank)
    pos = lambda *shape: torch.from_numpy(rng.random(shape) + 0.5).to(dt)
    a, b, x = pos(2, rank, n_in), pos(2, n_out, rank) / 64, pos(T, n_in)
    scale = torch.tensor([0.75, 1.25])
    ids = torch.from_numpy(rng.integers(0, 2, T).astype(np.int32))
    i = ids.long()
    update = np.empty((T, n_out))
    for k in range(2):
        on = np.nonzero(i.numpy() == k)[0]
        h = x.double().numpy()[on] @ a[k].double().numpy().T
        update[on] = float(scale[k]) * (h @ b[k].double().numpy().T)
    base = torch.from_numpy(-update).to(dt)
    want = base.double().numpy() + update
    out = run(*(t.cuda() for t in (a, b, scale, ids, x, base))).double().cpu().numpy()
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    tol = update * (n_in + rank + 8) * ref.U + np.abs(want) * ref.HALF[dtype] * 1.01 + tiny
    err = np.abs(out - want)
    assert np.all(err <= tol), (np.max(err / tol), np.mean(err > tol))


@pytest.mark.parametrize("T,rank", FORMS)
@pytest.mark.parametrize("where", ["a", "b"])
def test_fp16_matrices_beside_fp32_values_lose_nothing(T, rank, where):
    """One product per result: w = 1 + 7/1024 is two bf16 parts, v = 1 + 2^-8 + .. three, the last of
    255 * 2^-23, so that the product of their low parts is 3.45 u of the whole and always of the same sign.  Kept,
    the result is off by the last addition (at most a whole step, 2 u, if it truncates) and by the
    others, below 2^-8 of that; the two uses of w have nothing else to round."""
    print("fp16 matrices", T, rank, where, flush=True)
    n_in, n_out = 8, 72
    w = 1.0 + 7.0 / 1024
    a, b = torch.zeros(1, rank, n_in, dtype=torch.float16), torch.zeros(1, n_out, rank, dtype=torch.float16)
    a[0, 0, 0] = w if where == "a" else 1.0
    b[0, :, 0] = w if where == "b" else 1.0
    x = torch.zeros(T, n_in)
    x[:, 0] = 1.0 + 2.0 ** -8 + torch.arange(T) % 8 * 2.0 ** -14 + 255 * 2.0 ** -23      # below 1.005
    want = x[:, :1].double() * w
    out = run(a.cuda(), b.cuda(), torch.ones(1, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"),
              x.cuda(), torch.zeros(T, n_out, device="cuda")).double().cpu()
    off = ((out - want) / want).abs().max().item() / ref.U
    assert off <= 2.0 * (1 + 2.0 ** -7), off


def inputs(T, n, rank, dtype, wdtype, n_in=72, n_out=136, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda dt, *shape: torch.randn(*shape, generator=g).to(DT[dt]).cuda()
    ids = (torch.arange(T, dtype=torch.int32) * n // T).cuda()
    return dict(a=rand(wdtype, n, rank, n_in), b=rand(wdtype, n, n_out, rank), scale=torch.ones(n, device="cuda"),
                ids=ids, x=rand(dtype, T, n_in), base=rand(dtype, T, n_out))


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,rank", FORMS)
def test_what_is_not_finite_stays_in_its_rows(T, rank, dtype, wdtype):
    """NaN or an infinity in a row of x reaches that row, in a or b of an adapter its rows, and no others."""
    print("not finite", T, rank, dtype, wdtype, flush=True)
    d = inputs(T, 5, rank, dtype, wdtype)
    clean = run(**d)
    rows = [0, T // 2 + 1, T - 1]
    d["x"][rows[0], 3], d["x"][rows[1], 0], d["x"][rows[2]] = float("nan"), float("inf"), float("-inf")
    d["a"][1].fill_(float("nan"))
    d["b"][3, :, 0] = float("inf")
    got = run(**d)
    touched = (d["ids"] == 1) | (d["ids"] == 3)
    touched[rows] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert not got[touched].isfinite().any()


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,rank", FORMS)
def test_what_lies_past_an_adapters_own_rank_is_not_read(T, rank, dtype, wdtype):
    """Adapters of several ranks in a tile: NaN and infinities in the rows of a and columns of b past each
    one's own give what zeros give, and ranks outside [0, rank] what the nearest one gives."""
    print("own ranks", T, rank, dtype, wdtype, flush=True)
    n = 6
    d = inputs(T, n, rank, dtype, wdtype, seed=1)
    d["ids"] = (torch.arange(T, dtype=torch.int32) % n).cuda()
    own = [0, 1, rank - 3, rank // 2, rank, 5]
    d["ranks"] = torch.tensor(own, dtype=torch.int32, device="cuda")
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        for i, r in enumerate(own):
            d["a"][i, r:] = fill
            d["b"][i, :, r:] = fill
        outs.append(run(**d))
    d["ranks"][0], d["ranks"][4] = -2 ** 31, 2 ** 31 - 1
    outs.append(run(**d))
    assert outs[0].isfinite().all() and torch.equal(outs[0][::n], d["base"][::n])
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert not torch.equal(outs[0][1::n], d["base"][1::n])


@pytest.mark.parametrize("T,rank", [(8, 16)] + FORMS)
@pytest.mark.parametrize("wdtype", ["bf16", "f16"])
@pytest.mark.parametrize("e", [-112, -118, -126])
def test_tiny_values_lose_no_more_than_the_smallest_normal_number(T, rank, wdtype, e):
    """A product below 2^-126 may count as 0, and so may a part of a value: at most six products of two
    parts for each of the formula's, of factors below 4 and 2^-126, so 2^-126 * 6 * 4 a term of a * x, and as
    much a term of b * h."""
    print("tiny", T, rank, wdtype, e, flush=True)
    n_in, n_out = 64, 72
    g = torch.Generator().manual_seed(2)
    rand = lambda *shape: torch.rand(*shape, generator=g) * 2 - 1
    a, b = rand(1, rank, n_in).to(DT[wdtype]), rand(1, n_out, rank).to(DT[wdtype])
    x = rand(T, n_in) * 2.0 ** e
    out = run(a.cuda(), b.cuda(), torch.ones(1, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"),
              x.cuda(), torch.zeros(T, n_out, device="cuda")).double().cpu()
    A, B, X = a[0].double(), b[0].double(), x.double()
    want = X @ A.t() @ B.t()
    size = X.abs() @ A.abs().t() @ B.abs().t()
    lost = 2.0 ** -126 * 24 * (n_in * B.abs().sum(dim=1) + rank)
    assert bool(((out - want).abs() <= size * (n_in + rank + 8) * ref.U + lost).all())
