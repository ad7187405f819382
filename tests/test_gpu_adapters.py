"""Per-request low-rank adapters on the GPU against the plain 64-bit form:
one token to a few hundred, contiguous requests and shuffled rows, every type
combination, odd ranks, strided rows, rows without an adapter.

Bounds (u = 2^-24): the update is a chain of n_in, then rank additions whose
worst case is (n_in + rank + 8) u of the magnitudes; that is loose, so the
root mean square over a case is held to sqrt(n_in/8 + rank) u of the magnitudes' root
mean square as well: rounding errors of a chain add like a random walk, a
lost low part of the activations (2^-17) or of h does not pass."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TYPES = [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]


def values(a, dtype):
    t = torch.from_numpy(a).to(DT[dtype])
    return t, t.double().numpy()


def make(T, n, rank, n_in, n_out, dtype, wdtype, ids, seed=0, pad=0):
    rng = np.random.default_rng(seed)
    d = {}
    d["a"], a = values(rng.standard_normal((n, rank, n_in)) / np.sqrt(n_in), wdtype)
    d["b"], b = values(rng.standard_normal((n, n_out, rank)), wdtype)
    x = rng.standard_normal((T, n_in + pad))
    base = rng.standard_normal((T, n_out + 2 * pad))
    d["x"], x = values(x, dtype)
    d["base"], base = values(base, dtype)
    scale = (rng.random(n) + 0.5).astype(np.float32)
    ranks = rng.integers(0, rank + 1, n).astype(np.int32)
    ranks[0] = rank
    if n > 1:
        ranks[-1] = 0
    d = {k: v.cuda() for k, v in d.items()}
    d["x"], d["base"] = d["x"][:, :n_in], d["base"][:, :n_out]
    d["scale"], d["ranks"] = torch.from_numpy(scale).cuda(), torch.from_numpy(ranks).cuda()
    d["ids"] = torch.from_numpy(np.asarray(ids, np.int32)).cuda()
    want = ref.adapters(x[:, :n_in], base[:, :n_out], ids, a, b, scale.astype(np.float64), ranks)
    return d, want


def check(out, want, dtype, n_in, rank):
    out = out.double().cpu().numpy()
    value, update, size = want
    err = np.abs(out - value)
    half = ref.HALF[dtype]
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    assert np.all(err <= size * (n_in + rank + 8) * ref.U + np.abs(value) * (half + 2 * ref.U) * 1.01 + tiny)
    if dtype == "f32" and size.any():
        # the last rounding is of the sum with base
        rms = np.sqrt((err ** 2).mean())
        allowed = np.sqrt(n_in / 8 + rank) * ref.U * np.sqrt((size ** 2).mean()) + ref.U * np.sqrt((value ** 2).mean())
        assert rms <= allowed, (rms, allowed)


def run(d, T, out=None):
    s = moe.AdapterSet(d["a"], d["b"], d["scale"], rank=d["ranks"])
    nb = moe.moe_adapters_bytes(s, T)
    ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN patterns
    if out is None:
        whole = torch.full((T + 1, s.n_out), 9.0, dtype=d["base"].dtype, device="cuda")
        moe.moe_adapters(s, d["ids"], d["x"], d["base"], whole[:T], ws[:nb])
        torch.cuda.synchronize()
        assert (whole[T:] == 9.0).all()
        out = whole[:T]
    else:
        moe.moe_adapters(s, d["ids"], d["x"], d["base"], out, ws[:nb])
        torch.cuda.synchronize()
    assert (ws[nb:] == 0xFF).all()
    return out


def ids_of(kind, T, n, seed=1):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.zeros(T, np.int64)
    if kind == "runs":                          # requests of ragged lengths, some without an adapter
        ids, i = [], 0
        while len(ids) < T:
            ids += [rng.integers(-1, n)] * int(rng.integers(1, 70))
        return np.array(ids[:T])
    if kind == "mixed":
        return rng.integers(-1, n, T)
    if kind == "wild":                          # values outside the set: no adapter
        return rng.choice([-2 ** 31, -1, 0, n - 1, n, 2 ** 31 - 1], T)
    return np.full(T, -1)


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,n,rank,n_in,n_out", [
    (1, 1, 8, 8, 8), (1, 4, 16, 2560, 1280), (2, 3, 8, 64, 136), (15, 5, 24, 72, 64), (16, 2, 16, 256, 256),
    (17, 4, 64, 520, 264), (48, 32, 16, 2560, 128), (65, 3, 40, 96, 2560), (130, 7, 8, 1000, 72),
    (200, 3, 128, 136, 200), (33, 2, 256, 40, 48), (130, 7, 64, 1000, 2056), (97, 40, 128, 72, 136),
    (256, 3, 64, 264, 72), (250, 300, 56, 88, 96), (64, 2, 256, 40, 48), (129, 9, 104, 32, 1032)])
@pytest.mark.parametrize("kind", ["one", "runs", "mixed", "wild", "none"])
def test_adapters(T, n, rank, n_in, n_out, dtype, wdtype, kind):
    print("adapters", T, n, rank, n_in, n_out, dtype, wdtype, kind, flush=True)
    ids = ids_of(kind, T, n)
    d, want = make(T, n, rank, n_in, n_out, dtype, wdtype, ids, seed=T)
    out = run(d, T)
    check(out, want, dtype, n_in, rank)
    # rows without an adapter: base, bit for bit
    off = (ids < 0) | (ids >= n)
    if off.any():
        rows = torch.from_numpy(np.nonzero(off)[0]).cuda()
        assert torch.equal(out[rows], d["base"][rows])
    # in place: the same bits
    inner = d["base"].clone()
    d["base"] = inner
    assert torch.equal(run(d, T, out=inner), out)


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,rank", [(257, 16), (700, 32), (1500, 64), (4100, 32), (4101, 8), (8193, 8), (8200, 48), (8250, 72)])
def test_many_rows(T, rank, dtype, wdtype):
    """Long batches, contiguous and shuffled: a row's result does not depend on its neighbours."""
    n, n_in, n_out = 5, 264, 328
    print("adapters, many rows", T, rank, dtype, wdtype, flush=True)
    ids = ids_of("runs", T, n, seed=T)
    d, want = make(T, n, rank, n_in, n_out, dtype, wdtype, ids, seed=3, pad=8)
    out = run(d, T)
    check(out, want, dtype, n_in, rank)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(1)).cuda()
    for k in ("ids", "x", "base"):
        d[k] = d[k][perm].contiguous()
    assert torch.equal(run(d, T), out[perm])


@pytest.mark.parametrize("T,n,rank", [(257, 48, 72), (512, 5, 16), (700, 300, 40), (1000, 1000, 8), (1023, 1023, 24),
                                      (1024, 1022, 16), (1024, 1024, 16), (1025, 48, 16)])
@pytest.mark.parametrize("kind", ["mixed", "own", "two"])
def test_batches_in_any_order(T, n, rank, kind):
    """Hundreds of new tokens, their adapters in no order: taken by adapter up to 1,024 rows and 1,023
    adapters, in tiles of neighbours beyond, with the same results."""
    rng = np.random.default_rng(T + n)
    ids = {"mixed": rng.integers(-1, n, T), "own": rng.permutation(T) % n,
           "two": np.where(rng.random(T) < 0.5, 0, n - 1)}[kind]
    print("adapters in any order", T, n, rank, kind, flush=True)
    d, want = make(T, n, rank, 264, 1096, "f32", "bf16", ids, seed=T)
    out = run(d, T)
    check(out, want, "f32", 264, rank)
    order = torch.from_numpy(np.argsort(ids, kind="stable")).cuda()
    for k in ("ids", "x", "base"):
        d[k] = d[k][order].contiguous()
    assert torch.equal(run(d, T), out[order])


def test_strided_and_interleaved_rows():
    """x, base and out as column slices of one buffer; columns between them stay."""
    T, n, rank, n_in, n_out = 40, 3, 16, 72, 88
    ids = ids_of("mixed", T, n)
    d, want = make(T, n, rank, n_in, n_out, "f32", "bf16", ids, seed=8)
    buf = torch.full((T, 72 + 88 + 88 + 8), 5.0, device="cuda")
    buf[:, :72] = d["x"]
    buf[:, 72:160] = d["base"]
    d["x"], d["base"] = buf[:, :72], buf[:, 72:160]
    out = run(d, T, out=buf[:, 160:248])
    check(out, want, "f32", n_in, rank)
    assert (buf[:, 248:] == 5.0).all()


def test_hostile_ranks_are_clamped():
    T, n, rank = 20, 3, 16
    ids = np.arange(T) % n
    d, _ = make(T, n, rank, 64, 64, "f32", "f16", ids, seed=9)
    d["ranks"] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 17], dtype=torch.int32, device="cuda")
    out = run(d, T)
    d["ranks"] = torch.tensor([0, 16, 16], dtype=torch.int32, device="cuda")
    assert torch.equal(run(d, T), out)
    assert torch.equal(out[::3], d["base"][::3])


def test_infinities_and_nan_stay_in_their_row():
    """A row of NaN or infinities, and an adapter of NaN, reach the rows that use them and no others."""
    T, n = 64, 4
    ids = np.repeat(np.arange(4), 16)
    for dtype, wdtype in TYPES:
        d, want = make(T, n, 16, 128, 136, dtype, wdtype, ids, seed=11)
        d["ranks"].fill_(16)
        clean = run(d, T)
        d["x"][5, 3] = float("nan")
        d["x"][20, 0] = float("inf")
        d["a"][3].fill_(float("nan"))
        got = run(d, T)
        touched = torch.zeros(T, dtype=torch.bool, device="cuda")
        touched[5] = touched[20] = True
        touched[48:] = True
        assert torch.equal(got[~touched], clean[~touched])
        assert got[5].isnan().all() and got[48:].isnan().all() and not got[20].isfinite().any()


def test_rank_values_beyond_an_adapters_own_are_not_read():
    """Rows of a and columns of b past ranks[i] may hold anything."""
    T = 40
    ids = np.zeros(T, np.int64)
    for dtype, wdtype in TYPES:
        d, _ = make(T, 1, 24, 64, 72, dtype, wdtype, ids, seed=12)
        d["ranks"] = torch.tensor([5], dtype=torch.int32, device="cuda")
        d["a"][:, 5:] = 0
        d["b"][:, :, 5:] = 0
        want = run(d, T)
        d["a"][:, 5:] = float("nan")
        d["b"][:, :, 5:] = float("nan")
        assert torch.equal(run(d, T), want)


def test_far_apart_rows_pass_32_bit_offsets():
    T, ld = 3, 1 << 29                          # bf16: 2^30 bytes a row
    ids = np.array([0, 1, 0])
    d, want = make(T, 2, 8, 64, 64, "bf16", "bf16", ids, seed=13)
    d["ranks"].fill_(8)
    dense = run(d, T)
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    buf[:, :64], buf[:, 64:128] = d["x"], d["base"]
    d["x"], d["base"] = buf[:, :64], buf[:, 64:128]
    assert torch.equal(run(d, T, out=buf[:, 128:192]), dense)
