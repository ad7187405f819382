"""The steps together, as a layer runs them: logits -> route (with the balance
loss) -> device plan -> expert products -> combine -> adapters, and back:
output gradient -> combine's gradient -> router's gradient.  Eager against the
oracle and the plain forms, and captured into a HIP graph."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_scatter_amd as moe
from oracle import oracle
from quantized_moe_expert_scatter_amd import _lib
from quantized_moe_expert_scatter_amd import workloads as wl
from quantized_moe_expert_scatter_amd.layer import DeviceLayer
from tests import layer_ref as ref
from tests.gpu_common import GUARD, check_exact, w_tuple

pytestmark = pytest.mark.gpu


def make_adapters(n, rank, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn(n, rank, hidden, generator=g) / hidden ** 0.5).bfloat16()
    b = torch.randn(n, hidden, rank, generator=g).bfloat16()
    scale = torch.rand(n, generator=g) + 0.5
    return a, b, scale, moe.AdapterSet(a.cuda(), b.cuda(), scale.cuda())


@pytest.mark.parametrize("T,E,K,hidden,n_ff,renorm", [(64, 8, 2, 256, 128, True), (1, 16, 4, 128, 64, True),
                                                      (133, 60, 6, 320, 64, False)])
def test_layer_forward_and_backward(T, E, K, hidden, n_ff, renorm):
    print("layer", T, E, K, hidden, n_ff, renorm, flush=True)
    cfg = wl.small_config("chain", T, hidden, n_ff, E, K, seed=T)
    L = wl.make_layer(cfg)
    rng = np.random.default_rng(T)
    logits = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    logits[:, E - 1] = -np.inf                  # an expert out of service
    off = np.array([0, 0, max(T // 3, 1), max(T - 2, 1)], np.int32)
    a, b, scale, adapters = make_adapters(3, 8, hidden, seed=7)
    a_ids = rng.integers(-1, 3, T)
    D = DeviceLayer(L.x, None, L.w_gu, L.w_down, chunk_rows=64, guard=GUARD, logits=logits, topk=K, renorm=renorm,
                    seq_off=off, balance_coef=0.1, adapters=adapters, adapter_ids=a_ids)
    D.forward()
    dout = torch.from_numpy(rng.standard_normal((T, hidden)).astype(np.float32)).cuda()
    dloss = torch.tensor([0.5], device="cuda")
    D.backward(dout, dloss=dloss)
    torch.cuda.synchronize()

    l = logits.astype(np.float64)
    ids, w = ref.route(l, K, renorm)
    assert np.array_equal(D.ids_dev.cpu().numpy(), ids)
    counts, _, loss = ref.balance(l, ids, off, 0.1)
    assert np.array_equal(D.counts.cpu().numpy(), counts)
    assert abs(float(D.loss) - loss) <= loss * 64 * ref.U
    # the expert rows bit for bit, the combine from the library's own weights
    orc = oracle.layer(L.x, np.ascontiguousarray(ids, np.int32), E, n_ff, w_tuple(L.w_gu), w_tuple(L.w_down))
    dm = orc.dm.astype(np.float32)
    check_exact(D.dm_host(), dm, "expert rows")
    route_w = D.route_w.cpu().numpy()
    assert np.all(np.abs(route_w - w) <= w * 64 * ref.U + 2.0 ** -148)
    base = oracle.combine(dm, route_w)
    want, _, size = ref.adapters(L.x.astype(np.float64), base.astype(np.float64), a_ids, a.double().numpy(),
                                 b.double().numpy(), scale.double().numpy(), np.full(3, 8))
    assert np.all(np.abs(D.out_host() - want) <= size * (hidden + 16) * ref.U + np.abs(want) * 2 * ref.U)
    # back
    do = dout.double().cpu().numpy()
    terms = dm.astype(np.float64).reshape(T, K, hidden) * do[:, None, :]
    dw, dw_size = terms.sum(axis=2), np.abs(terms).sum(axis=2)
    assert np.all(np.abs(D.dw.cpu().numpy() - dw) <= dw_size * (hidden + 8) * ref.U)
    d, mag = ref.route_backward(l, ids, D.dw.double().cpu().numpy(), renorm, 1.0, off, 0.1, counts, 0.5)
    assert np.all(np.abs(D.dlogits.cpu().numpy() - d) <= mag * 128 * ref.U + 1e-38)

    # the whole gradient against differences of the layer in 64 bits (dm held: the experts are frozen)
    def value(x):
        p = ref.softmax(x)
        ww = np.take_along_axis(p, ids, 1)
        ww = ww / ww.sum(axis=1, keepdims=True) if renorm else ww
        out = (ww[:, :, None] * dm.astype(np.float64).reshape(T, K, hidden)).sum(axis=1)
        return (out * do).sum() + 0.5 * ref.balance_only(x, ids, off, 0.1, counts)

    got = D.dlogits.cpu().numpy()
    scale_of = np.abs(got).max() + 1.0
    for t, e in zip(rng.integers(0, T, 12), rng.integers(0, E - 1, 12)):
        up, dn = l.copy(), l.copy()
        up[t, e] += 1e-4
        dn[t, e] -= 1e-4
        diff = (value(up) - value(dn)) / 2e-4
        # h^2/6 of a third derivative of the gradient's size, cancellation 1e-16 * |value| / h, fp32 dw
        assert abs(diff - got[t, e]) <= 1e-5 * scale_of + 1e-11 * abs(value(l))
    D.close()


def test_captured_and_replayed():
    """Everything but the plan's host part in one graph (the plan in the library's own workspace):
    replays over changed inputs, eager work between them, every replay against the eager result."""
    cfg = wl.small_config("graph", 96, 256, 128, 16, 4, seed=3)
    L = wl.make_layer(cfg)
    rng = np.random.default_rng(0)
    T, E, K, H = cfg.tokens, cfg.n_expert, cfg.topk, cfg.hidden
    _, _, _, adapters = make_adapters(4, 16, H, seed=8)
    off = np.array([0, 30, 90], np.int32)

    def layer(logits, x, a_ids):
        return DeviceLayer(x, None, L.w_gu, L.w_down, chunk_rows=64, guard=GUARD, logits=logits, topk=K,
                           seq_off=off, balance_coef=0.1, adapters=adapters, adapter_ids=a_ids)

    def step(D, dout):
        moe.moe_route_balance(D.logits, D.seq_off, 0.1, D.ids_dev, D.route_w, D.counts, D.probs, D.loss,
                              D.balance_ws)
        D.plan = _lib.moe_prefill_plan_device_noalloc(D.ids_dev, T, K, E, 64, D.w_gu, D.w_dn)
        D.run_fused()
        D.combine()
        D.apply_adapters()
        D.backward(dout)

    def inputs(seed):
        r = np.random.default_rng(seed)
        return ((2 * r.standard_normal((T, E))).astype(np.float32), r.standard_normal((T, H)).astype(np.float32),
                r.integers(-1, 4, T).astype(np.int32), r.standard_normal((T, H)).astype(np.float32))

    lg, x, ai, do = inputs(100)
    G = layer(lg, x, ai)
    dout = torch.from_numpy(do).cuda()
    step(G, dout)                               # warm up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(G, dout)
    names = ("ids_dev", "route_w", "counts", "probs", "loss", "out", "dw", "dlogits")
    for seed in range(4):
        lg, x, ai, do = inputs(seed)
        A = layer(lg, x, ai)
        A.forward()
        A.backward(torch.from_numpy(do).cuda())
        torch.cuda.synchronize()
        want = {n: getattr(A, n).clone() for n in names}
        A.close()
        G.logits.copy_(torch.from_numpy(lg))
        G.x.copy_(torch.from_numpy(x))
        G.adapter_ids.copy_(torch.from_numpy(ai))
        dout.copy_(torch.from_numpy(do))
        for n in names:
            getattr(G, n).fill_(0)
        print("replay", seed, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(G, n).view(torch.int32), want[n].view(torch.int32)), n
    assert G.check_guards() == []


def test_empty_layer_and_one_without_logits():
    """No tokens: every step runs, the statistics are zeros.  Without logits there is nothing to go back to."""
    hidden, n_ff, E, K = 128, 64, 8, 2
    L = wl.make_layer(wl.small_config("empty", 4, hidden, n_ff, E, K, seed=1))
    _, _, _, adapters = make_adapters(2, 8, hidden, seed=8)
    D = DeviceLayer(L.x[:0], None, L.w_gu, L.w_down, chunk_rows=64, guard=GUARD, logits=np.zeros((0, E), np.float32),
                    topk=K, seq_off=np.zeros(3, np.int32), balance_coef=0.1, adapters=adapters,
                    adapter_ids=np.zeros(0, np.int32))
    D.forward()
    assert D.backward(torch.zeros(0, hidden, device="cuda")).shape == (0, E)
    torch.cuda.synchronize()
    assert not D.counts.any() and not D.probs.any() and float(D.loss) == 0.0
    D.close()
    D = DeviceLayer(L.x, L.ids, L.w_gu, L.w_down, chunk_rows=64)
    with pytest.raises(ValueError):
        D.backward(torch.zeros(4, hidden, device="cuda"))
    D.close()


@pytest.mark.parametrize("T,rank,dtype", [(300, 24, torch.float32), (300, 72, torch.bfloat16), (8200, 48, torch.float32)])
def test_long_batches_captured(T, rank, dtype):
    """The adapters' two-launch forms and the combine's gradient with the rows', replayed over changed inputs."""
    H = 256
    g = torch.Generator().manual_seed(T)
    a, b = torch.randn(5, rank, H, generator=g).bfloat16().cuda(), torch.randn(5, H, rank, generator=g).bfloat16().cuda()
    s = moe.AdapterSet(a, b, torch.rand(5, generator=g).cuda())
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    x, base, out = (torch.empty(T, H, dtype=dtype, device="cuda") for _ in range(3))
    ws = torch.empty(moe.moe_adapters_bytes(s, T), dtype=torch.uint8, device="cuda")
    dm, w, dout = torch.empty(T * 3, H, device="cuda"), torch.empty(T, 3, device="cuda"), torch.empty(T, H, device="cuda")
    dw, ddm = torch.empty(T, 3, device="cuda"), torch.empty(T * 3, H, device="cuda")

    def step(o, d, dd):
        moe.moe_adapters(s, ids, x, base, o, ws)
        moe.moe_combine_backward(dm, w, dout, d, dd)

    def fill(seed):
        h = torch.Generator().manual_seed(seed)
        ids.copy_(torch.randint(-1, 5, (T // 7 + 1,), generator=h, dtype=torch.int32).repeat_interleave(7)[:T])
        for t in (x, base, dm, w, dout):
            t.copy_(torch.randn(t.shape, generator=h))

    fill(0)
    step(out, dw, ddm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, dw, ddm)
    for seed in (1, 2, 3):
        fill(seed)
        eager = [torch.empty_like(t) for t in (out, dw, ddm)]
        step(*eager)
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        for t in (out, dw, ddm):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((out, dw, ddm), eager):
            assert torch.equal(got, want)


def test_two_at_once():
    """Two calls of each kind on two streams, with workspaces of their own, over the same inputs and
    matrices: each gives what it gives alone."""
    T, E, K, H = 1000, 64, 6, 256
    _, _, _, adapters = make_adapters(4, 16, H, seed=9)
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, H, generator=g).cuda()
    ids = torch.randint(-1, 4, (T,), generator=g, dtype=torch.int32).cuda()
    off = torch.tensor([0, 400, 1000], dtype=torch.int32, device="cuda")

    def buffers():
        return dict(ids=torch.empty(T, K, dtype=torch.int32, device="cuda"), w=torch.empty(T, K, device="cuda"),
                    counts=torch.empty(2, E, dtype=torch.int32, device="cuda"),
                    probs=torch.empty(2, E, device="cuda"), loss=torch.empty(1, device="cuda"),
                    ws=torch.empty(moe.moe_balance_bytes(T, E, 2), dtype=torch.uint8, device="cuda"),
                    out=torch.empty(T, H, device="cuda"),
                    aws=torch.empty(moe.moe_adapters_bytes(adapters, T), dtype=torch.uint8, device="cuda"))

    def call(o, stream=None):
        moe.moe_route_balance(logits, off, 0.2, o["ids"], o["w"], o["counts"], o["probs"], o["loss"], o["ws"],
                              stream=stream)
        moe.moe_adapters(adapters, ids, x, x, o["out"], o["aws"], stream=stream)

    alone = buffers()
    call(alone)
    pair = [buffers(), buffers()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, s in zip(pair, streams):
            call(o, s)
    torch.cuda.synchronize()
    for o in pair:
        for n in ("ids", "w", "counts", "probs", "loss", "out"):
            assert torch.equal(o[n].view(torch.int32), alone[n].view(torch.int32)), n
