"""The C ABI of include/moe_layer.h on the host (no GPU): exported symbols,
size queries, every refusal that comes before any HIP call, and the plain
forms the GPU tests compare with (their gradients against differences)."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from quantized_moe_expert_scatter_amd import _lib, _steps
from tests import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer.h")
P = 1 << 20                                     # an aligned stand-in address
OFF = 8                                         # ... and this much off it
EINVAL, EALIGN, EFORMAT, ESIZE = -1, -2, -3, -4


def test_every_declared_symbol_is_exported():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)) - {"if", "defined"})
    assert names == sorted(_steps.EXPORTS)
    for n in names:
        assert hasattr(_steps.lib(), n), n


def test_header_compiles_as_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    src = tmp_path / "h.c"
    src.write_text('#include "moe_layer.h"\nint main(void) { moe_adapter_set s = {0}; return s.rank; }\n')
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           str(src), "-o", str(tmp_path / "h")])


def test_host_side_links_without_the_kernels(tmp_path):
    """moe_layer.cpp against stubs of its launchers: no undefined symbol, so the
    sanitizer build of the host side loads."""
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ or the ROCm headers are not available")
    r = subprocess.run(["g++", "-O0", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include",
                        os.path.join(ROOT, "quantized_moe_expert_scatter_amd", "csrc", "moe_layer.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "host_stubs_layer.cpp"),
                        "-o", str(tmp_path / "l.so"), "-Wl,--no-undefined"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_sizes():
    assert _steps.moe_balance_bytes(16, 8, 0) == 0
    assert _steps.moe_balance_bytes(-1, 8, 1) == 0
    assert _steps.moe_balance_bytes(16, 2049, 1) == 0
    assert _steps.moe_balance_bytes(16, 0, 1) == 0
    assert _steps.moe_balance_bytes(0, 8, 1) > 0
    # no overflow at the largest sizes
    assert 0 < _steps.moe_balance_bytes(2 ** 31 - 1, 2048, 2 ** 20) < 2 ** 35
    s = make_set()
    assert _steps.lib().moe_adapters_bytes(ctypes.byref(s), 100) >= 100 * 16 * 4
    assert _steps.lib().moe_adapters_bytes(ctypes.byref(s), -1) == 0
    assert _steps.lib().moe_adapters_bytes(ctypes.byref(make_set(rank=12)), 100) == 0
    assert _steps.lib().moe_adapters_bytes(None, 100) == 0


ROUTE = dict(logits=P, ld=8, dtype=0, tokens=4, n_expert=8, topk=2, flags=1, scale=1.0)


def route(**kw):
    a = {**ROUTE, "ids": P, "w": P, **kw}
    return _steps.lib().moe_route(*[a[k] for k in ROUTE], a["ids"], a["w"], None)


ROUTE_REFUSALS = [
    (dict(logits=None), EINVAL), (dict(logits=P + OFF), EALIGN), (dict(ld=7), EINVAL),
    (dict(ld=1 << 41), EINVAL), (dict(dtype=3), EFORMAT), (dict(dtype=-1), EFORMAT),
    (dict(tokens=-1), EINVAL), (dict(n_expert=0, ld=8), EINVAL), (dict(n_expert=2049, ld=4096), EINVAL),
    (dict(topk=0), EINVAL), (dict(topk=9), EINVAL), (dict(topk=65, n_expert=128, ld=128), EINVAL),
    (dict(flags=2), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL)]


@pytest.mark.parametrize("kw,want", ROUTE_REFUSALS + [
    (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(ids=P + OFF), EALIGN), (dict(w=P + 4), EALIGN)])
def test_route_refusals(kw, want):
    assert route(**kw) == want


def test_nothing_to_do():
    """No tokens: accepted without buffers, nothing is launched."""
    assert route(tokens=0, logits=None, ids=None, w=None) == 0
    assert backward(tokens=0, logits=None, ids=None, dlogits=None) == 0
    assert combine(tokens=0, dm=None, w=None, dout=None, dw=None, ddm=None) == 0
    assert adapters(tokens=0, ids=None, x=None, base=None, out=None, ws=None, nb=0) == 0


def balance(**kw):
    a = {**ROUTE, "seq_off": P, "n_seq": 2, "coef": 0.01, "ids": P, "w": P, "counts": P, "probs": P,
         "loss": P, "ws": P, "nb": _steps.moe_balance_bytes(4, 8, 2), **kw}
    return _steps.lib().moe_route_balance(*[a[k] for k in list(ROUTE) + [
        "seq_off", "n_seq", "coef", "ids", "w", "counts", "probs", "loss", "ws", "nb"]], None)


@pytest.mark.parametrize("kw,want", ROUTE_REFUSALS + [
    (dict(n_seq=0), EINVAL), (dict(n_seq=-1), EINVAL), (dict(coef=float("nan")), EINVAL),
    (dict(nb=_steps.moe_balance_bytes(4, 8, 2) - 1), ESIZE), (dict(nb=0), ESIZE)]
    + [({k: None}, EINVAL) for k in ("seq_off", "ids", "w", "counts", "probs", "loss", "ws")]
    + [({k: P + OFF}, EALIGN) for k in ("seq_off", "ids", "w", "counts", "probs", "loss", "ws")])
def test_balance_refusals(kw, want):
    assert balance(**kw) == want


def backward(**kw):
    a = {**ROUTE, "ids": P, "dw": P, "seq_off": P, "n_seq": 2, "coef": 0.01, "counts": P, "dloss": P,
         "dlogits": 2 * P, "ldd": 8, **kw}
    return _steps.lib().moe_route_backward(*[a[k] for k in list(ROUTE) + [
        "ids", "dw", "seq_off", "n_seq", "coef", "counts", "dloss", "dlogits", "ldd"]], None)


@pytest.mark.parametrize("kw,want", ROUTE_REFUSALS + [
    (dict(ids=None), EINVAL), (dict(dlogits=None), EINVAL), (dict(ldd=7), EINVAL), (dict(n_seq=0), EINVAL),
    (dict(seq_off=None), EINVAL), (dict(counts=None), EINVAL), (dict(coef=float("inf")), EINVAL),
    (dict(dlogits=P, ldd=16), EINVAL)]
    + [({k: 2 * P + OFF}, EALIGN) for k in ("ids", "dw", "seq_off", "counts", "dloss", "dlogits")])
def test_backward_refusals(kw, want):
    assert backward(**kw) == want


def combine(**kw):
    a = dict(dm=P, w=P, dout=P, tokens=4, topk=2, hidden=64, dw=P, ddm=P)
    a.update(kw)
    return _steps.lib().moe_combine_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), EINVAL), (dict(topk=0), EINVAL), (dict(hidden=0), EINVAL), (dict(hidden=66), EFORMAT),
    (dict(tokens=1 << 30, topk=2), EINVAL), (dict(tokens=1 << 26, topk=8), EINVAL),
    (dict(tokens=1 << 25, topk=9), EINVAL), (dict(dout=None), EINVAL), (dict(dw=None, ddm=None), EINVAL),
    (dict(dm=None), EINVAL), (dict(w=None), EINVAL)]
    + [({k: P + OFF}, EALIGN) for k in ("dm", "w", "dout", "dw", "ddm")])
def test_combine_backward_refusals(kw, want):
    assert combine(**kw) == want


def make_set(**kw):
    a = dict(dtype=1, n_adapter=3, rank=16, n_in=64, n_out=128, a=P, b=P, scale=P, ranks=P)
    a.update(kw)
    return _steps.moe_adapter_set(*a.values())


def adapters(set_kw=None, **kw):
    s = None if set_kw is False else make_set(**(set_kw or {}))
    a = dict(ids=P, tokens=4, dtype=0, x=P, ldx=64, base=2 * P, ldb=128, out=3 * P, ldo=128, ws=4 * P, nb=1 << 20)
    a.update(kw)
    return _steps.lib().moe_adapters(None if s is None else ctypes.byref(s), *a.values(), None)


@pytest.mark.parametrize("set_kw,kw,want", [
    (False, {}, EINVAL), (dict(dtype=0), {}, EFORMAT), (dict(dtype=3), {}, EFORMAT), (dict(rank=12), {}, EFORMAT),
    (dict(n_in=60), dict(ldx=64), EFORMAT), (dict(n_out=100), {}, EFORMAT), (dict(rank=0), {}, EINVAL),
    (dict(rank=-8), {}, EINVAL), (dict(rank=264), {}, EINVAL), (dict(n_adapter=0), {}, EINVAL), (dict(n_in=0), {}, EINVAL),
    (dict(n_out=1 << 25), dict(ldb=1 << 25, ldo=1 << 25), EINVAL),
    (dict(a=None), {}, EINVAL), (dict(b=None), {}, EINVAL), (dict(scale=None), {}, EINVAL),
    (dict(a=P + OFF), {}, EALIGN), (dict(b=P + OFF), {}, EALIGN), (dict(scale=P + 4), {}, EALIGN),
    (dict(ranks=P + 4), {}, EALIGN),
    ({}, dict(dtype=2), EFORMAT), ({}, dict(dtype=5), EFORMAT), ({}, dict(tokens=-1), EINVAL),
    ({}, dict(ldx=56), EINVAL), ({}, dict(ldb=120), EINVAL), ({}, dict(ldo=120), EINVAL),
    ({}, dict(ldx=68), EALIGN), ({}, dict(ldb=132), EALIGN), ({}, dict(ldo=132), EALIGN),
    ({}, dict(tokens=(1 << 24) + 1), EINVAL), ({}, dict(tokens=1 << 24, nb=16), ESIZE),
    ({}, dict(ids=None), EINVAL), ({}, dict(x=None), EINVAL), ({}, dict(base=None), EINVAL),
    ({}, dict(out=None), EINVAL), ({}, dict(ws=None), EINVAL), ({}, dict(out=P, ldo=128), EINVAL),
    ({}, dict(out=2 * P, ldo=256), EINVAL), ({}, dict(nb=4 * 16 * 4 - 1), ESIZE)]
    + [({}, {k: 5 * P + OFF}, EALIGN) for k in ("ids", "x", "base", "out", "ws")])
def test_adapter_refusals(set_kw, kw, want):
    assert adapters(set_kw, **kw) == want


def test_binding_refuses_what_the_c_call_cannot_see():
    """Tensors in host memory and adapter matrices of the wrong shape or type, before the library is called."""
    l = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)

    def status(f, *a, **k):
        with pytest.raises(_lib.MoeError) as e:
            f(*a, **k)
        return e.value.status

    assert status(_steps.moe_route, l, ids, w, stream=0) == EINVAL
    assert status(_steps.moe_route, None, ids, w, stream=0) == EINVAL
    a, b, s = torch.zeros(2, 16, 64).bfloat16(), torch.zeros(2, 128, 16).bfloat16(), torch.zeros(2)
    assert status(_steps.AdapterSet, a[0], b, s) == EINVAL
    assert status(_steps.AdapterSet, a.float(), b, s) == EFORMAT
    assert status(_steps.AdapterSet, a, b, s) == EINVAL
    assert status(_steps.AdapterSet, None, b, s) == EINVAL
    assert status(_steps.AdapterSet, a, None, s) == EINVAL
    # row counts past an int, which ctypes would cut to 1
    assert status(_steps._matrix, torch.empty((1 << 32) + 1, 1, device="meta"), "logits") == EINVAL
    assert status(_steps._sequences, torch.empty((1 << 32) + 2, device="meta")) == EINVAL
    assert status(_steps._sequences, None) == EINVAL


# ------------------------------------------------ the plain forms themselves
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_gradient_matches_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, K = 7, 9, 3
    l = rng.standard_normal((T, E))
    l[2, :7] = -np.inf                          # fewer open experts than topk
    l[5] = -np.inf
    off = [0, 0, 3, 6]                          # an empty sequence, a padding row
    ids = ref.choice(l, K)
    counts, _, _ = ref.balance(l, ids, off, 1.0)
    dw = rng.standard_normal((T, K))

    def value(x):
        p = ref.softmax(x)
        w = np.take_along_axis(p, ids, 1)
        if renorm:
            s = w.sum(axis=1, keepdims=True)
            w = np.where(s == 0, 0.0, w / np.where(s == 0, 1.0, s))
        return (1.3 * w * dw).sum() + 0.7 * ref.balance_only(x, ids, off, 0.5, counts)

    d, _ = ref.route_backward(l, ids, dw, renorm, 1.3, off, 0.5, counts, 0.7)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert d[t, e] == 0.0
                continue
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            # the difference's own error: h^2/6 times a third derivative of order 1, and 1e-16/h
            assert abs((value(up) - value(dn)) / (2 * h) - d[t, e]) < 1e-9


def test_plain_loss_is_coef_when_balanced():
    l = np.zeros((4, 4))
    l[np.arange(4), np.arange(4)] = 1.0         # each token its own expert, p symmetric
    ids = ref.choice(l, 1)
    _, _, loss = ref.balance(l, ids, [0, 4], 0.25)
    assert abs(loss - 0.25) < 1e-15
