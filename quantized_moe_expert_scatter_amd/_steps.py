"""ctypes binding of the C ABI in include/moe_layer.h: the steps around the
expert products (router, balance loss, gradients, per-request adapters).

Every function keeps the C name and forwards to libmoe_prefill.so.  Tensors
are the caller's, on the current HIP device; what the C call cannot see (a
tensor's type, shape, strides and device) is checked here, and a bad one
raises MoeError with the status the C call would give.  Work is enqueued on
`stream`, by default torch's current stream; a tensor made on another stream
must be ready on it, and one freed early must be kept until the work has run.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import MoeError

MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_ROUTE_RENORM = 1

# every symbol include/moe_layer.h declares
EXPORTS = ["moe_route", "moe_balance_bytes", "moe_route_balance", "moe_route_backward",
           "moe_combine_backward", "moe_adapters_bytes", "moe_adapters"]


class moe_adapter_set(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("n_adapter", ctypes.c_int), ("rank", ctypes.c_int),
                ("n_in", ctypes.c_int), ("n_out", ctypes.c_int), ("a", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ranks", ctypes.c_void_p)]


_bound = None


def lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        L = _lib.lib()
        P, I, Z, F, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
        route = [P, L64, I, I, I, I, I, F]      # logits, ld, dtype, tokens, n_expert, topk, flags, scale
        L.moe_route.argtypes = route + [P, P, P]
        L.moe_balance_bytes.argtypes = [I, I, I]
        L.moe_balance_bytes.restype = Z
        L.moe_route_balance.argtypes = route + [P, I, F, P, P, P, P, P, P, Z, P]
        L.moe_route_backward.argtypes = route + [P, P, P, I, F, P, P, P, L64, P]
        L.moe_combine_backward.argtypes = [P, P, P, I, I, I, P, P, P]
        L.moe_adapters_bytes.argtypes = [ctypes.POINTER(moe_adapter_set), I]
        L.moe_adapters_bytes.restype = Z
        L.moe_adapters.argtypes = [ctypes.POINTER(moe_adapter_set), P, I, I, P, L64, P, L64, P, L64, P, Z, P]
        for name in EXPORTS:
            if not name.endswith("_bytes"):
                getattr(L, name).restype = I
        _bound = L
    return _bound


_torch = None
_codes = {}


def _load_torch():
    """torch, imported on first use like the library."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
        _codes.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16})
    return _torch


def _current(stream, t, what: str):
    """The current device, which has to hold t, and the raw stream (torch's current one by
    default).  A call is a few microseconds, half of them this module's: hence raw handles and
    few calls per tensor."""
    c = _load_torch()._C
    device = -1 if t is None else t.get_device()
    if device < 0 or device != c._cuda_getDevice():
        raise MoeError(-1, f"{what}: {'None' if t is None else t.device} is not the current device")
    if stream is None:
        return device, c._cuda_getCurrentRawStream(device)
    return device, stream if isinstance(stream, int) else stream.cuda_stream


def _dtype(t, what: str) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        raise MoeError(-3, f"{what}: {t.dtype}")
    return code


def _dense(device: int, t, what: str, dtype, shape):
    """The address of a dense tensor of the given type, shape and device (None: no tensor)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device >= 0:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise MoeError(-3, f"{what}: {t.dtype} instead of {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise MoeError(-1, f"{what}: shape {tuple(t.shape)}, strides {t.stride()}; dense {tuple(shape)} wanted")
    raise MoeError(-1, f"{what}: on {t.device}, the current device is cuda:{device}")


def _rows(device: int, t, what: str, shape, written: bool = False):
    """The address and row stride of a matrix with dense rows (that do not overlap, if written)."""
    if t.shape != shape:
        raise MoeError(-1, f"{what}: shape {tuple(t.shape)}; {tuple(shape)} wanted")
    ld, step = t.stride()
    if (step != 1 and shape[1] > 1 and shape[0] > 0) or (written and ld < shape[1] and shape[0] > 1):
        raise MoeError(-1, f"{what}: strides {t.stride()}; dense rows wanted")
    if t.get_device() != device:
        raise MoeError(-1, f"{what}: on {t.device}, the current device is cuda:{device}")
    # the strides of no row, and a single row's, say nothing: torch may give them any value
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _count(n: int, what: str) -> int:
    """n as the C call takes it: ctypes would cut a larger one to its low 32 bits."""
    if n > 0x7fffffff:
        raise MoeError(-1, f"{what}: a size of {n}")
    return n


def _ints(*sizes: int) -> bool:
    """Whether the C call can take the sizes of a query."""
    return all(abs(n) <= 0x7fffffff for n in sizes)


def _matrix(t, what: str):
    if t is None or t.dim() != 2:
        raise MoeError(-1, f"{what}: {None if t is None else tuple(t.shape)} is not a matrix")
    rows, cols = shape = t.shape
    if rows > 0x7fffffff or cols > 0x7fffffff:
        _count(max(shape), what)
    return shape


def _sequences(seq_off) -> int:
    if seq_off is None:
        raise MoeError(-1, "seq_off: None")
    return _count(seq_off.numel() - 1, "seq_off")


def _route(device: int, logits, topk: int, renorm: bool, scale: float):
    shape = _matrix(logits, "logits")
    ptr, ld = _rows(device, logits, "logits", shape)
    T, E = shape
    return (ptr, ld, _dtype(logits, "logits"), T, E, topk, MOE_ROUTE_RENORM if renorm else 0, scale)


def moe_route(logits, ids, w, renorm: bool = True, scale: float = 1.0, stream=None):
    """logits [T, E] (fp32, bf16 or fp16, dense rows) -> ids int32 [T, topk], w fp32 [T, topk]."""
    torch = _load_torch()
    dev, raw = _current(stream, logits, "logits")
    K = _matrix(ids, "ids")[1]
    head = _route(dev, logits, K, renorm, scale)
    shape = (head[3], K)
    st = lib().moe_route(*head, _dense(dev, ids, "ids", torch.int32, shape),
                         _dense(dev, w, "w", torch.float32, shape), raw)
    if st:
        raise MoeError(st, "moe_route")


def moe_balance_bytes(tokens: int, n_expert: int, n_seq: int) -> int:
    return int(lib().moe_balance_bytes(tokens, n_expert, n_seq)) if _ints(tokens, n_expert, n_seq) else 0


def moe_route_balance(logits, seq_off, coef: float, ids, w, counts, probs, loss, workspace,
                      renorm: bool = True, scale: float = 1.0, stream=None):
    """moe_route with the balance statistics of the sequences seq_off (int32 [S+1]) bounds:
    counts int32 [S, E], probs fp32 [S, E], loss fp32 [1]."""
    torch = _load_torch()
    dev, raw = _current(stream, logits, "logits")
    K = _matrix(ids, "ids")[1]
    head = _route(dev, logits, K, renorm, scale)
    T, E, S = head[3], head[4], _sequences(seq_off)
    f32, i32 = torch.float32, torch.int32
    st = lib().moe_route_balance(
        *head, _dense(dev, seq_off, "seq_off", i32, (S + 1,)), S, coef, _dense(dev, ids, "ids", i32, (T, K)),
        _dense(dev, w, "w", f32, (T, K)), _dense(dev, counts, "counts", i32, (S, E)),
        _dense(dev, probs, "probs", f32, (S, E)), _dense(dev, loss, "loss", f32, (1,)),
        *_workspace(dev, workspace), raw)
    if st:
        raise MoeError(st, "moe_route_balance")


def _workspace(device: int, t):
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise MoeError(-1, f"workspace: strides {t.stride()}")
    if t.get_device() != device:
        raise MoeError(-1, f"workspace: on {t.device}, the current device is cuda:{device}")
    return t.data_ptr(), t.numel() * t.element_size()


def moe_route_backward(logits, ids, dw, dlogits, renorm: bool = True, scale: float = 1.0, seq_off=None,
                       coef: float = 0.0, counts=None, dloss=None, stream=None):
    """The gradient of moe_route / moe_route_balance: dw fp32 [T, topk] (or None) and the loss's
    (seq_off and counts of the forward call, dloss fp32 [1] or None for 1) -> dlogits, the
    logits' type and shape."""
    torch = _load_torch()
    dev, raw = _current(stream, logits, "logits")
    K = _matrix(ids, "ids")[1]
    head = _route(dev, logits, K, renorm, scale)
    T, E = head[3], head[4]
    S = 0 if seq_off is None else _sequences(seq_off)
    f32, i32 = torch.float32, torch.int32
    if dlogits is None:
        raise MoeError(-1, "dlogits: None")
    if dlogits.dtype != logits.dtype:
        raise MoeError(-3, f"dlogits: {dlogits.dtype} instead of {logits.dtype}")
    d_ptr, ldd = _rows(dev, dlogits, "dlogits", (T, E), True)
    st = lib().moe_route_backward(
        *head, _dense(dev, ids, "ids", i32, (T, K)), _dense(dev, dw, "dw", f32, (T, K)),
        _dense(dev, seq_off, "seq_off", i32, (S + 1,)), S, coef, _dense(dev, counts, "counts", i32, (S, E)),
        _dense(dev, dloss, "dloss", f32, (1,)), d_ptr, ldd, raw)
    if st:
        raise MoeError(st, "moe_route_backward")


def moe_combine_backward(dm, w, dout, dw, ddm=None, stream=None):
    """The gradient of moe_combine: dout fp32 [T, H] -> dw fp32 [T, topk] and ddm fp32
    [T*topk, H] (either may be None; dm is read for dw, w [T, topk] for ddm)."""
    f32 = _load_torch().float32
    dev, raw = _current(stream, dout, "dout")
    T, H = _matrix(dout, "dout")
    K = _matrix(dw if dw is not None else w, "dw or w")[1]
    rows, per = (T * K, H), (T, K)
    st = lib().moe_combine_backward(
        _dense(dev, dm, "dm", f32, rows), _dense(dev, w, "w", f32, per), _dense(dev, dout, "dout", f32, (T, H)),
        T, K, H, _dense(dev, dw, "dw", f32, per), _dense(dev, ddm, "ddm", f32, rows), raw)
    if st:
        raise MoeError(st, "moe_combine_backward")


class AdapterSet:
    """The adapters of one projection (kept alive here, read in place): a
    [n, rank, n_in] and b [n, n_out, rank], both bf16 or both fp16, scale fp32
    [n], rank int32 [n] with each adapter's own rank (None: all full)."""

    def __init__(self, a, b, scale, rank=None):
        torch = _load_torch()
        if any(t is None or t.dim() != 3 for t in (a, b)):
            raise MoeError(-1, "AdapterSet: a and b " + " ".join("None" if t is None else str(tuple(t.shape))
                                                                  for t in (a, b)))
        n, r, n_in = a.shape
        n_out = b.shape[1]
        _count(max(n, r, n_in, n_out), "AdapterSet")
        code = _dtype(a, "a")
        if code == MOE_F32:
            raise MoeError(-3, f"a: {a.dtype}")
        dev = a.get_device() if a.is_cuda else -1
        self.tensors = (a, b, scale, rank)
        self.device, self.n_in, self.n_out, self.rank = dev, n_in, n_out, r
        self.struct = moe_adapter_set(
            code, n, r, n_in, n_out, _dense(dev, a, "a", a.dtype, (n, r, n_in)),
            _dense(dev, b, "b", a.dtype, (n, n_out, r)), _dense(dev, scale, "scale", torch.float32, (n,)),
            _dense(dev, rank, "rank", torch.int32, (n,)))
        self.ref = ctypes.byref(self.struct)


def moe_adapters_bytes(adapters: AdapterSet, tokens: int) -> int:
    return int(lib().moe_adapters_bytes(adapters.ref, tokens)) if _ints(tokens) else 0


def moe_adapters(adapters: AdapterSet, ids, x, base, out, workspace, stream=None):
    """out = base + each row's adapter over x: ids int32 [T] (negative: none), x [T, n_in], base
    and out [T, n_out] of fp32 or the set's type, dense rows; out may be base."""
    torch = _load_torch()
    dev, raw = _current(stream, x, "x")
    if adapters.device != dev:
        raise MoeError(-1, f"adapters: on cuda:{adapters.device}, the current device is cuda:{dev}")
    if ids is None or base is None or out is None:
        raise MoeError(-1, "moe_adapters: ids, base and out are needed")
    T = _count(ids.numel(), "ids")
    kind = x.dtype
    if base.dtype != kind or out.dtype != kind:
        raise MoeError(-3, f"moe_adapters: x {x.dtype}, base {base.dtype}, out {out.dtype}")
    shape = (T, adapters.n_out)
    st = lib().moe_adapters(
        adapters.ref, _dense(dev, ids, "ids", torch.int32, (T,)), T, _dtype(x, "x"),
        *_rows(dev, x, "x", (T, adapters.n_in)), *_rows(dev, base, "base", shape),
        *_rows(dev, out, "out", shape, True), *_workspace(dev, workspace), raw)
    if st:
        raise MoeError(st, "moe_adapters")
