"""Binding of include/mqconv_block.h: group norm with an activation, dropout
and the replay cache. Same names as the C entry points; only arguments are
marshalled here. Descriptors (mq_norm, mq_drop, MxCache) may be kept and used
again by the program that made them."""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional

import microscaling_quantized_convolution_mxq_amd as _mq

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
NORM_FWD, NORM_BWD = 0, 1
CACHE_COUNT_MAX = 4096


def _int32(what: str, *values: int):
    """Values of the library's 32-bit arguments: ctypes would pass the low bits of larger ones on."""
    for v in values:
        if not -2**31 <= v < 2**31:
            raise _mq.MqConvError(_mq.MQ_ERR_SHAPE, what, f"{v} does not fit 32 bits")
    return values


class mq_drop(ctypes.Structure):
    """Dropout with probability p. `step`: None, or a one-element int64 GPU
    tensor added to the seed when the kernel runs (a captured graph then draws
    a new mask at each replay)."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("step", ctypes.c_void_p)]

    def __init__(self, p: float, seed: int, step=None):
        super().__init__(p, int(seed) & (2**64 - 1), _mq._buf(step, 8, "int64", "step"))
        self._step = step  # its memory is read by every call


class mq_norm(ctypes.Structure):
    """Group norm of an [H][W][N][C] tensor with an activation."""
    _fields_ = [("h", ctypes.c_int32), ("w", ctypes.c_int32), ("n", ctypes.c_int32), ("c", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float)]

    def __init__(self, h: int, w: int, n: int, c: int, groups: int, act: int = ACT_NONE, eps: float = 1e-5):
        super().__init__(*_int32("mq_norm", h, w, n, c, groups, act), eps)


class mq_cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("fmt", ctypes.c_int32),
                ("slots", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32), ("c", ctypes.c_int32)]


EXPORTED_BLOCK = (
    "mqconv_dropout", "mqconv_dropout_mx", "mqconv_group_norm_workspace_bytes", "mqconv_group_norm",
    "mqconv_group_norm_mx", "mqconv_group_norm_backward", "mqconv_group_norm_backward_mx", "mqconv_cache_codes_bytes",
    "mqconv_cache_scales_bytes", "mqconv_cache_write", "mqconv_cache_read", "mqconv_cache_read_mx")

_fns = None


def _lib():
    """The loaded library with the signatures of this header (raises if it is not built)."""
    global _fns
    L = _mq.lib()
    if _fns is not L:
        P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        GN, DR, MX, CA = ctypes.POINTER(mq_norm), ctypes.POINTER(mq_drop), _mq.mq_mx, mq_cache
        sig = {
            "mqconv_dropout": (I, [P, P, I, I, I, I, DR, P, P]),
            "mqconv_dropout_mx": (I, [P, DR, MX, P]),
            "mqconv_group_norm_workspace_bytes": (S, [GN, I]),
            "mqconv_group_norm": (I, [GN, P, P, P, DR, P, P, P, P, S, P]),
            "mqconv_group_norm_mx": (I, [GN, P, P, P, DR, MX, P, P, P, S, P]),
            "mqconv_group_norm_backward": (I, [GN, P, P, P, P, P, P, DR, P, P, P, P, S, P]),
            "mqconv_group_norm_backward_mx": (I, [GN, P, P, P, P, P, P, DR, MX, P, P, P, S, P]),
            "mqconv_cache_codes_bytes": (S, [I, I, I, I, I]),
            "mqconv_cache_scales_bytes": (S, [I, I, I, I]),
            "mqconv_cache_write": (I, [CA, P, I, I, I, P, P]),
            "mqconv_cache_read": (I, [CA, P, I, P, I, I, P]),
            "mqconv_cache_read_mx": (I, [CA, P, MX, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _fns = L
    return L


def _floats(t, count: int, what: str) -> Optional[int]:
    return _mq._buf(t, 4 * count, "float32", what)


def _drop(drop: Optional[mq_drop]):
    return None if drop is None else ctypes.byref(drop)


# ---- dropout ------------------------------------------------------------------------------------
def _dims(t, what: str):
    if not hasattr(t, "shape") or len(t.shape) != 4:
        raise _mq.MqConvError(_mq.MQ_ERR_SHAPE, what, "a tensor of four dimensions [H][W][N][C] gives the sizes")
    return _int32(what, *t.shape)


def mqconv_dropout(x, drop: mq_drop, y, residual=None, stream=None) -> None:
    """y = drop(x) + residual; x is an [H][W][N][C] tensor."""
    h, w, n, c = _dims(x, "x")
    count = h * w * n * c
    _mq._check(_lib().mqconv_dropout(_floats(x, count, "x"), None if residual is None else _floats(residual, count, "residual"),
                                     h, w, n, c, _drop(drop), _floats(y, count, "y"), _mq._stream(stream)),
               "mqconv_dropout")


def mqconv_dropout_mx(x, drop: mq_drop, dst, stream=None) -> None:
    """drop(x) quantized into dst (an ACT or GRAD MxTensor)."""
    _mq._check(_lib().mqconv_dropout_mx(_floats(x, _mq._prod(_int32("dst", *dst.dims)), "x"), _drop(drop), dst.c_struct("dst"),
                                        _mq._stream(stream)), "mqconv_dropout_mx")


# ---- group norm ---------------------------------------------------------------------------------
def mqconv_group_norm_workspace_bytes(norm: mq_norm, op: int) -> int:
    return _lib().mqconv_group_norm_workspace_bytes(ctypes.byref(norm), op)


def _norm_inputs(g: mq_norm, x, gamma, beta):
    c = g.c
    return (_floats(x, g.h * g.w * g.n * c, "x"), None if gamma is None else _floats(gamma, c, "gamma"),
            None if beta is None else _floats(beta, c, "beta"))


def mqconv_group_norm(norm: mq_norm, x, gamma, beta, y, mean=None, rstd=None, ws=None, drop: Optional[mq_drop] = None,
                      stream=None) -> None:
    g = norm
    p, nb = _mq._ws(ws)
    ng = g.n * g.groups
    _mq._check(_lib().mqconv_group_norm(
        ctypes.byref(g), *_norm_inputs(g, x, gamma, beta), _drop(drop), _floats(y, g.h * g.w * g.n * g.c, "y"),
        None if mean is None else _floats(mean, ng, "mean"), None if rstd is None else _floats(rstd, ng, "rstd"), p, nb,
        _mq._stream(stream)), "mqconv_group_norm")


def mqconv_group_norm_mx(norm: mq_norm, x, gamma, beta, yq, mean=None, rstd=None, ws=None,
                         drop: Optional[mq_drop] = None, stream=None) -> None:
    """mqconv_group_norm with y quantized into the ACT MxTensor yq."""
    g = norm
    p, nb = _mq._ws(ws)
    ng = g.n * g.groups
    _mq._check(_lib().mqconv_group_norm_mx(
        ctypes.byref(g), *_norm_inputs(g, x, gamma, beta), _drop(drop), yq.c_struct("yq"),
        None if mean is None else _floats(mean, ng, "mean"), None if rstd is None else _floats(rstd, ng, "rstd"), p, nb,
        _mq._stream(stream)), "mqconv_group_norm_mx")


def mqconv_group_norm_backward(norm: mq_norm, dy, x, gamma, beta, mean, rstd, dx, dgamma=None, dbeta=None, ws=None,
                               drop: Optional[mq_drop] = None, stream=None) -> None:
    g = norm
    p, nb = _mq._ws(ws)
    e, ng = g.h * g.w * g.n * g.c, g.n * g.groups
    _mq._check(_lib().mqconv_group_norm_backward(
        ctypes.byref(g), _floats(dy, e, "dy"), *_norm_inputs(g, x, gamma, beta), _floats(mean, ng, "mean"),
        _floats(rstd, ng, "rstd"), _drop(drop), _floats(dx, e, "dx"),
        None if dgamma is None else _floats(dgamma, g.c, "dgamma"),
        None if dbeta is None else _floats(dbeta, g.c, "dbeta"), p, nb, _mq._stream(stream)),
        "mqconv_group_norm_backward")


def mqconv_group_norm_backward_mx(norm: mq_norm, dy, x, gamma, beta, mean, rstd, dxq, dgamma=None, dbeta=None, ws=None,
                                  drop: Optional[mq_drop] = None, stream=None) -> None:
    """mqconv_group_norm_backward with dx quantized into the GRAD MxTensor dxq."""
    g = norm
    p, nb = _mq._ws(ws)
    e, ng = g.h * g.w * g.n * g.c, g.n * g.groups
    _mq._check(_lib().mqconv_group_norm_backward_mx(
        ctypes.byref(g), _floats(dy, e, "dy"), *_norm_inputs(g, x, gamma, beta), _floats(mean, ng, "mean"),
        _floats(rstd, ng, "rstd"), _drop(drop), dxq.c_struct("dxq"),
        None if dgamma is None else _floats(dgamma, g.c, "dgamma"),
        None if dbeta is None else _floats(dbeta, g.c, "dbeta"), p, nb, _mq._stream(stream)),
        "mqconv_group_norm_backward_mx")


# ---- replay cache -------------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def mqconv_cache_codes_bytes(fmt: int, slots: int, h: int, w: int, c: int) -> int:
    return _lib().mqconv_cache_codes_bytes(fmt, slots, h, w, c)


@functools.lru_cache(maxsize=1024)
def mqconv_cache_scales_bytes(slots: int, h: int, w: int, c: int) -> int:
    return _lib().mqconv_cache_scales_bytes(slots, h, w, c)


@dataclasses.dataclass
class MxCache:
    """A replay cache on the device (layout in include/mqconv_block.h)."""
    codes: object  # torch.uint8 tensor
    scales: object  # torch.uint8 tensor
    fmt: int
    slots: int
    h: int
    w: int
    c: int

    @staticmethod
    def empty(fmt: int, slots: int, h: int, w: int, c: int, device="cuda") -> "MxCache":
        import torch
        _int32("MxCache.empty", slots, h, w, c)
        nc, ns = mqconv_cache_codes_bytes(fmt, slots, h, w, c), mqconv_cache_scales_bytes(slots, h, w, c)
        if nc == 0 or ns == 0:
            raise _mq.MqConvError(_mq.MQ_ERR_SHAPE, "MxCache.empty")
        return MxCache(torch.empty(nc, dtype=torch.uint8, device=device),
                       torch.empty(ns, dtype=torch.uint8, device=device), fmt, slots, h, w, c)

    def c_struct(self) -> mq_cache:
        """The C view; tensor buffers are checked against the sizes the layout needs."""
        t = _int32("cache", self.slots, self.h, self.w, self.c)
        return mq_cache(_mq._buf(self.codes, mqconv_cache_codes_bytes(self.fmt, *t), "uint8", "cache.codes"),
                        _mq._buf(self.scales, mqconv_cache_scales_bytes(*t), "uint8", "cache.scales"), self.fmt, *t)


def _slots(slot, count: int) -> Optional[int]:
    return _mq._buf(slot, 4 * count, "int32", "slot")


def _count(slot) -> int:
    if not hasattr(slot, "numel"):
        raise _mq.MqConvError(_mq.MQ_ERR_SHAPE, "slot", "a tensor gives the number of samples")
    return _int32("slot", slot.numel())[0]


def _batch(x, c: MxCache, what: str):
    """Samples of an [H][W][N][C] tensor that goes into or comes from the cache."""
    h, w, n, ch = _dims(x, what)
    if (h, w, ch) != (c.h, c.w, c.c):
        raise _mq.MqConvError(_mq.MQ_ERR_SHAPE, what, f"sizes {tuple(x.shape)}, the cache holds {(c.h, c.w, c.c)}")
    return n, _floats(x, h * w * n * ch, what)


def mqconv_cache_write(cache: MxCache, x, slot, n0: int = 0, stream=None) -> None:
    """Stores samples n0 .. of x [H][W][N][C], one for each entry of `slot` (int32), in these slots."""
    n, p = _batch(x, cache, "x")
    count = _count(slot)
    _mq._check(_lib().mqconv_cache_write(cache.c_struct(), p, n, *_int32("n0", n0), count, _slots(slot, count),
                                         _mq._stream(stream)), "mqconv_cache_write")


def mqconv_cache_read(cache: MxCache, slot, x, n0: int = 0, stream=None) -> None:
    """Writes the values of the slots to samples n0 .. of x [H][W][N][C]."""
    n, p = _batch(x, cache, "x")
    count = _count(slot)
    _mq._check(_lib().mqconv_cache_read(cache.c_struct(), _slots(slot, count), count, p, n, *_int32("n0", n0),
                                        _mq._stream(stream)), "mqconv_cache_read")


def mqconv_cache_read_mx(cache: MxCache, slot, xq, stream=None) -> None:
    """The slots' samples as the ACT MxTensor xq, one for each of its samples."""
    _mq._check(_lib().mqconv_cache_read_mx(cache.c_struct(), _slots(slot, xq.dims[2]), xq.c_struct("xq"),
                                           _mq._stream(stream)), "mqconv_cache_read_mx")
