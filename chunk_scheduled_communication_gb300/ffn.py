"""ctypes binding of the gated feed-forward block (include/syn_ffn.h).

Argument marshalling only: every step of the operators runs in libsyn.so.
Matrices are 2-D with any row stride (a multiple of 8 elements) and contiguous
rows; outputs are the caller's."""
from __future__ import annotations

import ctypes
import struct

from torch.cuda import current_device

from . import syn
from .norm import matrix_of
from .rope import DTYPES, packed, torch_dtype

_P = ctypes.c_void_p
_I64 = ctypes.c_int64

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class FfnCfg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("d", ctypes.c_int), ("d_ff", ctypes.c_int), ("act", ctypes.c_int),
                ("backward", ctypes.c_int), ("saved_f32", ctypes.c_int), ("timeout_ns", ctypes.c_uint64)]


class Mat(ctypes.Structure):
    _fields_ = [("p", _P), ("row", _I64)]


_M = ctypes.POINTER(Mat)
SIGS = {
    "syn_ffn_cfg_default": (ctypes.c_int, [ctypes.POINTER(FfnCfg)]),
    "syn_ffn_plan_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.POINTER(FfnCfg)]),
    "syn_ffn_plan_destroy": (ctypes.c_int, [_P]),
    "syn_ffn_plan_parts": (ctypes.c_int, [_P, _I64, ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "syn_gated_ffn": (ctypes.c_int, [_P, _M, _M, _M, _M, _M, _M, _I64, _P]),
    "syn_gated_ffn_backward": (ctypes.c_int, [_P, _M, _M, _M, _M, _M, _M, _M, _M, _M, _M, _M, _I64, _P]),
    "syn_ffn_sync_status": (ctypes.c_int, [_P, _P]),
}

_bound = None
_pack = struct.Struct("Pq").pack  # (structures as packed bytes: see rope.packed)


def lib():
    """libsyn.so with the gated block's signatures bound (raises if the library is missing)."""
    global _bound
    L = syn.lib()
    if _bound is not L:
        for name, (res, args) in SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return L


def _check(status, where):
    if status != syn.OK:
        raise syn.SynError(status, where)


class FfnPlan:
    """Gated feed-forward block on the current CUDA device (wraps syn_ffn_plan_t):
    X [tokens, d], Wg and Wu [d, d_ff], H, G and U [tokens, d_ff].  ``saved``: the type of G
    and U, "fp32" or (None) that of the others."""

    def __init__(self, d=4096, d_ff=14336, act="silu", dtype="bf16", backward=True, saved=None, timeout_ns=0):
        self._L = lib()
        self._h = _P()
        c = FfnCfg()
        _check(self._L.syn_ffn_cfg_default(ctypes.byref(c)), "syn_ffn_cfg_default")
        c.dtype, c.d, c.d_ff, c.act = DTYPES[dtype], d, d_ff, ACTS[act]
        if saved not in (None, dtype, "fp32"):
            raise ValueError(f"saved must be None, {dtype!r} or 'fp32'")
        c.backward, c.saved_f32, c.timeout_ns = int(bool(backward)), int(saved == "fp32"), timeout_ns
        self.cfg, self.dtype, self.saved = c, torch_dtype(dtype), torch_dtype(saved or dtype)
        self._forward, self._backward = (packed(self._L, SIGS, n) for n in ("syn_gated_ffn", "syn_gated_ffn_backward"))
        _check(self._L.syn_ffn_plan_create(ctypes.byref(self._h), ctypes.byref(c)), "syn_ffn_plan_create")
        self._device = current_device()

    def close(self):
        if self._h:
            self._L.syn_ffn_plan_destroy(self._h)
            self._h = _P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def _x(self, name, t, n):
        return None if t is None else _pack(*matrix_of(name, t, self.dtype, n, self.cfg.d, self._device))

    def _w(self, name, t):
        return None if t is None else _pack(*matrix_of(name, t, self.dtype, self.cfg.d, self.cfg.d_ff, self._device))

    def _f(self, name, t, n):
        return None if t is None else _pack(*matrix_of(name, t, self.dtype, n, self.cfg.d_ff, self._device))

    def _s(self, name, t, n):
        return None if t is None else _pack(*matrix_of(name, t, self.saved, n, self.cfg.d_ff, self._device))

    def parts(self, tokens, dX=True, dW=True):
        """Parts that the longer tiles of forward's and backward's products are cut into (1: whole)."""
        forward, backward = ctypes.c_int(), ctypes.c_int()
        _check(self._L.syn_ffn_plan_parts(self._h, tokens, int(dX) + 2 * int(dW), ctypes.byref(forward), ctypes.byref(backward)),
               "syn_ffn_plan_parts")
        return forward.value, backward.value

    def forward(self, X, Wg, Wu, H, G=None, U=None, stream=None):
        """H = act(X Wg) * (X Wu); G and U, which backward needs, where given."""
        n = X.shape[0]
        _check(self._forward(self._h, self._x("X", X, n), self._w("Wg", Wg), self._w("Wu", Wu), self._f("H", H, n),
                             self._s("G", G, n), self._s("U", U, n), n, syn._stream(stream)), "syn_gated_ffn")

    def backward(self, dH, X, Wg, Wu, G, U, dG, dU, dX=None, dWg=None, dWu=None, stream=None):
        """dG and dU (in place where G and U are of their type: dG=G, dU=U), dX (None: not wanted), dWg and dWu
        (None: not wanted) from dH, the forward's inputs and its G and U."""
        n = dH.shape[0]
        _check(self._backward(self._h, self._f("dH", dH, n), self._x("X", X, n), self._w("Wg", Wg), self._w("Wu", Wu),
                              self._s("G", G, n), self._s("U", U, n), self._f("dG", dG, n), self._f("dU", dU, n),
                              self._x("dX", dX, n), self._w("dWg", dWg), self._w("dWu", dWu), n, syn._stream(stream)),
               "syn_gated_ffn_backward")

    def sync(self, stream=None) -> int:
        return int(self._L.syn_ffn_sync_status(self._h, syn._stream(stream)))

    def check(self, stream=None):
        _check(self.sync(stream), "syn_ffn_sync_status")
