"""ctypes binding of the rotary-position and head-norm entry points (include/syn_rope.h).

Argument marshalling only: every step of the operators runs in libsyn.so.
Tensors are ``[tokens, heads, d]`` with any token and head strides and
contiguous heads; outputs are the caller's."""
from __future__ import annotations

import ctypes
import struct

import numpy as np
from torch import float32 as _float32, int64 as _int64

from . import syn

_P = ctypes.c_void_p
_I64 = ctypes.c_int64

DTYPES = {"bf16": 0, "fp16": 1, "fp32": 2}
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}


class RopeCfg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("d", ctypes.c_int), ("d_rot", ctypes.c_int), ("layout", ctypes.c_int),
                ("base", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("original_context", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


class Rows(ctypes.Structure):
    _fields_ = [("x", _P), ("x_token", _I64), ("x_head", _I64), ("y", _P), ("y_token", _I64), ("y_head", _I64),
                ("heads", ctypes.c_int)]


class Grad(ctypes.Structure):
    _fields_ = [("x", _P), ("x_token", _I64), ("x_head", _I64), ("dy", _P), ("dy_token", _I64), ("dy_head", _I64),
                ("dx", _P), ("dx_token", _I64), ("dx_head", _I64), ("w", _P), ("dw", _P), ("heads", ctypes.c_int)]


_R, _G = ctypes.POINTER(Rows), ctypes.POINTER(Grad)
SIGS = {
    "syn_rope_cfg_default": (ctypes.c_int, [ctypes.POINTER(RopeCfg)]),
    "syn_rope_plan_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.POINTER(RopeCfg)]),
    "syn_rope_plan_destroy": (ctypes.c_int, [_P]),
    "syn_rope_plan_frequencies": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_double)]),
    "syn_rope": (ctypes.c_int, [_P, _R, _R, _R, _P, _I64, _P, _I64, _I64, _P]),
    "syn_rope_backward": (ctypes.c_int, [_P, _R, _R, _P, _I64, _I64, _P]),
    "syn_qk_norm_rope": (ctypes.c_int, [_P, _R, _P, _R, _P, ctypes.c_float, _R, _P, _I64, _P, _I64, _I64, _P]),
    "syn_qk_norm_rope_backward": (ctypes.c_int, [_P, _G, _G, ctypes.c_float, _P, _I64, _I64, _P]),
}

_bound = None
# the same calls with the structures as packed bytes, which cost a small call a third of what
# structure objects do (a decoding step's calls are bound by the host)
_pack_rows = struct.Struct("PqqPqqi4x").pack
assert struct.calcsize("PqqPqqi4x") == ctypes.sizeof(Rows)


def lib():
    """libsyn.so with the rotary signatures bound (raises if the library is missing)."""
    global _bound
    L = syn.lib()
    if _bound is not L:
        for name, (res, args) in SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return L


def packed(L, sigs, name):
    """Function `name` with pointers to structures taken as bytes."""
    res, args = sigs[name]
    plain = [a if issubclass(a, ctypes._SimpleCData) else _P for a in args]
    return ctypes.CFUNCTYPE(res, *plain)((name, L))


def _check(status, where):
    if status != syn.OK:
        raise syn.SynError(status, where)


def make_cfg(d=128, d_rot=None, layout="half", base=10000.0, scaling=None, attn_factor=0.0, dtype="bf16") -> RopeCfg:
    """scaling: None or a dict of ``kind`` ("linear", "ntk", "llama3", "yarn") and that kind's fields."""
    c = RopeCfg()
    _check(lib().syn_rope_cfg_default(ctypes.byref(c)), "syn_rope_cfg_default")
    c.d, c.d_rot = d, d if d_rot is None else d_rot
    c.layout, c.base, c.attn_factor, c.dtype = LAYOUTS[layout], base, attn_factor, DTYPES[dtype]
    more = dict(scaling or {})
    c.scaling = SCALINGS[more.pop("kind", "none")]
    for name, value in more.items():
        if name not in ("factor", "low_freq_factor", "high_freq_factor", "original_context", "beta_fast", "beta_slow"):
            raise ValueError(f"unknown scaling field {name!r}")
        setattr(c, name, float(value))
    return c


def torch_dtype(dtype):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]


def heads_of(name, t, dtype, d, tokens, heads=None):
    """(address, token stride, head stride, heads) of a CUDA tensor [tokens,
    heads, d] of type `dtype` with contiguous heads; None: any number."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3 and t.dtype is dtype and t.is_cuda:
        n, h, e = shape
        if e == d and (stride[2] == 1 or d == 1) and (tokens is None or n == tokens) and (heads is None or h == heads):
            return t.data_ptr(), stride[0], stride[1], h
    if t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of type {dtype}")
    if len(shape) != 3 or shape[2] != d or (stride[2] != 1 and d > 1):
        raise ValueError(f"{name} must be [tokens, heads, {d}] with contiguous heads")
    raise ValueError(f"{name} must have {tokens} rows of {heads} heads")


def check_vector(name, t, dtype, n):
    if t.dtype is not dtype or not t.is_cuda or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} {dtype}")
    return t.data_ptr()


class RopePlan:
    """Rotary positions on the current CUDA device (wraps syn_rope_plan_t)."""

    def __init__(self, **cfg):
        self._L = lib()
        self._h = _P()
        self.cfg = make_cfg(**cfg)
        self.dtype, self._d = torch_dtype(cfg.get("dtype", "bf16")), self.cfg.d
        self._rope, self._norm, self._back = (packed(self._L, SIGS, n) for n in ("syn_rope", "syn_qk_norm_rope",
                                                                                 "syn_rope_backward"))
        _check(self._L.syn_rope_plan_create(ctypes.byref(self._h), ctypes.byref(self.cfg)), "syn_rope_plan_create")

    def close(self):
        if self._h:
            self._L.syn_rope_plan_destroy(self._h)
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

    def frequencies(self):
        """(radians per position of each pair, factor on the rotated elements)."""
        f, a = np.empty(self.cfg.d_rot // 2, np.float64), ctypes.c_double()
        _check(self._L.syn_rope_plan_frequencies(self._h, f.ctypes.data, ctypes.byref(a)), "syn_rope_plan_frequencies")
        return f, a.value

    def _rows(self, name, x, y, tokens, slots=False):
        if x is None:
            return None
        d, dtype = self._d, self.dtype
        p, xt, xh, heads = heads_of(name, x, dtype, d, tokens)
        q, yt, yh, _ = heads_of(name + "_out", y, dtype, d, None if slots else tokens, heads)
        return _pack_rows(p, xt, xh, q, yt, yh, heads)

    def _forward(self, q, q_out, wq, k, k_out, wk, eps, v, v_out, positions, pos0, slots, stream, norm):
        first = q if q is not None else k if k is not None else v
        if first is None:
            raise ValueError("one of q, k and v is needed")
        n, scatter, n_slots = first.shape[0], slots is not None, 0
        rq = self._rows("q", q, q_out, n)
        rk, rv = self._rows("k", k, k_out, n, scatter), self._rows("v", v, v_out, n, scatter)
        pos = None if positions is None else check_vector("positions", positions, _int64, n)
        slot = None
        if scatter:
            slot = check_vector("slots", slots, _int64, n)
            n_slots = min((o.shape[0] for t, o in ((k, k_out), (v, v_out)) if t is not None), default=0)
        if not norm:
            _check(self._rope(self._h, rq, rk, rv, pos, pos0, slot, n_slots, n, syn._stream(stream)), "syn_rope")
            return
        a = None if wq is None else check_vector("wq", wq, self.dtype, self._d)
        b = None if wk is None else check_vector("wk", wk, self.dtype, self._d)
        _check(self._norm(self._h, rq, a, rk, b, eps, rv, pos, pos0, slot, n_slots, n, syn._stream(stream)),
               "syn_qk_norm_rope")

    def rotate(self, q, q_out, k=None, k_out=None, v=None, v_out=None, positions=None, pos0=0, slots=None, stream=None):
        """Rotate q and k, copy v; with `slots`, k and v go to those rows of k_out and v_out."""
        self._forward(q, q_out, None, k, k_out, None, 0.0, v, v_out, positions, pos0, slots, stream, False)

    def norm_rotate(self, q, q_out, wq, k=None, k_out=None, wk=None, v=None, v_out=None, positions=None, pos0=0,
                    eps=1e-6, slots=None, stream=None):
        """Norm of each head with weights wq, wk (None: ones), then `rotate`."""
        self._forward(q, q_out, wq, k, k_out, wk, eps, v, v_out, positions, pos0, slots, stream, True)

    def rotate_backward(self, dq_out, dq, dk_out=None, dk=None, positions=None, pos0=0, stream=None):
        """dq, dk from the gradients dq_out, dk_out of rotate's outputs."""
        first = dq_out if dq_out is not None else dk_out
        if first is None:
            raise ValueError("one of dq_out and dk_out is needed")
        n = first.shape[0]
        pos = None if positions is None else check_vector("positions", positions, _int64, n)
        _check(self._back(self._h, self._rows("dq_out", dq_out, dq, n), self._rows("dk_out", dk_out, dk, n),
                                         pos, pos0, n, syn._stream(stream)), "syn_rope_backward")

    def _grad(self, name, x, dy, dx, w, dw, n):
        if x is None:
            return None
        d, dtype = self._d, self.dtype
        p, xt, xh, heads = heads_of(name, x, dtype, d, n)
        g, gt, gh, _ = heads_of("d" + name + "_out", dy, dtype, d, n, heads)
        o, ot, oh, _ = heads_of("d" + name, dx, dtype, d, n, heads)
        a = None if w is None else check_vector("w" + name, w, dtype, d)
        b = None if dw is None else check_vector("dw" + name, dw, _float32, d)
        return Grad(p, xt, xh, g, gt, gh, o, ot, oh, a, b, heads)

    def norm_rotate_backward(self, q, dq_out, dq, wq, dwq, k=None, dk_out=None, dk=None, wk=None, dwk=None,
                             positions=None, pos0=0, eps=1e-6, stream=None):
        """dq, dk and the weights' gradients dwq, dwk (fp32, None: not wanted)
        from norm_rotate's inputs and the gradients of its outputs."""
        first = q if q is not None else k
        if first is None:
            raise ValueError("one of q and k is needed")
        n = first.shape[0]
        pos = None if positions is None else check_vector("positions", positions, _int64, n)
        _check(self._L.syn_qk_norm_rope_backward(self._h, self._grad("q", q, dq_out, dq, wq, dwq, n),
                                                 self._grad("k", k, dk_out, dk, wk, dwk, n), eps, pos, pos0, n,
                                                 syn._stream(stream)), "syn_qk_norm_rope_backward")
