"""ctypes binding of the windowed attention and its decoding step (include/syn_window.h).

Argument marshalling only: every step of the operators runs in libsyn.so.
Tensors are ``[rows, heads, d]`` with contiguous heads; outputs are the
caller's."""
from __future__ import annotations

import ctypes
import struct

import numpy as np
from torch import float32 as _float32, int32 as _int32

from . import syn
from .rope import DTYPES, check_vector, heads_of, packed, torch_dtype

_P = ctypes.c_void_p
_I64 = ctypes.c_int64


class WindowCfg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int),
                ("window", _I64), ("sinks", ctypes.c_int), ("scale", ctypes.c_float), ("backward", ctypes.c_int),
                ("timeout_ns", ctypes.c_uint64)]


class Rows(ctypes.Structure):
    _fields_ = [("p", _P), ("token", _I64), ("head", _I64)]


class WindowInfo(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_items", ctypes.c_int), ("n_bwd_items", ctypes.c_int),
                ("n_parts", ctypes.c_int), ("grid", ctypes.c_int), ("q_rows", _I64), ("k_rows", _I64), ("pairs", _I64),
                ("workspace_bytes", _I64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class DecodeCfg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("max_seqs", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("d", ctypes.c_int), ("window", _I64), ("sinks", ctypes.c_int), ("page_size", ctypes.c_int),
                ("scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("p", _P), ("page", _I64), ("token", _I64), ("head", _I64)]


_R, _C = ctypes.POINTER(Rows), ctypes.POINTER(Cache)
SIGS = {
    "syn_window_cfg_default": (ctypes.c_int, [ctypes.POINTER(WindowCfg)]),
    "syn_window_plan_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.POINTER(WindowCfg), ctypes.c_int, _P, _P]),
    "syn_window_plan_destroy": (ctypes.c_int, [_P]),
    "syn_window_plan_query": (ctypes.c_int, [_P, ctypes.POINTER(WindowInfo)]),
    "syn_window_attention": (ctypes.c_int, [_P, _R, _R, _R, _R, _P, _P]),
    "syn_window_attention_backward": (ctypes.c_int, [_P, _R, _R, _R, _R, _R, _P, _R, _R, _R, _P]),
    "syn_window_sync_status": (ctypes.c_int, [_P, _P]),
    "syn_decode_cfg_default": (ctypes.c_int, [ctypes.POINTER(DecodeCfg)]),
    "syn_decode_plan_create": (ctypes.c_int, [ctypes.POINTER(_P), ctypes.POINTER(DecodeCfg)]),
    "syn_decode_plan_destroy": (ctypes.c_int, [_P]),
    "syn_window_decode": (ctypes.c_int, [_P, _R, _C, _C, _P, _I64, _I64, _P, ctypes.c_int, _R, _P, _P]),
    "syn_decode_sync_status": (ctypes.c_int, [_P, _P]),
}

_bound = None
# the decoding step's structures as packed bytes (see rope.packed)
_pack_rows, _pack_cache = struct.Struct("Pqq").pack, struct.Struct("Pqqq").pack


def lib():
    """libsyn.so with the windowed-attention signatures bound (raises if the library is missing)."""
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


def _rows(name, t, dtype, d, rows, heads):
    return Rows(*heads_of(name, t, dtype, d, rows, heads)[:3])


def _lse(lse, rows, heads):
    if lse is None:
        return None
    if lse.dtype is not _float32 or not lse.is_cuda or lse.shape != (rows, heads) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous CUDA tensor [{rows}, {heads}] of float32")
    return lse.data_ptr()


class WindowPlan:
    """Attention of ragged sequences with a sliding window and sinks on the
    current CUDA device (wraps syn_window_plan_t).

    The plan depends on the lengths alone: make it once for a batch, use it in
    every layer.  ``window`` 0 sees all earlier keys."""

    def __init__(self, q_lens, k_lens=None, H_q=1, H_kv=1, d=128, window=0, sinks=0, scale=0.0, dtype="bf16",
                 backward=False, timeout_ns=0):
        self._L = lib()
        self._h = _P()
        q = np.ascontiguousarray(q_lens, dtype=np.int64).reshape(-1)
        k = q if k_lens is None else np.ascontiguousarray(k_lens, dtype=np.int64).reshape(-1)
        if q.shape != k.shape:
            raise ValueError("q_lens and k_lens need one entry per sequence")
        c = WindowCfg()
        _check(self._L.syn_window_cfg_default(ctypes.byref(c)), "syn_window_cfg_default")
        c.dtype, c.H_q, c.H_kv, c.d, c.window, c.sinks = DTYPES[dtype], H_q, H_kv, d, window, sinks
        c.scale, c.backward, c.timeout_ns = scale, int(bool(backward)), timeout_ns
        self.cfg, self.dtype = c, torch_dtype(dtype)
        _check(self._L.syn_window_plan_create(ctypes.byref(self._h), ctypes.byref(c), len(q), q.ctypes.data, k.ctypes.data),
               "syn_window_plan_create")
        self.q_rows, self.k_rows = int(q.sum()), int(k.sum())

    def close(self):
        if self._h:
            self._L.syn_window_plan_destroy(self._h)
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

    def info(self) -> dict:
        i = WindowInfo()
        _check(self._L.syn_window_plan_query(self._h, ctypes.byref(i)), "syn_window_plan_query")
        return i.as_dict()

    def _q(self, name, t):
        return _rows(name, t, self.dtype, self.cfg.d, self.q_rows, self.cfg.H_q)

    def _k(self, name, t):
        return _rows(name, t, self.dtype, self.cfg.d, self.k_rows, self.cfg.H_kv)

    def forward(self, Q, K, V, O, lse=None, stream=None):
        """O (and lse, fp32 [rows, H_q]) of Q over K, V."""
        _check(self._L.syn_window_attention(self._h, self._q("Q", Q), self._k("K", K), self._k("V", V), self._q("O", O),
                                            _lse(lse, self.q_rows, self.cfg.H_q), syn._stream(stream)),
               "syn_window_attention")

    def backward(self, dO, Q, K, V, O, lse, dQ, dK, dV, stream=None):
        """dQ, dK, dV from dO, the forward's inputs, its O and lse."""
        if lse is None:
            raise ValueError("backward needs the forward's lse")
        _check(self._L.syn_window_attention_backward(
            self._h, self._q("dO", dO), self._q("Q", Q), self._k("K", K), self._k("V", V), self._q("O", O),
            _lse(lse, self.q_rows, self.cfg.H_q), self._q("dQ", dQ), self._k("dK", dK), self._k("dV", dV),
            syn._stream(stream)), "syn_window_attention_backward")

    def sync(self, stream=None) -> int:
        return int(self._L.syn_window_sync_status(self._h, syn._stream(stream)))

    def check(self, stream=None):
        _check(self.sync(stream), "syn_window_sync_status")


class DecodePlan:
    """One query token per sequence over a paged cache ``[pages, page_size,
    H_kv, d]`` on the current CUDA device (wraps syn_decode_plan_t)."""

    def __init__(self, max_seqs=1, H_q=1, H_kv=1, d=128, window=0, sinks=0, page_size=64, scale=0.0, dtype="bf16"):
        self._L = lib()
        self._h = _P()
        c = DecodeCfg()
        _check(self._L.syn_decode_cfg_default(ctypes.byref(c)), "syn_decode_cfg_default")
        c.dtype, c.max_seqs, c.H_q, c.H_kv, c.d = DTYPES[dtype], max_seqs, H_q, H_kv, d
        c.window, c.sinks, c.page_size, c.scale = window, sinks, page_size, scale
        self.cfg, self.dtype, self._page = c, torch_dtype(dtype), (page_size, H_kv, d)
        self._decode = packed(self._L, SIGS, "syn_window_decode")
        _check(self._L.syn_decode_plan_create(ctypes.byref(self._h), ctypes.byref(c)), "syn_decode_plan_create")

    def close(self):
        if self._h:
            self._L.syn_decode_plan_destroy(self._h)
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

    def _cache(self, name, t):
        c, shape, stride = self.cfg, t.shape, t.stride()
        if t.dtype is not self.dtype or not t.is_cuda or len(shape) != 4 or shape[1:] != self._page or stride[3] != 1:
            raise ValueError(f"{name} must be a CUDA tensor [pages, {c.page_size}, {c.H_kv}, {c.d}] of type {self.dtype} "
                             "with contiguous heads")
        return _pack_cache(t.data_ptr(), stride[0], stride[1], stride[2])

    def run(self, q, k_cache, v_cache, seq_lens, O, lse=None, page_table=None, stream=None):
        """O of each sequence's last token q[s] over its seq_lens[s] cached tokens.
        page_table: int32 [sequences, pages of a sequence]; None: sequence s is page s."""
        c, n = self.cfg, q.shape[0]
        d, heads = c.d, c.H_q
        qr = _pack_rows(*heads_of("q", q, self.dtype, d, n, heads)[:3])
        out = _pack_rows(*heads_of("O", O, self.dtype, d, n, heads)[:3])
        k, v = self._cache("k_cache", k_cache), self._cache("v_cache", v_cache)
        pages = k_cache.shape[0]
        if v_cache.shape[0] != pages:
            raise ValueError("k_cache and v_cache must have the same pages")
        lens, table, stride = check_vector("seq_lens", seq_lens, _int32, n), None, 0
        if page_table is not None:
            shape = page_table.shape
            if page_table.dtype is not _int32 or not page_table.is_cuda or len(shape) != 2 or shape[0] != n or \
                    not page_table.is_contiguous():
                raise ValueError(f"page_table must be a contiguous CUDA tensor [{n}, pages] of int32")
            # (a table without entries has no address, and no table would mean a contiguous cache: any address, never read)
            table, stride = page_table.data_ptr() or lens, shape[1]
        _check(self._decode(self._h, qr, k, v, table, stride, pages, lens, n, out, _lse(lse, n, heads),
                                         syn._stream(stream)), "syn_window_decode")

    def sync(self, stream=None) -> int:
        return int(self._L.syn_decode_sync_status(self._h, syn._stream(stream)))

    def check(self, stream=None):
        _check(self.sync(stream), "syn_decode_sync_status")
