"""Orthogonalised updates of libkfac.so (include/kfac_orthogonal.h).

    Orthogonal       the nearest-to-orthogonal update of a matrix, or of a batch of one shape
    OrthogonalStep   momentum, that update, weight decay and the parameter write for a stack of layers

``OrthogonalStep`` is a third step beside ``KfacStack``'s two: it needs only
the gradients of the weights, and its cost does not grow with the rows of a
batch.  Its tensors may be a ``KfacStack``'s state.  One object is for one call
at a time, and a graph that captured its calls works in its workspace.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import F32, HParams, KFAC_ERR_ARG, KFAC_ERR_DTYPE, KFAC_OK, KfacError, LINEAR, Layer, layer_array, load, make_layer
from .objectives import _DTYPES, _Operator, _Plan

PRODUCTS_HALF, PRODUCTS_FULL = 0, 1
SCALE_NONE, SCALE_ASPECT, SCALE_RMS = 0, 1, 2
EXPORTS = ("kfac_orthogonal_workspace_size", "kfac_orthogonal_step_workspace_size", "kfac_orthogonalize",
           "kfac_step_orthogonal")
COEFS = (3.4445, -4.7750, 2.0315)
_PRODUCTS = {"half": PRODUCTS_HALF, "full": PRODUCTS_FULL}
_SCALES = {"none": SCALE_NONE, "aspect": SCALE_ASPECT, "rms": SCALE_RMS}

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class How(ctypes.Structure):
    """Mirror of kfac_orthogonal_t."""
    _fields_ = [("coefs", _vp), ("eps", ctypes.c_double), ("steps", _i32), ("products", _i32), ("nesterov", _i32),
                ("scale", _i32)]


class Matrix(ctypes.Structure):
    """Mirror of kfac_orthogonal_matrix_t."""
    _fields_ = [("x", _vp), ("y", _vp), ("ld", _i64), ("stride", _i64), ("y_ld", _i64), ("y_stride", _i64),
                ("rows", _i32), ("cols", _i32), ("batch", _i32), ("dtype", _i32)]


class _OrthogonalPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("m", Matrix), ("how", How)]


class _StepPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("layers", _vp), ("weights", _vp), ("n", _i64), ("how", How), ("hp", HParams)]


_lib = None
_native = None


def _library() -> ctypes.CDLL:
    """The library with the argument types of this module's functions set."""
    global _lib, _native
    if _lib is not None:
        return _lib
    from . import tokens
    lib = load()
    sz, how = ctypes.c_size_t, ctypes.POINTER(How)
    lib.kfac_orthogonal_workspace_size.argtypes = [ctypes.POINTER(Matrix), how, ctypes.POINTER(sz)]
    lib.kfac_orthogonal_step_workspace_size.argtypes = [ctypes.POINTER(Layer), _i32, how, ctypes.POINTER(sz)]
    lib.kfac_orthogonalize.argtypes = [ctypes.POINTER(Matrix), how, _vp, sz, _vp]
    lib.kfac_step_orthogonal.argtypes = [ctypes.POINTER(Layer), _i32, ctypes.POINTER(HParams), how, _vp, sz, _vp]
    for name in EXPORTS:
        getattr(lib, name).restype = _i32
    _native = tokens._extension()
    _lib = lib
    return lib


class _Iteration(_Operator):
    """The iteration's constants."""

    def _how(self, steps, coefs, eps, products, nesterov=0, scale="none") -> How:
        if not 1 <= steps <= 16:
            self._fail("steps must lie in 1 .. 16")
        flat = list(coefs)
        if len(flat) == 3 and not hasattr(flat[0], "__len__"):
            flat = flat * steps
        else:
            if len(flat) != steps or any(len(c) != 3 for c in flat):
                self._fail("coefs must be (a, b, c), or one such triple a step")
            flat = [v for c in flat for v in c]
        if any(not abs(v) <= 64.0 for v in flat):
            self._fail("coefs must lie in [-64, 64]")
        if not 0.0 <= eps < float("inf"):
            self._fail("eps must be at least 0 and finite")
        if products not in _PRODUCTS:
            self._fail("products must be 'half' or 'full'")
        if scale not in _SCALES:
            self._fail("scale must be 'none', 'aspect' or 'rms'")
        self._coefs = (ctypes.c_float * len(flat))(*flat)
        return How(coefs=ctypes.addressof(self._coefs), eps=eps, steps=steps, products=_PRODUCTS[products],
                   nesterov=int(nesterov), scale=_SCALES[scale])


class Orthogonal(_Iteration):
    """O(x) of kfac_orthogonal.h: x's singular values brought near 1 by `steps` Newton-Schulz products.

    rows, cols, batch: the shape of x.  dtype: "bf16" or "f32", of x and the
    result.  coefs: (a, b, c) of every step, or one such triple a step.
    products: "half" holds the iteration's matrices in 11 bits (the default
    for bf16; off by 5e-4 to 1.2e-3, and by up to 1.2e-2 for matrices without
    rank or with equal singular values), "full" in 22 (for f32; as exact as
    float32 products make it).
    """

    def __init__(self, rows: int, cols: int, batch: int = 1, dtype: str = "bf16", steps: int = 5, coefs=COEFS,
                 eps: float = 1e-7, products: Optional[str] = None, device="cuda"):
        self._where = type(self).__name__
        if dtype not in _DTYPES:
            self._fail("dtype must be 'bf16' or 'f32'", KFAC_ERR_DTYPE)
        if rows < 1 or cols < 1 or batch < 0 or max(rows, cols, batch) >= 1 << 31:
            self._fail("rows and cols must be at least 1, batch at least 0")
        how = self._how(steps, coefs, eps, products or ("half" if dtype == "bf16" else "full"))
        m = Matrix(rows=rows, cols=cols, batch=batch, dtype=_DTYPES[dtype][0])
        size = ctypes.c_size_t(0)
        st = _library().kfac_orthogonal_workspace_size(ctypes.byref(m), ctypes.byref(how), ctypes.byref(size))
        if st != KFAC_OK:
            raise KfacError(st, f"{self._where}: kfac_orthogonal_workspace_size")
        plan = _OrthogonalPlan()
        super().__init__(plan, dtype, device, ws_bytes=size.value)
        plan.m, plan.how = m, how

    def run(self, x, out=None, stream=None):
        """O(x), of x's shape: [batch, rows, cols], or [rows, cols] where batch is 1 (rows and matrices any
        stride apart).  out: where to write; it may be x itself.  The result is outside autograd."""
        if stream is None:
            return _native.orthogonalize(self._at, x, out)
        return self._on(stream, _native.orthogonalize, x, out)


class OrthogonalStep(_Iteration):
    """One step of a stack of layers (kfac_step_orthogonal gives the formulas).

    weights, momenta: float32 [d_out, d_in] each, contiguous, written in
    place, where each tensor's memory is when run() is called (a captured step
    goes on writing where it was).  biases, bias_momenta: [d_out] each, or None
    for a layer without one.  nesterov: whether the update looks ahead by the
    momentum.  scale: the factor of a layer's step, "aspect" sqrt(max(1,
    d_out / d_in)), "rms" 0.2 sqrt(max(d_out, d_in)) or "none" 1.  products:
    "full" (the update as exact as float32 products make it) or "half" (11 bits
    between the products, a third of the operations; Orthogonal says how far
    off).
    """

    def __init__(self, weights: Sequence, momenta: Sequence, biases: Optional[Sequence] = None,
                 bias_momenta: Optional[Sequence] = None, steps: int = 5, coefs=COEFS, eps: float = 1e-7,
                 nesterov: bool = True, scale: str = "aspect", products: str = "full"):
        self._where = type(self).__name__
        n = len(weights)
        if n < 1 or len(momenta) != n:
            self._fail("weights and momenta must be lists of the same length")
        biases = [None] * n if biases is None else list(biases)
        bias_momenta = [None] * n if bias_momenta is None else list(bias_momenta)
        if len(biases) != n or len(bias_momenta) != n:
            self._fail("biases and bias_momenta must be as many as weights")
        written = [*weights, *momenta, *[b for b in (*biases, *bias_momenta) if b is not None]]
        if not all(isinstance(t, torch.Tensor) for t in written):
            self._fail("weights, momenta and biases must be tensors")
        dev = weights[0].device
        for t in written:
            if t.dtype != torch.float32:
                self._fail("weights, momenta and biases must be float32", KFAC_ERR_DTYPE)
            if t.device != dev or not t.is_contiguous():
                self._fail("weights, momenta and biases must be contiguous, on one device")
        spans = sorted((t.data_ptr(), t.data_ptr() + 4 * t.numel()) for t in written)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            self._fail("weights, momenta and biases must not share memory")
        descs = []
        for w, m, b, bm in zip(weights, momenta, biases, bias_momenta):
            if w.dim() != 2 or w.numel() == 0 or m.shape != w.shape:
                self._fail("a weight must be [d_out, d_in], and its momentum as large")
            if (b is None) != (bm is None):
                self._fail("a bias needs its momentum")
            if b is not None and (b.shape != (w.shape[0],) or bm.shape != b.shape):
                self._fail("a bias and its momentum must be [d_out]")
            more = {} if b is None else {"b": b, "mom_b": bm}
            descs.append(make_layer(LINEAR, w.shape[1], w.shape[0], 0, b is not None, w=w, mom_w=m, **more))
        how = self._how(steps, coefs, eps, products, nesterov, scale)
        self._layers = layer_array(descs)
        size = ctypes.c_size_t(0)
        st = _library().kfac_orthogonal_step_workspace_size(self._layers, n, ctypes.byref(how), ctypes.byref(size))
        if st != KFAC_OK:
            raise KfacError(st, f"{self._where}: kfac_orthogonal_step_workspace_size")
        plan = _StepPlan()
        super().__init__(plan, "f32", dev, ws_bytes=size.value)
        self._written = written
        plan.layers = ctypes.addressof(self._layers)
        plan.weights = id(self._written)
        plan.n, plan.how = n, how

    def run(self, grads, bias_grads=None, lr: float = 0.02, momentum: float = 0.95, weight_decay: float = 0.0,
            stream=None):
        """One step in place: grads [d_out, d_in] float32, contiguous, one a weight; bias_grads [d_out], None
        for a layer without bias."""
        if stream is None:
            return _native.orthogonal_step(self._at, grads, bias_grads, lr, momentum, weight_decay)
        return self._on(stream, _native.orthogonal_step, grads, bias_grads, lr, momentum, weight_decay)
