"""Operators between tokens and rows of libkfac.so (include/kfac_tokens.h).

    Sampler     a token of each row of logits, with temperature, top-k, top-p and min-p
    Embedding   rows of a table by token, scaled; the table's gradient and the tokens' counts

A round of training a policy over tokens begins and ends with them: the
embedding makes the first layer's rows, the sampler the labels and the old
log-probabilities that ``objectives.PolicyLoss`` takes, and the embedding's
gradient takes what has come back through the layers.  A negative token is one
that is left out in all three.

Each class holds the shape, the constants and the workspace of one operator, in
the manner of ``objectives``: ``run`` checks its tensors, allocates the outputs
that are not given and makes one call into the library on the current (or the
given) stream; the embedding is inside autograd.  One object is for one call at
a time, and a graph that captured its calls works in its workspace.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import KFAC_ERR_ARG, KFAC_ERR_DTYPE, KFAC_ERR_UNSUPPORTED, KFAC_OK, KfacError, load
from .objectives import _DTYPES, _Operator, _Plan

TOK_SAMPLE, TOK_EMBEDDING = 0, 1
EXPORTS = ("kfac_token_workspace_size", "kfac_sample_tokens", "kfac_embedding_lookup", "kfac_embedding_grad")

_vp, _i32, _i64, _f32, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double


class Sample(ctypes.Structure):
    """Mirror of kfac_sample_t."""
    _fields_ = [("logits", _vp), ("u", _vp), ("row_temperature", _vp), ("row_top_k", _vp), ("row_top_p", _vp),
                ("row_min_p", _vp), ("token", _vp), ("logp", _vp), ("kept", _vp), ("rows", _i64), ("ld", _i64),
                ("temperature", _f64), ("top_p", _f64), ("min_p", _f64), ("top_k", _i32), ("vocab", _i32),
                ("dtype", _i32), ("reserved", _i32)]


class EmbeddingArgs(ctypes.Structure):
    """Mirror of kfac_embedding_t."""
    _fields_ = [("table", _vp), ("y", _vp), ("ids", _vp), ("counts", _vp), ("tokens", _i64), ("table_ld", _i64),
                ("y_ld", _i64), ("vocab", _i32), ("width", _i32), ("dtype", _i32), ("table_dtype", _i32),
                ("id_type", _i32), ("scale", _f32), ("accumulate", _i32), ("reserved", _i32)]


class _SamplePlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("s", Sample)]


class _EmbeddingPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("e", EmbeddingArgs)]


_lib = None
_native = None


def _extension():
    """The _tokens extension, bound to the library; orthogonal's calls are in it too."""
    global _native
    if _native is not None:
        return _native
    from . import orthogonal
    try:
        from . import _tokens
    except ModuleNotFoundError as e:
        raise FileNotFoundError(f"{os.path.join(os.path.dirname(__file__), '_tokens.so')} is missing: build it "
                                "with `python -m second_order_optimizer_amd.build`") from e
    plans = (_SamplePlan, _EmbeddingPlan, orthogonal._OrthogonalPlan, orthogonal._StepPlan)
    if _tokens.plan_sizes() != tuple(ctypes.sizeof(p) for p in plans):
        raise RuntimeError("the _tokens extension is of another build than this package")
    lib = load()
    names = EXPORTS[1:] + orthogonal.EXPORTS[2:]
    _tokens.bind(KfacError, *[ctypes.cast(getattr(lib, name), _vp).value for name in names])
    _native = _tokens
    return _native


def _library() -> ctypes.CDLL:
    """The library with the argument types of this module's functions set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = load()
    sz = ctypes.c_size_t
    lib.kfac_token_workspace_size.argtypes = [_i32, _i64, _i32, _i32, ctypes.POINTER(sz)]
    lib.kfac_sample_tokens.argtypes = [ctypes.POINTER(Sample), _vp, sz, _vp]
    lib.kfac_embedding_lookup.argtypes = [ctypes.POINTER(EmbeddingArgs), _vp, sz, _vp]
    lib.kfac_embedding_grad.argtypes = [ctypes.POINTER(EmbeddingArgs), _vp, sz, _vp]
    for name in EXPORTS:
        getattr(lib, name).restype = _i32
    _extension()
    _lib = lib
    return lib


def workspace_size(op: int, rows: int, vocab: int, width: int = 1) -> int:
    """kfac_token_workspace_size."""
    out = ctypes.c_size_t(0)
    st = _library().kfac_token_workspace_size(op, rows, vocab, width, ctypes.byref(out))
    if st != KFAC_OK:
        raise KfacError(st, "kfac_token_workspace_size")
    return out.value


class Sampler(_Operator):
    """A token of each row of logits (kfac_sample_t gives the order of the columns and what is kept of it).

    dtype: "bf16" or "f32" (of the logits).  temperature: 0 takes the largest
    logit.  top_k: at most so many tokens are kept (0: all); top_p: the least
    number whose probabilities, of those that top_k keeps, add up to it (1:
    all); min_p: those of at least this share of the likeliest one's
    probability (0: all).
    """

    def __init__(self, rows: int, vocab: int, dtype: str = "bf16", temperature: float = 1.0, top_k: int = 0,
                 top_p: float = 1.0, min_p: float = 0.0, device="cuda"):
        self._where = type(self).__name__
        if rows < 0 or vocab < 1:
            self._fail("rows must be at least 0 and vocab at least 1")
        if vocab >= 1 << 20:
            self._fail("vocab must be below 2^20", KFAC_ERR_UNSUPPORTED)
        if not 0.0 <= temperature < float("inf"):
            self._fail("temperature must be at least 0 and finite")
        if not 0 <= top_k < 1 << 31:
            self._fail("top_k must be at least 0")
        if not 0.0 <= top_p <= 1.0 or not 0.0 <= min_p <= 1.0:
            self._fail("top_p and min_p must lie in [0, 1]")
        plan = _SamplePlan()
        super().__init__(plan, dtype, device, ws_bytes=workspace_size(TOK_SAMPLE, rows, vocab))
        self.rows, self.vocab = rows, vocab
        plan.s = Sample(rows=rows, vocab=vocab, dtype=self.code, temperature=temperature, top_k=top_k, top_p=top_p,
                        min_p=min_p)

    def run(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
        """Returns (token [rows] int64, logp [rows] float32, kept [rows] int32).

        logits [rows, vocab] (any row stride; minus infinity is never taken),
        u [rows] float32 in [0, 1): the draw.  temperature, top_p, min_p
        [rows] float32 and top_k [rows] int32 replace the operator's own, row
        by row.  logp is the token's log-probability in the whole row at its
        temperature, kept the number of tokens that were to choose from; a
        row without any has token -1, as one has whose values are no numbers
        (flagged).
        """
        if stream is None:
            return _native.sample(self._at, logits, u, temperature, top_k, top_p, min_p)
        return self._on(stream, _native.sample, logits, u, temperature, top_k, top_p, min_p)


class _EmbeddingNode(torch.autograd.Function):
    """The lookup's place in autograd: the table's gradient is dense."""

    @staticmethod
    def forward(ctx, table, ids, op, stream):
        # A leaf adds up its gradient on the stream where the first living graph found it, and the default
        # stream cannot take part in a capture: such a backward pass would end the process.
        if torch.cuda.is_current_stream_capturing() and _native.gathers_on_default(table):
            op._fail("a graph made on the default stream outside this capture still holds the table: drop its "
                     "result first, or make it on another stream", KFAC_ERR_UNSUPPORTED)
        ctx.op = op
        ctx.save_for_backward(ids)
        return op.run(table, ids, None, stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        return ctx.op.backward(dy.contiguous(), ids)[0], None, None, None


class Embedding(_Operator):
    """Rows of a table by token, times ``scale``, and the table's gradient.

    dtype: "bf16" or "f32", of the rows; table_dtype: of the table and its
    gradient (default: the rows').  Where the table requires grad, the result
    is part of autograd's graph; tensors with a forward-mode tangent are refused.
    """

    def __init__(self, rows: int, vocab: int, width: int, dtype: str = "bf16", table_dtype: Optional[str] = None,
                 scale: float = 1.0, device="cuda"):
        self._where = type(self).__name__
        table_dtype = dtype if table_dtype is None else table_dtype
        if table_dtype not in _DTYPES:
            self._fail("table_dtype must be 'bf16' or 'f32'", KFAC_ERR_DTYPE)
        if rows < 0 or vocab < 1 or width < 1:
            self._fail("rows must be at least 0, vocab and width at least 1")
        if not abs(scale) < float("inf"):
            self._fail("scale must be finite")
        if vocab >= 1 << 31 or width >= 1 << 31:
            self._fail("vocab and width must be below 2^31", KFAC_ERR_UNSUPPORTED)
        plan = _EmbeddingPlan()
        super().__init__(plan, dtype, device, ws_bytes=workspace_size(TOK_EMBEDDING, rows, vocab, width))
        self.rows, self.vocab, self.width = rows, vocab, width
        plan.e = EmbeddingArgs(tokens=rows, vocab=vocab, width=width, dtype=self.code,
                               table_dtype=_DTYPES[table_dtype][0], scale=scale)

    def run(self, table, ids, out=None, stream=None):
        """scale table[ids], [rows, width].

        table [vocab, width] (any row stride), ids [rows] int32 or int64: a
        negative one gives a row of zeros, one of at least vocab too (flagged).
        out: where to write, for calls outside autograd.  Inside a capture
        the call is refused while a graph of the same table lives, of this
        operator or any other (tied weights), that was made on the default
        stream.
        """
        if stream is None:
            y = _native.embedding(self._at, table, ids, out)
        else:
            y = self._on(stream, _native.embedding, table, ids, out)
        if y is None:           # the table requires grad, and autograd is on
            return _EmbeddingNode.apply(table, ids, self, stream)
        return y

    def backward(self, dy, ids, grad=None, accumulate: bool = False, stream=None):
        """(grad [vocab, width], counts [vocab] int32) from d loss / dy and the ids of run().

        grad: where to write it; with accumulate it is added there, and rows
        of tokens that do not occur are not touched.  A token's rows are
        added in their order, in float32: the same call gives the same bits.
        """
        if stream is None:
            return _native.embedding_grad(self._at, dy, ids, grad, accumulate)
        return self._on(stream, _native.embedding_grad, dy, ids, grad, accumulate)
