"""Training objectives and dropout of libkfac.so (include/kfac_objectives.h):
what stands on either side of an optimizer step and makes the rows it reads.

    TokenLogp        log-probability of each row's label
    PolicyLoss       clipped policy loss with a KL term, logit gradients
    PreferenceLoss   loss over pairs of sequences, logit gradients
    BalanceLoss      router balance loss with per-expert counts, gradients
    Dropout          dropout from a counter-based generator, no mask stored

Each class holds the shape, the constants and the workspace of one operator;
``run`` checks its tensors, allocates the outputs that are not given and makes
one call into the library on the current (or the given) stream.  Losses return
their gradients with the loss.  With the default weights (a mean over rows)
and ``grad_scale=rows`` the gradients are per-row ones, the rows ``g`` that a
``KfacStack`` layer takes.  Argument marshalling only, as in the package: every
operator runs in the library's HIP kernels and there is no fallback.

One object is for one call at a time: calls on different streams or host
threads take objects of their own.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import (BF16, F32, KFAC_ERR_ARG, KFAC_ERR_DTYPE, KFAC_ERR_UNSUPPORTED, KFAC_OK, KfacError, load,
               read_flags)

I32, I64 = 0, 1
FLAG_BAD_INDEX = 4
OBJ_LOGP, OBJ_POLICY, OBJ_PREFERENCE, OBJ_BALANCE = range(4)
PREF_SIGMOID, PREF_SQUARED = 0, 1

EXPORTS = ("kfac_objective_workspace_size", "kfac_token_logp", "kfac_policy_loss", "kfac_preference_loss",
           "kfac_balance_loss", "kfac_dropout")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class TokenRows(ctypes.Structure):
    """Mirror of kfac_token_rows_t."""
    _fields_ = [("logits", _vp), ("labels", _vp), ("logp", _vp), ("grad", _vp), ("rows", _i64), ("ld", _i64),
                ("grad_ld", _i64), ("vocab", _i32), ("dtype", _i32), ("label_type", _i32), ("logit_scale", _f32),
                ("grad_scale", _f32), ("reserved", _i32)]


class Policy(ctypes.Structure):
    """Mirror of kfac_policy_t."""
    _fields_ = [("advantage", _vp), ("weight", _vp), ("old_logp", _vp), ("ref_logp", _vp), ("stats", _vp),
                ("clip_low", _f32), ("clip_high", _f32), ("kl_coef", _f32), ("reserved", _i32)]


class Preference(ctypes.Structure):
    """Mirror of kfac_preference_t."""
    _fields_ = [("offsets", _vp), ("ref_logp", _vp), ("pair_weight", _vp), ("seq", _vp), ("stats", _vp),
                ("pairs", _i32), ("kind", _i32), ("beta", _f32), ("label_smoothing", _f32), ("average", _i32),
                ("reserved", _i32)]


class Balance(ctypes.Structure):
    """Mirror of kfac_balance_t."""
    _fields_ = [("logits", _vp), ("chosen", _vp), ("mask", _vp), ("counts", _vp), ("prob", _vp), ("stats", _vp),
                ("grad", _vp), ("tokens", _i64), ("ld", _i64), ("grad_ld", _i64), ("experts", _i32), ("top_k", _i32),
                ("dtype", _i32), ("index_type", _i32), ("coef", _f32), ("z_coef", _f32), ("grad_scale", _f32),
                ("reserved", _i32)]


class DropoutArgs(ctypes.Structure):
    """Mirror of kfac_dropout_t."""
    _fields_ = [("x", _vp), ("residual", _vp), ("y", _vp), ("offset_dev", _vp), ("rows", _i64), ("cols", _i64),
                ("ld", _i64), ("residual_ld", _i64), ("y_ld", _i64), ("seed", ctypes.c_uint64),
                ("offset", ctypes.c_uint64), ("p", ctypes.c_double), ("dtype", _i32), ("reserved", _i32)]


_ready = None


def _library() -> ctypes.CDLL:
    """The library, with the argument types of this module's functions set."""
    global _ready
    if _ready is None:
        lib = load()
        sz = ctypes.c_size_t
        lib.kfac_objective_workspace_size.argtypes = [_i32, _i64, _i32, ctypes.POINTER(sz)]
        lib.kfac_token_logp.argtypes = [ctypes.POINTER(TokenRows), _vp, sz, _vp]
        lib.kfac_policy_loss.argtypes = [ctypes.POINTER(TokenRows), ctypes.POINTER(Policy), _vp, sz, _vp]
        lib.kfac_preference_loss.argtypes = [ctypes.POINTER(TokenRows), ctypes.POINTER(Preference), _vp, sz, _vp]
        lib.kfac_balance_loss.argtypes = [ctypes.POINTER(Balance), _vp, sz, _vp]
        lib.kfac_dropout.argtypes = [ctypes.POINTER(DropoutArgs), _vp]
        for name in EXPORTS:
            getattr(lib, name).restype = _i32
        _ready = lib
    return _ready


def workspace_size(objective: int, rows: int, groups: int = 0) -> int:
    """kfac_objective_workspace_size: groups = pairs (preference) or experts (balance)."""
    out = ctypes.c_size_t(0)
    st = _library().kfac_objective_workspace_size(objective, rows, groups, ctypes.byref(out))
    if st != KFAC_OK:
        raise KfacError(st, "kfac_objective_workspace_size")
    return out.value


_DTYPES = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}
_INDEX = {torch.int32: I32, torch.int64: I64}


class _Operator:
    """Shape, device and workspace shared by the operators."""

    def __init__(self, dtype: str, device, objective: Optional[int] = None, rows: int = 0, groups: int = 0):
        self._where = type(self).__name__
        if dtype not in _DTYPES:
            self._fail("dtype must be 'bf16' or 'f32'", KFAC_ERR_DTYPE)
        self.code, self.dt = _DTYPES[dtype]
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.dev = dev
        self.ws_ptr = self.ws_bytes = 0
        if objective is not None:
            self.ws_bytes = workspace_size(objective, rows, groups)
            self._ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=dev)
            self.ws_ptr = (self._ws.data_ptr() + 255) // 256 * 256
            if dev.type == "cuda":      # the workspace may be used on any stream from here on
                torch.cuda.current_stream(dev).synchronize()

    def _fail(self, what: str, status: int = KFAC_ERR_ARG):
        raise KfacError(status, f"{self._where}: {what}")

    def _matrix(self, t, name: str, rows: int, cols: int) -> int:
        """Checks [rows, cols] of the operator's dtype, columns adjacent; returns its row stride."""
        if t.dtype is not self.dt:
            self._fail(f"{name} must be {self.dt}", KFAC_ERR_DTYPE)
        if t.shape != (rows, cols) or t.device != self.dev:
            self._fail(f"{name} must be [{rows}, {cols}] on {self.dev}")
        ld, step = t.stride()
        if rows < 2:
            ld = cols
        if (step != 1 and cols > 1) or ld < cols:
            self._fail(f"{name} must have adjacent columns and rows that do not overlap")
        return ld

    def _vector(self, t, name: str, n: int, dtype=torch.float32) -> int:
        """Checks n contiguous values of `dtype`; returns their address."""
        if t.dtype is not dtype:
            self._fail(f"{name} must be {dtype}", KFAC_ERR_DTYPE)
        if t.numel() != n or t.device != self.dev or not t.is_contiguous():
            self._fail(f"{name} must be {n} contiguous values on {self.dev}")
        return t.data_ptr()

    def _indices(self, t, name: str, shape) -> int:
        """Checks contiguous int32 or int64 indices; returns their type code."""
        code = _INDEX.get(t.dtype)
        if code is None:
            self._fail(f"{name} must be int32 or int64", KFAC_ERR_DTYPE)
        if t.shape != shape or t.device != self.dev or not t.is_contiguous():
            self._fail(f"{name} must be {list(shape)}, contiguous, on {self.dev}")
        return code

    def _grad(self, x, ld: int, given):
        """The gradient tensor of logits x: `given`, or a new one whose rows lie as x's do."""
        if given is not None:
            return given, self._matrix(given, "grad", *x.shape)
        rows, cols = x.shape
        # the same place within 16 bytes for every row, at the least width
        per = 16 // x.element_size()
        width = cols + (ld - cols) % per
        if width == cols:
            return torch.empty(rows, cols, dtype=self.dt, device=self.dev), cols
        return torch.empty(rows, width, dtype=self.dt, device=self.dev)[:, :cols], width

    def _check(self, status: int, fn: str):
        if status != KFAC_OK:
            raise KfacError(status, fn)

    def flags(self, clear: bool = False) -> int:
        """The sticky flags (FLAG_NONFINITE, FLAG_BAD_INDEX); waits for the current stream."""
        return read_flags(self.ws_ptr, clear)

    def _stream(self, stream) -> int:
        if self.dev.type != "cuda":
            self._fail("the operators run on a GPU only", KFAC_ERR_UNSUPPORTED)
        if stream is None:
            return torch.cuda.current_stream(self.dev).cuda_stream
        return stream if isinstance(stream, int) else stream.cuda_stream


class _OnStream:
    """Output allocation on the stream that the call runs on (the caching allocator then knows their use)."""

    def __init__(self, stream, dev):
        self.ctx = None
        if stream is not None and dev.type == "cuda":
            s = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
            self.ctx = torch.cuda.stream(s)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


class _Tokens(_Operator):
    """Shape checks shared by the operators over rows of logits."""

    def __init__(self, rows, vocab, dtype, logit_scale, grad_scale, device, objective, groups=0):
        super().__init__(dtype, device, objective, rows, groups)
        if rows < 0 or vocab < 1:
            self._fail("rows must be at least 0 and vocab at least 1")
        if not 0.0 < logit_scale < float("inf"):
            self._fail("logit_scale must be positive and finite")
        self.rows, self.vocab = rows, vocab
        self._t = TokenRows(rows=rows, vocab=vocab, dtype=self.code, logit_scale=logit_scale, grad_scale=grad_scale)
        self._t_ref = ctypes.byref(self._t)

    def _take(self, logits, labels):
        t = self._t
        t.ld = self._matrix(logits, "logits", self.rows, self.vocab)
        t.label_type = self._indices(labels, "labels", (self.rows,))
        t.logits, t.labels = logits.data_ptr(), labels.data_ptr()

    def _logp(self):
        out = torch.empty(self.rows, dtype=torch.float32, device=self.dev)
        self._t.logp = out.data_ptr()
        return out


class TokenLogp(_Tokens):
    """logp[r] = s logits[r, labels[r]] - log sum_j exp(s logits[r, j]), 0 where the label is negative.

    dtype: "bf16" or "f32" (of the logits).  s = logit_scale (1 / temperature).
    """

    def __init__(self, rows: int, vocab: int, dtype: str = "bf16", logit_scale: float = 1.0, device="cuda"):
        super().__init__(rows, vocab, dtype, logit_scale, 1.0, device, OBJ_LOGP)

    def run(self, logits, labels, stream=None):
        """logits [rows, vocab] (any row stride), labels [rows] int32 or int64; returns logp [rows] float32."""
        self._take(logits, labels)
        with _OnStream(stream, self.dev):
            logp = self._logp()
        self._check(_library().kfac_token_logp(self._t_ref, self.ws_ptr, self.ws_bytes, self._stream(stream)),
                    "kfac_token_logp")
        return logp


class PolicyLoss(_Tokens):
    """Clipped policy loss with a KL term (kfac_policy_t gives the formulas).

    clip_low, clip_high: the ratio is held to [1 - clip_low, 1 + clip_high].
    kl_coef: factor of exp(d) - d - 1, d = ref_logp - logp.  grad_scale:
    factor of the gradients only.
    """

    def __init__(self, rows: int, vocab: int, dtype: str = "bf16", clip_low: float = 0.2, clip_high: float = 0.2,
                 kl_coef: float = 0.0, logit_scale: float = 1.0, grad_scale: float = 1.0, device="cuda"):
        super().__init__(rows, vocab, dtype, logit_scale, grad_scale, device, OBJ_POLICY)
        if not 0.0 <= clip_low <= 1.0 or not 0.0 <= clip_high < float("inf"):
            self._fail("clip_low must lie in [0, 1], clip_high must be at least 0 and finite")
        if not 0.0 <= kl_coef < float("inf"):
            self._fail("kl_coef must be at least 0 and finite")
        self._p = Policy(clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef)
        self._p_ref = ctypes.byref(self._p)
        self.kl_coef = kl_coef

    def run(self, logits, labels, advantage, weight=None, old_logp=None, ref_logp=None, grad=None, stream=None):
        """Returns (stats, logp, grad): stats [4] = loss, clipped term, KL term, clipped share (each
        weighted), logp [rows], grad [rows, vocab] of the logits' dtype.

        weight [rows] (default 1 / rows; 0 leaves a row out, as a negative
        label does), old_logp [rows] (default: the policy's own, ratio 1),
        ref_logp [rows] (needed where kl_coef > 0).  grad: where to write the
        gradient; it may be `logits` itself.
        """
        p, n = self._p, self.rows
        self._take(logits, labels)
        p.advantage = self._vector(advantage, "advantage", n)
        p.weight = None if weight is None else self._vector(weight, "weight", n)
        p.old_logp = None if old_logp is None else self._vector(old_logp, "old_logp", n)
        p.ref_logp = None if ref_logp is None else self._vector(ref_logp, "ref_logp", n)
        if ref_logp is None and self.kl_coef > 0.0:
            self._fail("kl_coef > 0 needs ref_logp")
        with _OnStream(stream, self.dev):
            logp = self._logp()
            stats = torch.empty(4, dtype=torch.float32, device=self.dev)
            grad, self._t.grad_ld = self._grad(logits, self._t.ld, grad)
        p.stats, self._t.grad = stats.data_ptr(), grad.data_ptr()
        self._check(_library().kfac_policy_loss(self._t_ref, self._p_ref, self.ws_ptr, self.ws_bytes,
                                                self._stream(stream)), "kfac_policy_loss")
        return stats, logp, grad


class PreferenceLoss(_Tokens):
    """Loss over pairs of sequences (kfac_preference_t gives the formulas).

    rows: tokens of all sequences; the `pairs` preferred sequences come
    first, then the rejected ones in the same order.  kind: "sigmoid" (with
    label_smoothing) or "squared".  average: log ratios are averaged over a
    sequence's labelled tokens rather than summed.
    """

    def __init__(self, rows: int, pairs: int, vocab: int, dtype: str = "bf16", beta: float = 0.1,
                 kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False, logit_scale: float = 1.0,
                 grad_scale: float = 1.0, device="cuda"):
        super().__init__(rows, vocab, dtype, logit_scale, grad_scale, device, OBJ_PREFERENCE, pairs)
        kinds = {"sigmoid": PREF_SIGMOID, "squared": PREF_SQUARED}
        if kind not in kinds:
            self._fail("kind must be 'sigmoid' or 'squared'")
        if not 0.0 < beta < float("inf"):
            self._fail("beta must be positive and finite")
        if not 0.0 <= label_smoothing < 0.5:
            self._fail("label_smoothing must lie in [0, 0.5)")
        self.pairs = pairs
        # the squared loss has no smoothing to apply
        smooth = label_smoothing if kind == "sigmoid" else 0.0
        self._p = Preference(pairs=pairs, kind=kinds[kind], beta=beta, label_smoothing=smooth, average=int(average))
        self._p_ref = ctypes.byref(self._p)

    def run(self, logits, labels, offsets, ref_logp=None, pair_weight=None, grad=None, stream=None):
        """Returns (stats, seq, logp, grad): stats [4] = loss, share of pairs in the right order, beta h,
        weights (sums over pairs), seq [2 pairs] the sequences' log ratios, logp [rows], grad [rows, vocab].

        offsets [2 pairs + 1] int32 on the GPU: sequence i holds rows
        offsets[i] .. offsets[i + 1] - 1.  ref_logp [rows] (default 0),
        pair_weight [pairs] (default 1 / pairs).
        """
        p = self._p
        self._take(logits, labels)
        p.offsets = self._vector(offsets, "offsets", 2 * self.pairs + 1, torch.int32)
        p.ref_logp = None if ref_logp is None else self._vector(ref_logp, "ref_logp", self.rows)
        p.pair_weight = None if pair_weight is None else self._vector(pair_weight, "pair_weight", self.pairs)
        with _OnStream(stream, self.dev):
            logp = self._logp()
            stats = torch.empty(4, dtype=torch.float32, device=self.dev)
            seq = torch.empty(2 * self.pairs, dtype=torch.float32, device=self.dev)
            grad, self._t.grad_ld = self._grad(logits, self._t.ld, grad)
        p.stats, p.seq, self._t.grad = stats.data_ptr(), seq.data_ptr(), grad.data_ptr()
        self._check(_library().kfac_preference_loss(self._t_ref, self._p_ref, self.ws_ptr, self.ws_bytes,
                                                    self._stream(stream)), "kfac_preference_loss")
        return stats, seq, logp, grad


class BalanceLoss(_Operator):
    """Router balance loss with per-expert counts (kfac_balance_t gives the formulas)."""

    def __init__(self, tokens: int, experts: int, top_k: int, dtype: str = "bf16", coef: float = 0.01,
                 z_coef: float = 0.0, grad_scale: float = 1.0, device="cuda"):
        super().__init__(dtype, device, OBJ_BALANCE, tokens, experts)
        if tokens < 0 or not 1 <= top_k <= experts:
            self._fail("tokens must be at least 0 and top_k between 1 and experts")
        self.tokens, self.experts, self.top_k = tokens, experts, top_k
        self._b = Balance(tokens=tokens, experts=experts, top_k=top_k, dtype=self.code, coef=coef, z_coef=z_coef,
                          grad_scale=grad_scale)
        self._b_ref = ctypes.byref(self._b)

    def run(self, logits, chosen, mask=None, grad=None, stream=None):
        """Returns (stats, counts, prob, grad): stats [4] = balance + z, balance, z, tokens counted;
        counts [experts] int32, prob [experts], grad [tokens, experts] of the logits' dtype.

        chosen [tokens, top_k] int32 or int64, negative for a dropped slot;
        mask [tokens] bool (default: all count).
        """
        b = self._b
        b.ld = self._matrix(logits, "logits", self.tokens, self.experts)
        b.index_type = self._indices(chosen, "chosen", (self.tokens, self.top_k))
        b.mask = None if mask is None else self._vector(mask, "mask", self.tokens, torch.bool)
        b.logits, b.chosen = logits.data_ptr(), chosen.data_ptr()
        with _OnStream(stream, self.dev):
            counts = torch.empty(self.experts, dtype=torch.int32, device=self.dev)
            prob = torch.empty(self.experts, dtype=torch.float32, device=self.dev)
            stats = torch.empty(4, dtype=torch.float32, device=self.dev)
            grad, b.grad_ld = self._grad(logits, b.ld, grad)
        b.counts, b.prob, b.stats, b.grad = counts.data_ptr(), prob.data_ptr(), stats.data_ptr(), grad.data_ptr()
        self._check(_library().kfac_balance_loss(self._b_ref, self.ws_ptr, self.ws_bytes, self._stream(stream)),
                    "kfac_balance_loss")
        return stats, counts, prob, grad


class Dropout(_Operator):
    """Dropout whose mask is a function of (seed, offset, position): kept with probability 1 - p, scaled
    by 1 / (1 - p) (p to 16 bits), nothing stored between forward and backward."""

    def __init__(self, rows: int, cols: int, dtype: str = "bf16", p: float = 0.1, device="cuda"):
        super().__init__(dtype, device)
        if rows < 0 or cols < 1:
            self._fail("rows must be at least 0 and cols at least 1")
        if not 0.0 <= p <= 1.0:
            self._fail("p must lie in [0, 1]")
        self.rows, self.cols = rows, cols
        self._d = DropoutArgs(rows=rows, cols=cols, p=p, dtype=self.code)
        self._d_ref = ctypes.byref(self._d)

    def run(self, x, seed: int, offset: int = 0, residual=None, out=None, offset_tensor=None, stream=None):
        """dropout(x) + residual, [rows, cols].

        seed, offset: 64-bit numbers that name the mask; a caller takes
        another offset for every layer and step.  offset_tensor: one int64 on
        the GPU, added to offset when the kernel runs (for captured graphs).
        out: where to write; it may be x or residual itself.
        """
        d = self._d
        d.ld = self._matrix(x, "x", self.rows, self.cols)
        d.x = x.data_ptr()
        if residual is None:
            d.residual = None
        else:
            d.residual_ld = self._matrix(residual, "residual", self.rows, self.cols)
            d.residual = residual.data_ptr()
        d.offset_dev = None if offset_tensor is None else self._vector(offset_tensor, "offset_tensor", 1, torch.int64)
        d.seed, d.offset = seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF
        if out is None:
            with _OnStream(stream, self.dev):
                out = torch.empty(self.rows, self.cols, dtype=self.dt, device=self.dev)
            d.y_ld = self.cols
        else:
            d.y_ld = self._matrix(out, "out", self.rows, self.cols)
        d.y = out.data_ptr()
        self._check(_library().kfac_dropout(self._d_ref, self._stream(stream)), "kfac_dropout")
        return out

    def backward(self, dy, seed: int, offset: int = 0, out=None, offset_tensor=None, stream=None):
        """d loss / dx from d loss / dy, with the mask of run(x, seed, offset); the residual's gradient is dy."""
        return self.run(dy, seed, offset, None, out, offset_tensor, stream)

    def flags(self, clear: bool = False) -> int:
        """Dropout has no workspace and raises no flags."""
        return 0
