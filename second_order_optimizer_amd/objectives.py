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
their gradients with the loss; these and the log-probabilities are outside
autograd (``logits.backward(grad)`` hands a gradient on), dropout is inside.
With the default weights (a mean over rows) and ``grad_scale=rows`` the
gradients are per-row ones, the rows ``g`` that a ``KfacStack`` layer takes.
They are contiguous there: give the layer's buffer as ``grad``, or copy (a new
gradient has the logits' row stride modulo 16 bytes).  Argument marshalling
only, as in the package: every operator runs in the library's HIP kernels and
there is no fallback.  The marshalling of a call is native (csrc/binding.cpp,
the ``_objectives`` extension).

One object is for one call at a time: calls on different streams or host
threads take objects of their own.  Its shape is fixed, and making one
allocates and synchronises: keep one per shape.  A graph that captured its
calls works in its workspace: keep the object as long as the graph.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import BF16, F32, KFAC_ERR_ARG, KFAC_ERR_DTYPE, KFAC_OK, KfacError, load, read_flags

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


class _Plan(ctypes.Structure):
    """Mirror of csrc/binding.cpp's Plan: workspace, its tensor and stream, device (-1: not a GPU), dtype."""
    _fields_ = [("ws", _vp), ("ws_bytes", ctypes.c_size_t), ("ws_tensor", _vp), ("home", _vp),
                ("name", ctypes.c_char_p), ("device", _i32), ("dtype", _i32)]


class _TokenPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("t", TokenRows)]


class _PolicyPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("t", TokenRows), ("p", Policy)]


class _PreferencePlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("t", TokenRows), ("p", Preference)]


class _BalancePlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("b", Balance)]


class _DropoutPlan(ctypes.Structure):
    _fields_ = [("base", _Plan), ("d", DropoutArgs)]


_lib = None
_native = None


def _library() -> ctypes.CDLL:
    """The library with the argument types of this module's functions set, bound to the extension."""
    global _lib, _native
    if _lib is not None:
        return _lib
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
    try:
        from . import _objectives
    except ModuleNotFoundError as e:
        raise FileNotFoundError(f"{os.path.join(os.path.dirname(__file__), '_objectives.so')} is missing: build it "
                                "with `python -m second_order_optimizer_amd.build`") from e
    plans = (_TokenPlan, _PolicyPlan, _PreferencePlan, _BalancePlan, _DropoutPlan)
    if _objectives.plan_sizes() != tuple(ctypes.sizeof(p) for p in plans):
        raise RuntimeError("the _objectives extension is of another build than this package")
    _objectives.bind(KfacError, *[ctypes.cast(getattr(lib, name), _vp).value for name in EXPORTS[1:]])
    _lib, _native = lib, _objectives
    return lib


def workspace_size(objective: int, rows: int, groups: int = 0) -> int:
    """kfac_objective_workspace_size: groups = pairs (preference) or experts (balance)."""
    out = ctypes.c_size_t(0)
    st = _library().kfac_objective_workspace_size(objective, rows, groups, ctypes.byref(out))
    if st != KFAC_OK:
        raise KfacError(st, "kfac_objective_workspace_size")
    return out.value


_DTYPES = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}


class _Operator:
    """Shape, device and workspace shared by the operators."""

    def __init__(self, plan, dtype: str, device, objective: Optional[int] = None, rows: int = 0, groups: int = 0,
                 ws_bytes: Optional[int] = None):
        self._where = type(self).__name__
        if dtype not in _DTYPES:
            self._fail("dtype must be 'bf16' or 'f32'", KFAC_ERR_DTYPE)
        _library()
        self.code, self.dt = _DTYPES[dtype]
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.dev = dev
        self.ws_ptr = self.ws_bytes = 0
        tensor = home = None
        if objective is not None:
            ws_bytes = workspace_size(objective, rows, groups)
        if ws_bytes is not None:
            self.ws_bytes = ws_bytes
            self._ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=dev)
            self.ws_ptr = (self._ws.data_ptr() + 255) // 256 * 256
            if dev.type == "cuda":      # the workspace may be used on any stream from here on
                here = torch.cuda.current_stream(dev)
                here.synchronize()
                tensor, home = id(self._ws), here.cuda_stream
        self._plan = plan
        self._name = self._where.encode()
        plan.base = _Plan(self.ws_ptr, self.ws_bytes, tensor, home, self._name,
                          dev.index if dev.type == "cuda" else -1, self.code)
        self._at = ctypes.addressof(plan)

    def _fail(self, what: str, status: int = KFAC_ERR_ARG):
        raise KfacError(status, f"{self._where}: {what}")

    def _on(self, stream, call, *args):
        """The call on `stream` (a torch stream or a handle), its outputs allocated there."""
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.dev)
        with torch.cuda.stream(stream):
            return call(self._at, *args)

    def flags(self, clear: bool = False) -> int:
        """The sticky flags (FLAG_NONFINITE, FLAG_BAD_INDEX); waits for the current stream of the operator's
        GPU (a call that was given another stream has to be waited for by the caller)."""
        with torch.cuda.device(self.dev):
            return read_flags(self.ws_ptr, clear)


class _Tokens(_Operator):
    """Shape checks shared by the operators over rows of logits."""

    def __init__(self, plan, rows, vocab, dtype, logit_scale, grad_scale, device, objective, groups=0):
        super().__init__(plan, dtype, device, objective, rows, groups)
        if rows < 0 or vocab < 1:
            self._fail("rows must be at least 0 and vocab at least 1")
        if not 0.0 < logit_scale < float("inf"):
            self._fail("logit_scale must be positive and finite")
        self.rows, self.vocab = rows, vocab
        plan.t = TokenRows(rows=rows, vocab=vocab, dtype=self.code, logit_scale=logit_scale, grad_scale=grad_scale)


class TokenLogp(_Tokens):
    """logp[r] = s logits[r, labels[r]] - log sum_j exp(s logits[r, j]), 0 where the label is negative.

    dtype: "bf16" or "f32" (of the logits).  s = logit_scale (1 / temperature).
    """

    def __init__(self, rows: int, vocab: int, dtype: str = "bf16", logit_scale: float = 1.0, device="cuda"):
        super().__init__(_TokenPlan(), rows, vocab, dtype, logit_scale, 1.0, device, OBJ_LOGP)

    def run(self, logits, labels, stream=None):
        """logits [rows, vocab] (any row stride), labels [rows] int32 or int64; returns logp [rows] float32."""
        if stream is None:
            return _native.token_logp(self._at, logits, labels)
        return self._on(stream, _native.token_logp, logits, labels)


class PolicyLoss(_Tokens):
    """Clipped policy loss with a KL term (kfac_policy_t gives the formulas).

    clip_low, clip_high: the ratio is held to [1 - clip_low, 1 + clip_high].
    kl_coef: factor of exp(d) - d - 1, d = ref_logp - logp.  grad_scale:
    factor of the gradients only.
    """

    def __init__(self, rows: int, vocab: int, dtype: str = "bf16", clip_low: float = 0.2, clip_high: float = 0.2,
                 kl_coef: float = 0.0, logit_scale: float = 1.0, grad_scale: float = 1.0, device="cuda"):
        super().__init__(_PolicyPlan(), rows, vocab, dtype, logit_scale, grad_scale, device, OBJ_POLICY)
        if not 0.0 <= clip_low <= 1.0 or not 0.0 <= clip_high < float("inf"):
            self._fail("clip_low must lie in [0, 1], clip_high must be at least 0 and finite")
        if not 0.0 <= kl_coef < float("inf"):
            self._fail("kl_coef must be at least 0 and finite")
        self._plan.p = Policy(clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef)

    def run(self, logits, labels, advantage, weight=None, old_logp=None, ref_logp=None, grad=None, stream=None):
        """Returns (stats, logp, grad): stats [4] = loss, clipped term, KL term, clipped share (each
        weighted), logp [rows], grad [rows, vocab] of the logits' dtype.

        weight [rows] (default 1 / rows; 0 leaves a row out, as a negative
        label does), old_logp [rows] (default: the policy's own, ratio 1),
        ref_logp [rows] (needed where kl_coef > 0).  grad: where to write the
        gradient; it may be `logits` itself.
        """
        if stream is None:
            return _native.policy_loss(self._at, logits, labels, advantage, weight, old_logp, ref_logp, grad)
        return self._on(stream, _native.policy_loss, logits, labels, advantage, weight, old_logp, ref_logp, grad)


class PreferenceLoss(_Tokens):
    """Loss over pairs of sequences (kfac_preference_t gives the formulas).

    rows: tokens of all sequences; the `pairs` preferred sequences come
    first, then the rejected ones in the same order.  kind: "sigmoid" (with
    label_smoothing) or "squared" (which has none, whatever is given).
    average: log ratios are averaged over a sequence's labelled tokens rather
    than summed.
    """

    def __init__(self, rows: int, pairs: int, vocab: int, dtype: str = "bf16", beta: float = 0.1,
                 kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False, logit_scale: float = 1.0,
                 grad_scale: float = 1.0, device="cuda"):
        super().__init__(_PreferencePlan(), rows, vocab, dtype, logit_scale, grad_scale, device, OBJ_PREFERENCE, pairs)
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
        self._plan.p = Preference(pairs=pairs, kind=kinds[kind], beta=beta, label_smoothing=smooth,
                                  average=int(average))

    def run(self, logits, labels, offsets, ref_logp=None, pair_weight=None, grad=None, stream=None):
        """Returns (stats, seq, logp, grad): stats [4] = loss, share of pairs in the right order, beta h,
        weights (sums over pairs), seq [2 pairs] the sequences' log ratios, logp [rows], grad [rows, vocab].

        offsets [2 pairs + 1] int32 on the GPU: sequence i holds rows
        offsets[i] .. offsets[i + 1] - 1.  ref_logp [rows] (default 0),
        pair_weight [pairs] (default 1 / pairs).
        """
        if stream is None:
            return _native.preference_loss(self._at, logits, labels, offsets, ref_logp, pair_weight, grad)
        return self._on(stream, _native.preference_loss, logits, labels, offsets, ref_logp, pair_weight, grad)


class BalanceLoss(_Operator):
    """Router balance loss with per-expert counts (kfac_balance_t gives the formulas)."""

    def __init__(self, tokens: int, experts: int, top_k: int, dtype: str = "bf16", coef: float = 0.01,
                 z_coef: float = 0.0, grad_scale: float = 1.0, device="cuda"):
        super().__init__(_BalancePlan(), dtype, device, OBJ_BALANCE, tokens, experts)
        if tokens < 0 or not 1 <= top_k <= experts:
            self._fail("tokens must be at least 0 and top_k between 1 and experts")
        self.tokens, self.experts, self.top_k = tokens, experts, top_k
        self._plan.b = Balance(tokens=tokens, experts=experts, top_k=top_k, dtype=self.code, coef=coef, z_coef=z_coef,
                               grad_scale=grad_scale)

    def run(self, logits, chosen, mask=None, grad=None, stream=None):
        """Returns (stats, counts, prob, grad): stats [4] = balance + z, balance, z, tokens counted;
        counts [experts] int32, prob [experts], grad [tokens, experts] of the logits' dtype.

        chosen [tokens, top_k] int32 or int64, negative for a dropped slot;
        mask [tokens] bool (default: all count).
        """
        if stream is None:
            return _native.balance_loss(self._at, logits, chosen, mask, grad)
        return self._on(stream, _native.balance_loss, logits, chosen, mask, grad)


class _DropoutNode(torch.autograd.Function):
    """Dropout's place in autograd: the backward pass is the same call on the output gradient."""

    @staticmethod
    def forward(ctx, x, residual, op, seed, offset, offset_tensor, stream):
        y = op.run(x, seed, offset, residual, None, offset_tensor, stream)
        ctx.call = op, seed, offset
        ctx.save_for_backward(offset_tensor)
        return y

    @staticmethod
    def backward(ctx, dy):
        op, seed, offset = ctx.call
        offset_tensor, = ctx.saved_tensors
        dx = op.backward(dy.contiguous(), seed, offset, None, offset_tensor) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None, None, None


class Dropout(_Operator):
    """Dropout whose mask is a function of (seed, offset, position): kept with probability 1 - p, scaled
    by 1 / (1 - p) (p to 16 bits), nothing stored between forward and backward.  Where x or residual
    requires grad, the result is part of autograd's graph; tensors with a forward-mode tangent are refused."""

    def __init__(self, rows: int, cols: int, dtype: str = "bf16", p: float = 0.1, device="cuda"):
        super().__init__(_DropoutPlan(), dtype, device)
        if rows < 0 or cols < 1:
            self._fail("rows must be at least 0 and cols at least 1")
        if not 0.0 <= p <= 1.0:
            self._fail("p must lie in [0, 1]")
        self.rows, self.cols = rows, cols
        self._plan.d = DropoutArgs(rows=rows, cols=cols, p=p, dtype=self.code)

    def run(self, x, seed: int, offset: int = 0, residual=None, out=None, offset_tensor=None, stream=None):
        """dropout(x) + residual, [rows, cols].

        seed, offset: 64-bit numbers that name the mask; a caller takes
        another offset for every layer and step.  offset_tensor: one int64 on
        the GPU, added to offset when the kernel runs (for captured graphs).
        out: where to write; it may be x or residual itself.  It is for
        calls outside autograd: refused where x or residual requires grad.
        """
        if stream is None:
            y = _native.dropout(self._at, x, seed, offset, residual, out, offset_tensor)
        else:
            y = self._on(stream, _native.dropout, x, seed, offset, residual, out, offset_tensor)
        if y is None:           # x or residual requires grad, and autograd is on
            return _DropoutNode.apply(x, residual, self, seed, offset, offset_tensor, stream)
        return y

    def backward(self, dy, seed: int, offset: int = 0, out=None, offset_tensor=None, stream=None):
        """d loss / dx from d loss / dy, with the mask of run(x, seed, offset); the residual's gradient is dy."""
        return self.run(dy, seed, offset, None, out, offset_tensor, stream)

    def flags(self, clear: bool = False) -> int:
        """Dropout has no workspace and raises no flags."""
        return 0
