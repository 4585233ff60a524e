"""The objectives' C ABI and binding on the host: exports, struct layout, and
every refusal, at the C entry points (well-formed addresses that are never
read) and at the Python classes (CPU tensors, which are never used)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import objectives as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kfac_objectives.h")
WS = 0x100000
STRUCTS = {"kfac_token_rows_t": Q.TokenRows, "kfac_policy_t": Q.Policy, "kfac_preference_t": Q.Preference,
           "kfac_balance_t": Q.Balance, "kfac_dropout_t": Q.DropoutArgs}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from second_order_optimizer_amd import build
        build.build()
    return Q._library()


def test_exports_every_declared_function(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(kfac_[a-z_]+)\s*\(", src))
    assert names == set(Q.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    lines, want = [], []
    for name, mirror in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(mirror))
        for f, _ in mirror._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(mirror, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void){",
                            *lines, "return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(c), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want


def test_workspace_sizes(lib):
    for obj, groups in ((Q.OBJ_LOGP, 0), (Q.OBJ_POLICY, 0), (Q.OBJ_PREFERENCE, 3), (Q.OBJ_BALANCE, 5)):
        for rows in (0, 1, 1000, 1 << 20):
            n = Q.workspace_size(obj, rows, groups)
            assert n >= 256 and n % 256 == 0
    for args, code in (((4, 1, 1), K.KFAC_ERR_ARG), ((0, -1, 0), K.KFAC_ERR_ARG), ((2, 1, 0), K.KFAC_ERR_ARG),
                       ((2, 1 << 31, 1), K.KFAC_ERR_UNSUPPORTED), ((3, 1, 0), K.KFAC_ERR_ARG),
                       ((3, 1, 1025), K.KFAC_ERR_UNSUPPORTED)):
        with pytest.raises(K.KfacError) as e:
            Q.workspace_size(*args)
        assert e.value.status == code, args


def rows(**over):
    v = dict(logits=0x10000, labels=0x20000, logp=0x30000, grad=0x40000, rows=4, ld=16, grad_ld=16, vocab=16,
             dtype=K.BF16, label_type=Q.I64, logit_scale=1.0, grad_scale=1.0, reserved=0)
    v.update(over)
    return Q.TokenRows(**v)


ROWS_BAD = [
    (dict(reserved=1), K.KFAC_ERR_ARG), (dict(dtype=2), K.KFAC_ERR_DTYPE), (dict(label_type=2), K.KFAC_ERR_DTYPE),
    (dict(rows=-1), K.KFAC_ERR_ARG), (dict(vocab=0), K.KFAC_ERR_ARG), (dict(ld=15), K.KFAC_ERR_ARG),
    (dict(logit_scale=0.0), K.KFAC_ERR_ARG), (dict(logit_scale=float("nan")), K.KFAC_ERR_ARG),
    (dict(logit_scale=float("inf")), K.KFAC_ERR_ARG), (dict(logits=None), K.KFAC_ERR_ARG),
    (dict(labels=None), K.KFAC_ERR_ARG), (dict(logp=None), K.KFAC_ERR_ARG), (dict(logits=0x10001), K.KFAC_ERR_ALIGN),
    (dict(labels=0x20004), K.KFAC_ERR_ALIGN), (dict(logp=0x30002), K.KFAC_ERR_ALIGN),
    (dict(rows=1 << 40, ld=1 << 40), K.KFAC_ERR_UNSUPPORTED),
]
GRAD_BAD = [
    (dict(grad=None), K.KFAC_ERR_ARG), (dict(grad=0x40001), K.KFAC_ERR_ALIGN), (dict(grad_ld=8), K.KFAC_ERR_ARG),
    (dict(grad_scale=float("inf")), K.KFAC_ERR_ARG), (dict(grad=0x10000, grad_ld=24), K.KFAC_ERR_ARG),
]


def call(fn, *structs, ws=WS, n=1 << 30):
    return fn(*[None if s is None else ctypes.byref(s) for s in structs], ws, n, None)


@pytest.mark.parametrize("bad,code", ROWS_BAD)
def test_rows_refusals(lib, bad, code):
    """Every refusal comes before any HIP call (a call that got through would give KFAC_ERR_HIP here)."""
    assert call(lib.kfac_token_logp, rows(**bad)) == code
    assert call(lib.kfac_policy_loss, rows(**bad), policy()) == code
    assert call(lib.kfac_preference_loss, rows(**bad), preference()) == code


@pytest.mark.parametrize("bad,code", GRAD_BAD)
def test_gradient_refusals(lib, bad, code):
    assert call(lib.kfac_policy_loss, rows(**bad), policy()) == code
    assert call(lib.kfac_preference_loss, rows(**bad), preference()) == code


def policy(**over):
    v = dict(advantage=0x50000, weight=0x51000, old_logp=0x52000, ref_logp=0x53000, stats=0x54000, clip_low=0.2,
             clip_high=0.2, kl_coef=0.1, reserved=0)
    v.update(over)
    return Q.Policy(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=3), K.KFAC_ERR_ARG), (dict(clip_low=1.5), K.KFAC_ERR_ARG), (dict(clip_low=-0.1), K.KFAC_ERR_ARG),
    (dict(clip_high=-0.1), K.KFAC_ERR_ARG), (dict(clip_high=float("inf")), K.KFAC_ERR_ARG),
    (dict(kl_coef=-1.0), K.KFAC_ERR_ARG), (dict(kl_coef=float("nan")), K.KFAC_ERR_ARG),
    (dict(ref_logp=None), K.KFAC_ERR_ARG), (dict(advantage=None), K.KFAC_ERR_ARG), (dict(stats=None), K.KFAC_ERR_ARG),
    (dict(weight=0x51002), K.KFAC_ERR_ALIGN), (dict(old_logp=0x51002), K.KFAC_ERR_ALIGN),
])
def test_policy_refusals(lib, bad, code):
    assert call(lib.kfac_policy_loss, rows(), policy(**bad)) == code


def preference(**over):
    v = dict(offsets=0x60000, ref_logp=0x61000, pair_weight=0x62000, seq=0x63000, stats=0x64000, pairs=2, kind=0,
             beta=0.1, label_smoothing=0.1, average=0, reserved=0)
    v.update(over)
    return Q.Preference(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=1), K.KFAC_ERR_ARG), (dict(pairs=0), K.KFAC_ERR_ARG), (dict(kind=2), K.KFAC_ERR_ARG),
    (dict(beta=0.0), K.KFAC_ERR_ARG), (dict(beta=float("inf")), K.KFAC_ERR_ARG),
    (dict(label_smoothing=0.5), K.KFAC_ERR_ARG), (dict(label_smoothing=-0.1), K.KFAC_ERR_ARG),
    (dict(kind=1), K.KFAC_ERR_ARG),                       # the squared loss takes no smoothing
    (dict(average=2), K.KFAC_ERR_ARG), (dict(offsets=None), K.KFAC_ERR_ARG), (dict(seq=None), K.KFAC_ERR_ARG),
    (dict(stats=None), K.KFAC_ERR_ARG), (dict(offsets=0x60002), K.KFAC_ERR_ALIGN),
])
def test_preference_refusals(lib, bad, code):
    assert call(lib.kfac_preference_loss, rows(), preference(**bad)) == code


def test_workspace_refusals(lib):
    for fn, args, need in ((lib.kfac_token_logp, (rows(),), Q.workspace_size(Q.OBJ_LOGP, 4)),
                           (lib.kfac_policy_loss, (rows(), policy()), Q.workspace_size(Q.OBJ_POLICY, 4)),
                           (lib.kfac_preference_loss, (rows(), preference()), Q.workspace_size(Q.OBJ_PREFERENCE, 4, 2)),
                           (lib.kfac_balance_loss, (balance(),), Q.workspace_size(Q.OBJ_BALANCE, 4, 8))):
        assert call(fn, *args, ws=None) == K.KFAC_ERR_WORKSPACE
        assert call(fn, *args, n=need - 1) == K.KFAC_ERR_WORKSPACE
        assert call(fn, *args, ws=WS + 16) == K.KFAC_ERR_ALIGN
        assert call(fn, *[None] * len(args)) == K.KFAC_ERR_ARG
    assert call(lib.kfac_policy_loss, rows(), None) == K.KFAC_ERR_ARG
    assert call(lib.kfac_preference_loss, rows(), None) == K.KFAC_ERR_ARG


def balance(**over):
    v = dict(logits=0x10000, chosen=0x20000, mask=0x21000, counts=0x22000, prob=0x23000, stats=0x24000, grad=0x30000,
             tokens=4, ld=8, grad_ld=8, experts=8, top_k=2, dtype=K.F32, index_type=Q.I32, coef=0.01, z_coef=0.0,
             grad_scale=1.0, reserved=0)
    v.update(over)
    return Q.Balance(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=1), K.KFAC_ERR_ARG), (dict(dtype=7), K.KFAC_ERR_DTYPE), (dict(index_type=-1), K.KFAC_ERR_DTYPE),
    (dict(tokens=-1), K.KFAC_ERR_ARG), (dict(experts=0), K.KFAC_ERR_ARG), (dict(top_k=0), K.KFAC_ERR_ARG),
    (dict(top_k=9), K.KFAC_ERR_ARG), (dict(experts=1025, ld=1025, grad_ld=1025), K.KFAC_ERR_UNSUPPORTED),
    (dict(ld=7), K.KFAC_ERR_ARG), (dict(grad_ld=7), K.KFAC_ERR_ARG), (dict(coef=float("nan")), K.KFAC_ERR_ARG),
    (dict(z_coef=float("inf")), K.KFAC_ERR_ARG), (dict(grad_scale=float("nan")), K.KFAC_ERR_ARG),
    (dict(tokens=1 << 31), K.KFAC_ERR_UNSUPPORTED), (dict(logits=None), K.KFAC_ERR_ARG),
    (dict(chosen=None), K.KFAC_ERR_ARG), (dict(grad=None), K.KFAC_ERR_ARG), (dict(counts=None), K.KFAC_ERR_ARG),
    (dict(prob=None), K.KFAC_ERR_ARG), (dict(stats=None), K.KFAC_ERR_ARG), (dict(logits=0x10002), K.KFAC_ERR_ALIGN),
    (dict(grad=0x10000, grad_ld=9), K.KFAC_ERR_ARG),
])
def test_balance_refusals(lib, bad, code):
    assert call(lib.kfac_balance_loss, balance(**bad)) == code


def dropout(**over):
    v = dict(x=0x10000, residual=0x20000, y=0x30000, offset_dev=None, rows=4, cols=16, ld=16, residual_ld=16, y_ld=16,
             seed=1, offset=0, p=0.1, dtype=K.F32, reserved=0)
    v.update(over)
    return Q.DropoutArgs(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=1), K.KFAC_ERR_ARG), (dict(dtype=3), K.KFAC_ERR_DTYPE), (dict(rows=-1), K.KFAC_ERR_ARG),
    (dict(cols=0), K.KFAC_ERR_ARG), (dict(ld=15), K.KFAC_ERR_ARG), (dict(y_ld=15), K.KFAC_ERR_ARG),
    (dict(residual_ld=15), K.KFAC_ERR_ARG), (dict(p=-0.1), K.KFAC_ERR_ARG), (dict(p=1.1), K.KFAC_ERR_ARG),
    (dict(p=float("nan")), K.KFAC_ERR_ARG), (dict(x=None), K.KFAC_ERR_ARG), (dict(y=None), K.KFAC_ERR_ARG),
    (dict(x=0x10002), K.KFAC_ERR_ALIGN), (dict(offset_dev=0x10004), K.KFAC_ERR_ALIGN),
    (dict(y=0x10000, y_ld=17), K.KFAC_ERR_ARG), (dict(y=0x20000, residual_ld=17), K.KFAC_ERR_ARG),
    (dict(rows=1 << 39, cols=1 << 20, ld=1 << 20, residual_ld=1 << 20, y_ld=1 << 20), K.KFAC_ERR_UNSUPPORTED),
])
def test_dropout_refusals(lib, bad, code):
    d = dropout(**bad)
    assert lib.kfac_dropout(ctypes.byref(d), None) == code
    assert lib.kfac_dropout(None, None) == K.KFAC_ERR_ARG


def test_dropout_past_one_launch_is_refused(lib):
    """More than 2^32 - 1024 generator blocks (2^35 elements) do not fit a launch's count of threads."""
    for r, cols in ((1 << 32, 8), (1 << 20, 1 << 15), (1, 1 << 36), ((1 << 32) - 1023, 1)):
        d = dropout(rows=r, cols=cols, ld=cols, residual_ld=cols, y_ld=cols)
        assert lib.kfac_dropout(ctypes.byref(d), None) == K.KFAC_ERR_UNSUPPORTED, (r, cols)


def test_dropout_of_nothing(lib):
    """No rows: nothing to do, no pointers needed, no launch."""
    d = dropout(rows=0, x=None, y=None, residual=None)
    assert lib.kfac_dropout(ctypes.byref(d), None) == K.KFAC_OK


# -- the Python classes: tensors on the CPU reach every check and are refused at the end --------

def refused(status, fn, *a, **kw):
    with pytest.raises(K.KfacError) as e:
        fn(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_constructor_refusals(lib):
    A, D = K.KFAC_ERR_ARG, K.KFAC_ERR_DTYPE
    cpu = dict(device="cpu")
    refused(D, Q.TokenLogp, 4, 8, dtype="f64", **cpu)
    refused(A, Q.TokenLogp, -1, 8, **cpu)
    refused(A, Q.TokenLogp, 4, 0, **cpu)
    refused(A, Q.TokenLogp, 4, 8, logit_scale=0.0, **cpu)
    refused(A, Q.PolicyLoss, 4, 8, clip_low=1.5, **cpu)
    refused(A, Q.PolicyLoss, 4, 8, clip_high=-1.0, **cpu)
    refused(A, Q.PolicyLoss, 4, 8, kl_coef=-1.0, **cpu)
    refused(A, Q.PreferenceLoss, 4, 0, 8, **cpu)
    refused(A, Q.PreferenceLoss, 4, 1, 8, kind="cubic", **cpu)
    refused(A, Q.PreferenceLoss, 4, 1, 8, beta=0.0, **cpu)
    refused(A, Q.PreferenceLoss, 4, 1, 8, label_smoothing=0.5, **cpu)
    refused(A, Q.BalanceLoss, 4, 8, 9, **cpu)
    refused(A, Q.BalanceLoss, 4, 8, 0, **cpu)
    refused(K.KFAC_ERR_UNSUPPORTED, Q.BalanceLoss, 4, 2000, 2, **cpu)
    refused(A, Q.Dropout, 4, 8, p=1.5, **cpu)
    refused(A, Q.Dropout, 4, 0, **cpu)


def test_run_refusals(lib):
    A, D, U = K.KFAC_ERR_ARG, K.KFAC_ERR_DTYPE, K.KFAC_ERR_UNSUPPORTED
    x, lab, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    op = Q.TokenLogp(4, 8, dtype="f32", device="cpu")
    refused(U, op.run, x, lab)                                  # valid, but not on a GPU
    refused(D, op.run, x.bfloat16(), lab)
    refused(D, op.run, x, lab.short())
    refused(A, op.run, torch.zeros(4, 9), lab)
    refused(A, op.run, torch.zeros(8, 4).t(), lab)              # columns not adjacent
    refused(A, op.run, torch.zeros(1, 8).expand(4, 8), lab)     # rows on top of each other
    refused(A, op.run, x, torch.zeros(5, dtype=torch.int64))
    refused(A, op.run, x, torch.zeros(8, dtype=torch.int64)[::2])
    pol = Q.PolicyLoss(4, 8, dtype="f32", kl_coef=0.1, device="cpu")
    refused(U, pol.run, x, lab, f, ref_logp=f)
    refused(A, pol.run, x, lab, f)                              # a KL term without a reference
    refused(D, pol.run, x, lab, f.double(), ref_logp=f)
    refused(A, pol.run, x, lab, torch.zeros(3), ref_logp=f)
    refused(A, pol.run, x, lab, f, weight=torch.zeros(8)[::2], ref_logp=f)
    refused(A, pol.run, x, lab, f, ref_logp=f, grad=torch.zeros(4, 9))
    refused(D, pol.run, x, lab, f, ref_logp=f, grad=x.bfloat16())
    pre = Q.PreferenceLoss(4, 1, 8, dtype="f32", device="cpu")
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    refused(U, pre.run, x, lab, off)
    refused(D, pre.run, x, lab, off.long())
    refused(A, pre.run, x, lab, off[:2])
    refused(A, pre.run, x, lab, off, pair_weight=f)
    bal = Q.BalanceLoss(4, 8, 2, dtype="f32", device="cpu")
    ids = torch.zeros(4, 2, dtype=torch.int32)
    refused(U, bal.run, x, ids)
    refused(A, bal.run, x, ids[:, :1])
    refused(D, bal.run, x, ids.short())
    refused(D, bal.run, x, ids, mask=torch.zeros(4, dtype=torch.uint8))
    drop = Q.Dropout(4, 8, dtype="f32", device="cpu")
    refused(U, drop.run, x, 1)
    refused(A, drop.run, torch.zeros(4, 7), 1)
    refused(D, drop.run, x, 1, residual=x.bfloat16())
    refused(D, drop.run, x, 1, offset_tensor=off[:1])
    refused(A, drop.backward, x, 1, out=torch.zeros(4, 16)[:, ::2])


def test_calls_that_are_not_tensors(lib):
    """Anything but a tensor, and numbers that are not whole, are refused without a crash."""
    x, lab = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    op = Q.TokenLogp(4, 8, dtype="f32", device="cpu")
    refused(K.KFAC_ERR_ARG, op.run, None, lab)
    refused(K.KFAC_ERR_ARG, op.run, [1.0], lab)
    refused(K.KFAC_ERR_ARG, op.run, x, "labels")
    refused(K.KFAC_ERR_ARG, op.run, x.to_sparse(), lab)
    drop = Q.Dropout(4, 8, dtype="f32", device="cpu")
    with pytest.raises(TypeError):
        drop.run(x, 1.5)
    with pytest.raises(TypeError):
        drop.run(x, 1, offset="two")
    refused(K.KFAC_ERR_UNSUPPORTED, drop.run, x, -1, offset=1 << 70)      # taken modulo 2^64
