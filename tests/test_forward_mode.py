"""Operators inside autograd have backward passes only: a tensor with a forward-mode tangent is refused, as a result
without one would stand for a derivative of zero."""
import os

import pytest
import torch
from torch.autograd import forward_ad as F

import second_order_optimizer_amd as K
from second_order_optimizer_amd import objectives as O
from second_order_optimizer_amd import tokens as T


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(K.LIB_PATH):
        from second_order_optimizer_amd import build
        build.build()


def refused(what, fn, *a, **kw):
    """What a valid call on the CPU gives is the same status for another reason."""
    with pytest.raises(K.KfacError) as e:
        fn(*a, **kw)
    assert e.value.status == K.KFAC_ERR_UNSUPPORTED and what in str(e.value), str(e.value)


def dual(*shape):
    return F.make_dual(torch.zeros(*shape), torch.ones(*shape))


def test_embedding():
    op = T.Embedding(4, 8, 16, dtype="f32", device="cpu")
    table, ids, dy = torch.zeros(8, 16), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 16)
    refused("GPU only", op.run, table, ids)
    with F.dual_level():
        refused("tangent", op.run, dual(8, 16), ids)
        refused("tangent", op.run, F.make_dual(torch.zeros(8, 16, requires_grad=True), torch.ones(8, 16)), ids)
        refused("tangent", op.run, table, ids, out=dual(4, 16))
        refused("tangent", op.backward, dual(4, 16), ids)
        refused("tangent", op.backward, dy, ids, grad=dual(8, 16), accumulate=True)
        refused("GPU only", op.run, table, ids)
        refused("GPU only", op.run, F.unpack_dual(dual(8, 16)).primal, ids)
        with F._set_fwd_grad_enabled(False):
            refused("GPU only", op.run, dual(8, 16), ids)
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: op.run(t, ids), (table,), (table,))


def test_dropout():
    op = O.Dropout(4, 16, dtype="f32", p=0.5, device="cpu")
    x = torch.zeros(4, 16)
    refused("GPU only", op.run, x, 1, residual=x)
    with F.dual_level():
        refused("tangent", op.run, dual(4, 16), 1)
        refused("tangent", op.run, F.make_dual(torch.zeros(4, 16, requires_grad=True), torch.ones(4, 16)), 1)
        refused("tangent", op.run, x, 1, residual=dual(4, 16))
        refused("tangent", op.run, x, 1, out=dual(4, 16))
        refused("tangent", op.backward, dual(4, 16), 1)
        refused("GPU only", op.run, x, 1, residual=x)
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: op.run(t, 1), (x,), (x,))
