"""Calls of the embedding and the orthogonalised update that their documentation allows or rules out, on the host."""
import os

import numpy as np
import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import orthogonal as M
from second_order_optimizer_amd import tokens as T

A, U = K.KFAC_ERR_ARG, K.KFAC_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(K.LIB_PATH):
        from second_order_optimizer_amd import build
        build.build()
    M._library()
    return T._library()


def refused(status, fn, *a, **kw):
    """(A valid call on the CPU is refused as unsupported.)"""
    with pytest.raises(K.KfacError) as e:
        fn(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_accumulate_is_any_truth_value():
    op = T.Embedding(4, 8, 16, dtype="f32", device="cpu")
    dy, ids = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    for yes in (True, 1, np.True_, torch.tensor(True)):
        refused(A, op.backward, dy, ids, accumulate=yes)             # there is no gradient to add to
        refused(U, op.backward, dy, ids, grad=torch.zeros(8, 16), accumulate=yes)
    for no in (False, 0, None, np.False_):
        refused(U, op.backward, dy, ids, accumulate=no)
    with pytest.raises(RuntimeError):
        op.backward(dy, ids, grad=torch.zeros(8, 16), accumulate=torch.zeros(2))


@pytest.mark.gpu
def test_accumulate_by_a_number(gpu_lib):
    op = T.Embedding(4, 8, 16, dtype="f32")
    dy, ids = torch.ones(4, 16, device="cuda"), torch.tensor([1, 1, 3, -1], device="cuda")
    for yes in (1, np.True_):
        grad = torch.full((8, 16), 5.0, device="cuda")
        op.backward(dy, ids, grad=grad, accumulate=yes)
        assert grad[:, 0].tolist() == [5, 7, 5, 6, 5, 5, 5, 5]
