"""Further refusals of the objectives, on the host: what belongs to autograd, and sizes past one launch."""
import ctypes

import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import objectives as Q


def test_dropout_refuses_out_where_a_gradient_is_wanted():
    """It would cut the graph, or leave the dropout out of it."""
    op = Q.Dropout(4, 8, dtype="f32", device="cpu")
    x, g = torch.zeros(4, 8), torch.zeros(4, 8, requires_grad=True)
    for kw in (dict(x=g), dict(x=x, residual=g)):
        for out in (torch.zeros(4, 8), g):
            with pytest.raises(K.KfacError) as e:
                op.run(seed=1, out=out, **kw)
            assert e.value.status == K.KFAC_ERR_ARG
            with torch.no_grad(), pytest.raises(K.KfacError) as e:
                op.run(seed=1, out=out, **kw)
            assert e.value.status == K.KFAC_ERR_UNSUPPORTED        # as far as a GPU is needed


def test_pairs_past_one_launch_are_refused():
    """A workgroup of 1024 threads a pair: from 2^22 pairs a launch has more than 2^32 - 1 threads, and would fail
    after the log-probabilities were enqueued."""
    lib = Q._library()
    rows = Q.TokenRows(logits=0x10000, labels=0x20000, logp=0x30000, grad=0x40000, rows=4, ld=16, grad_ld=16, vocab=16,
                       dtype=K.BF16, label_type=Q.I64, logit_scale=1.0, grad_scale=1.0)
    for pairs in (1 << 22, (1 << 22) + 1, (1 << 30) - 1, 1 << 30):
        with pytest.raises(K.KfacError) as e:
            Q.workspace_size(Q.OBJ_PREFERENCE, 4, pairs)
        assert e.value.status == K.KFAC_ERR_UNSUPPORTED, pairs
        pref = Q.Preference(offsets=0x60000, seq=0x63000, stats=0x64000, pairs=pairs, beta=0.1)
        st = lib.kfac_preference_loss(ctypes.byref(rows), ctypes.byref(pref), 0x100000, 1 << 40, None)
        assert st == K.KFAC_ERR_UNSUPPORTED, pairs
    assert Q.workspace_size(Q.OBJ_PREFERENCE, 4, (1 << 22) - 1) > 1 << 27


def test_flags_are_read_on_the_objects_device(monkeypatch):
    """The stream that flags() waits for is the current one of the operator's GPU, not of the current GPU."""
    op = Q.PolicyLoss(4, 8, dtype="f32", device="cpu")
    op.dev = torch.device("cuda", 1)
    here, seen = [0], []

    class On:
        def __init__(self, dev):
            self.dev = torch.device(dev).index

        def __enter__(self):
            self.before, here[0] = here[0], self.dev

        def __exit__(self, *exc):
            here[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(Q, "read_flags", lambda ws, clear=False, stream=None: seen.append((here[0], ws, clear)) or 2)
    assert op.flags(clear=True) == 2
    assert seen == [(1, op.ws_ptr, True)] and here == [0]
