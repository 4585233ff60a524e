"""What memory an orthogonalised step works on."""
import os

import numpy as np
import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import orthogonal as M

A, U = K.KFAC_ERR_ARG, K.KFAC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from second_order_optimizer_amd import build
        build.build()
    return M._library()


def refused(status, fn, *a, **kw):
    with pytest.raises(K.KfacError) as e:
        fn(*a, **kw)
    assert e.value.status == status, str(e.value)


def layers(device="cpu"):
    f = lambda *s: torch.randn(*s, device=device)  # noqa: E731
    w, m, g = ([f(4, 8), f(6, 5), f(3, 3)] for _ in range(3))
    b, bm, bg = ([f(4), None, f(3)] for _ in range(3))
    return w, m, b, bm, g, bg


def test_tensors_that_were_given_other_memory(lib):
    """Each call takes the memory that the tensors have then; one that has no longer the layer's shape is refused."""
    w, m, b, bm, g, bg = layers()
    s = M.OrthogonalStep(w, m, b, bm)
    for t in (w[0], w[2], m[1], b[2], bm[0]):
        t.data = torch.randn_like(t)
    flat = torch.randn(30)
    w[1].data = flat.view(6, 5)
    refused(U, s.run, g, bg)                    # valid, but not on a GPU
    for i, L in enumerate(s._layers):
        assert (L.w, L.mom_w) == (w[i].data_ptr(), m[i].data_ptr())
        if b[i] is not None:
            assert (L.b, L.mom_b) == (b[i].data_ptr(), bm[i].data_ptr())
    for t, other in ((w[0], torch.zeros(8, 4)), (w[0], torch.zeros(8, 4).t()), (m[1], torch.zeros(5)), (b[2], torch.zeros(4)),
                     (bm[0], torch.zeros(8)[::2])):
        was = t.data
        t.data = other
        refused(A, s.run, g, bg)
        t.data = was
    refused(U, s.run, g, bg)


@pytest.mark.gpu
def test_step_of_weights_that_moved(gpu_lib):
    """The step after `w.data = v` writes v, as a step of tensors that were there from the start."""
    w, m, b, bm, g, bg = layers("cuda")
    copy = lambda v: [None if t is None else t.clone() for t in v]  # noqa: E731
    start = [copy(v) for v in (w, m, b, bm)]
    s = M.OrthogonalStep(w, m, b, bm)
    s.run(g, bg)
    old = [t.data for v in (w, m, b, bm) for t in v if t is not None]
    was = [t.clone() for t in old]
    for now, v in zip((w, m, b, bm), start):
        for t, u in zip(now, v):
            if t is not None:
                t.data = u.clone()
    other = M.OrthogonalStep(*start)
    for _ in range(2):
        s.run(g, bg)
        other.run(g, bg)
    torch.cuda.synchronize()
    for now, v in zip((w, m, b, bm), start):
        for t, u in zip(now, v):
            assert t is None or torch.equal(t, u)
    assert all(torch.equal(t, u) for t, u in zip(old, was))


def test_gradients_that_are_written(lib):
    """A gradient that is another layer's weight, momentum or bias, whole or in part, and tensors that came to share
    memory later."""
    w, m, b, bm, g, bg = layers()
    s = M.OrthogonalStep(w, m, b, bm)
    room = torch.randn(100)
    w[2].data = room[50:59].view(3, 3)
    refused(U, s.run, g, bg)                                                 # valid, but not on a GPU
    for i, bad in ((2, w[2]), (2, m[2]), (2, room[46:55].view(3, 3)), (2, room[58:67].view(3, 3)), (0, room[30:62].view(4, 8)),
                   (0, w[0]), (0, m[0])):
        refused(A, s.run, [bad if j == i else t for j, t in enumerate(g)], bg)
    for i, bad in ((0, b[0]), (0, bm[0]), (2, b[0][:3]), (2, bm[0][1:]), (0, room[55:59])):
        refused(A, s.run, g, [bad if j == i else t for j, t in enumerate(bg)])
    refused(A, s.run, [g[0], g[1], w[0].view(-1)[:9].view(3, 3)], bg)        # of another layer
    refused(U, s.run, [g[0], g[1], room[41:50].view(3, 3)], bg)              # beside it
    refused(U, s.run, [g[0], g[1], g[0].view(-1)[:9].view(3, 3)], bg)        # gradients are only read
    w[2].data = m[0].view(-1)[:9].view(3, 3)
    refused(A, s.run, g, bg)


@pytest.mark.parametrize("over", [dict(grad_w=0x30000), dict(grad_w=0x20000 + 4 * 6999), dict(grad_b=0x50004), dict(mom_b=0x50000 + 4 * 99),
                                  dict(w=0x70000, mom_w=0x70000 + 4 * 14), dict(w=0x10000 + 4 * 6999), dict(b=0x40000)])
def test_shared_memory_at_the_c_entry(lib, over):
    """The second of two layers on memory of the first, or on its own (addresses that are never read)."""
    from tests.test_tokens_abi import layer, step
    apart = dict(d_in=3, d_out=5, grad_w=0x100000, w=0x110000, mom_w=0x120000, grad_b=0x130000, b=0x140000, mom_b=0x150000)
    assert step(lib, [layer(), layer(**{**apart, **over})]) == A
