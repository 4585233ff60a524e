"""The objectives on the GPU beside their numbers: batches of nothing, workspaces, autograd and flags."""
import ctypes

import numpy as np
import pytest
import torch

import second_order_optimizer_amd as K
from oracle import objectives as O
from tests.test_gpu_objectives import DT, U, gpu, near

pytestmark = pytest.mark.gpu


@pytest.fixture()
def Q(gpu_lib):
    from second_order_optimizer_amd import objectives
    return objectives


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [5, 513, 2052, 4104, 32768, 140003])
def test_no_rows_of_any_length(Q, vocab, dtype):
    """No rows: empty outputs; every pair's sequences are empty, and its loss at h = 0 counts."""
    x, f = torch.empty(0, vocab, dtype=DT[dtype], device="cuda"), torch.empty(0, device="cuda")
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    assert Q.TokenLogp(0, vocab, dtype).run(x, lab).shape == (0,)
    stats, logp, grad = Q.PolicyLoss(0, vocab, dtype).run(x, lab, f)
    assert stats.tolist() == [0, 0, 0, 0] and grad.shape == (0, vocab)
    op = Q.PreferenceLoss(0, 3, vocab, dtype)
    stats, seq, logp, grad = op.run(x, lab, torch.zeros(7, dtype=torch.int32, device="cuda"))
    near(stats, np.array([np.log(2), 0, 0, 1]), 4 * U)
    assert not seq.any() and logp.shape == (0,) and grad.shape == (0, vocab) and op.flags() == 0


class Shared:
    """C calls on one workspace, zeroed once."""
    def __init__(self, Q, nbytes):
        self.Q, self.lib = Q, Q._library()
        self.buf = torch.zeros(nbytes + 256, dtype=torch.uint8, device="cuda")
        self.ws, self.n = (self.buf.data_ptr() + 255) // 256 * 256, nbytes

    def call(self, fn, *structs):
        assert fn(*[ctypes.byref(s) for s in structs], self.ws, self.n, torch.cuda.current_stream().cuda_stream) == K.KFAC_OK

    def rows(self, x, labels):
        self.logp, self.grad = torch.empty(x.shape[0], device="cuda"), torch.empty_like(x)
        return self.Q.TokenRows(logits=x.data_ptr(), labels=labels.data_ptr(), logp=self.logp.data_ptr(),
                                grad=self.grad.data_ptr(), rows=x.shape[0], ld=x.shape[1], grad_ld=x.shape[1],
                                vocab=x.shape[1], dtype=K.F32, label_type=self.Q.I64, logit_scale=1.0, grad_scale=1.0)

    def policy(self, x, labels, adv):
        stats = torch.full((4,), float("nan"), device="cuda")
        self.call(self.lib.kfac_policy_loss, self.rows(x, labels),
                  self.Q.Policy(advantage=adv.data_ptr(), stats=stats.data_ptr(), clip_low=0.2, clip_high=0.2))
        return stats, self.logp, self.grad

    def preference(self, x, labels, offsets):
        seq, stats = torch.empty(offsets.numel() - 1, device="cuda"), torch.empty(4, device="cuda")
        self.call(self.lib.kfac_preference_loss, self.rows(x, labels),
                  self.Q.Preference(offsets=offsets.data_ptr(), seq=seq.data_ptr(), stats=stats.data_ptr(),
                                    pairs=seq.numel() // 2, beta=0.1))
        return stats, seq, self.logp, self.grad

    def balance(self, x, chosen):
        tokens, E = x.shape
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        prob, stats, grad = torch.empty(E, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(x)
        self.call(self.lib.kfac_balance_loss,
                  self.Q.Balance(logits=x.data_ptr(), chosen=chosen.data_ptr(), counts=counts.data_ptr(),
                                 prob=prob.data_ptr(), stats=stats.data_ptr(), grad=grad.data_ptr(), tokens=tokens, ld=E,
                                 grad_ld=E, experts=E, top_k=chosen.shape[1], dtype=K.F32, index_type=self.Q.I64, coef=0.01,
                                 z_coef=1e-3, grad_scale=1.0))
        return stats, counts, prob, grad


def test_objectives_in_turn_on_one_workspace(Q):
    """Other objectives between two policy losses on the same workspace leave its counters alone."""
    x, router = torch.randn(3000, 1500, device="cuda"), torch.randn(9000, 256, device="cuda")
    lab, adv = torch.randint(0, 1500, (3000,), device="cuda"), torch.randn(3000, device="cuda")
    off, ids = gpu([0, 1000, 3000], torch.int32), torch.randint(0, 256, (9000, 2), device="cuda")
    want = (Q.PolicyLoss(3000, 1500, "f32").run(x, lab, adv), Q.PreferenceLoss(3000, 1, 1500, "f32").run(x, lab, off),
            Q.BalanceLoss(9000, 256, 2, "f32", z_coef=1e-3).run(router, ids))
    s = Shared(Q, max(Q.workspace_size(Q.OBJ_POLICY, 3000), Q.workspace_size(Q.OBJ_PREFERENCE, 3000, 1),
                      Q.workspace_size(Q.OBJ_BALANCE, 9000, 256)))
    for turn in range(2):
        for other in range(1, 3):
            got = s.preference(x, lab, off) if other == 1 else s.balance(router, ids)
            assert all(torch.equal(a, b) for a, b in zip(want[other], got)), (turn, other)
            assert all(torch.equal(a, b) for a, b in zip(want[0], s.policy(x, lab, adv))), (turn, other)


def test_writes_are_seen_by_autograd(Q):
    """A tensor given to be written counts the write, so that a backward pass which saved it is refused."""
    x, lab, f = torch.randn(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    off, ids = gpu([0, 2, 4], torch.int32), torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    calls = (lambda g: Q.PolicyLoss(4, 8, "f32").run(x, lab, f, grad=g),
             lambda g: Q.PreferenceLoss(4, 1, 8, "f32").run(x, lab, off, grad=g),
             lambda g: Q.BalanceLoss(4, 8, 2, "f32").run(x, ids, grad=g),
             lambda g: Q.Dropout(4, 8, "f32").run(x, 1, out=g))
    for call in calls:
        g = torch.empty_like(x)
        before = g._version
        call(g)
        assert g._version == before + 1 and x._version == 0
        with torch.inference_mode():
            g = torch.empty_like(x)
        call(g)                               # outside the mode: written, nothing to count
    h = torch.relu(torch.randn(4, 8, device="cuda", requires_grad=True))
    Q.Dropout(4, 8, "f32", 0.5).run(h.detach(), 1, out=h.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        h.sum().backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_in_autograd(Q, dtype):
    """The gradient of x is backward()'s of the output gradient, and the residual's is that itself; for any strides of
    the output gradient, on a stream, and twice."""
    op = Q.Dropout(9, 33, dtype, 0.3)
    x, r, dy = (torch.randn(9, 33, device="cuda").to(DT[dtype]) for _ in range(3))
    want, dx = op.run(x, 5, 6, residual=r), op.backward(dy, 5, 6)
    xg, rg = x.clone().requires_grad_(), r.clone().requires_grad_()
    y = op.run(xg, 5, 6, residual=rg)
    assert torch.equal(y, want) and y.requires_grad
    a, b = torch.autograd.grad(y, (xg, rg), dy)
    assert torch.equal(a, dx) and torch.equal(b, dy)
    assert torch.equal(torch.autograd.grad(op.run(xg, 5, 6), xg, dy.t().contiguous().t())[0], dx)
    ones = torch.autograd.grad(op.run(xg, 5, 6, residual=r).float().sum(), xg)[0]          # a broadcast output gradient
    assert torch.equal(ones, op.backward(torch.ones_like(x), 5, 6))
    assert torch.equal(torch.autograd.grad(op.run(x, 5, 6, residual=rg), rg, dy)[0], dy)
    # linear: the gradient's gradient is the same mask again
    v = torch.ones_like(x, requires_grad=True)
    g, = torch.autograd.grad(op.run(xg, 5, 6), xg, v, create_graph=True)
    assert torch.equal(torch.autograd.grad(g, v, dy)[0], dx)
    with torch.no_grad():
        assert not op.run(xg, 5, 6).requires_grad
    assert not op.run(xg.detach(), 5, 6).requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = op.run(xg, 5, 6, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(torch.autograd.grad(y, xg, dy)[0], dx)


def test_dropout_gradient_against_differences(Q):
    """Linear in x: half the difference of two values along a direction is the gradient's product with it, up to the
    roundings of those values (2 u each, over 297 entries)."""
    op = Q.Dropout(9, 33, "f32", 0.3)
    x, d, dy = (torch.randn(9, 33, device="cuda", dtype=torch.float64).float() for _ in range(3))
    xg = x.clone().requires_grad_()
    g = torch.autograd.grad(op.run(xg, 5, 6), xg, dy)[0].double()
    up, down = op.run(x + d, 5, 6).double(), op.run(x - d, 5, 6).double()
    lim = 4 * U * (dy.double().abs() * (up.abs() + down.abs())).sum() + 4 * U * (g * d.double()).abs().sum()
    assert abs((g * d.double()).sum() - ((up - down) / 2 * dy.double()).sum()) <= lim


def test_dropout_backward_sees_a_moved_offset(Q):
    """A mask that offset_tensor named is found again in the backward pass, or that pass is refused."""
    op = Q.Dropout(9, 33, "f32", 0.3)
    x, step = torch.randn(9, 33, device="cuda", requires_grad=True), torch.full((1,), 4, dtype=torch.int64, device="cuda")
    y = op.run(x, 5, 6, offset_tensor=step)
    dy = torch.ones_like(x)
    assert torch.equal(torch.autograd.grad(y, x, dy, retain_graph=True)[0], op.backward(dy, 5, 10))
    step.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(y, x, dy)


# -- results beyond float32 --------------------------------------------------------------------

def test_policy_sum_beyond_float32_is_flagged(Q):
    """Rows whose losses are finite and whose sum is not."""
    x, lab = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    op = Q.PolicyLoss(4, 8, "f32", grad_scale=1e-3)
    w = torch.ones(4, device="cuda")
    stats, _, grad = op.run(x, lab, torch.full((4,), 2e38, device="cuda"), weight=w)
    assert stats[0].isinf() and grad.isfinite().all() and op.flags(clear=True) == K.FLAG_NONFINITE
    assert op.run(x, lab, torch.full((4,), 2e37, device="cuda"), weight=w)[0].isfinite().all() and op.flags() == 0


def test_preference_loss_beyond_float32_is_flagged(Q):
    x, lab, off = torch.zeros(2, 8, device="cuda"), gpu([2, 3]), gpu([0, 1, 2], torch.int32)
    op = Q.PreferenceLoss(2, 1, 8, "f32", kind="squared")
    stats, _, _, grad = op.run(x, lab, off, ref_logp=gpu([-1e25, 0], torch.float32))
    assert stats[0].isinf() and grad.isfinite().all() and op.flags(clear=True) == K.FLAG_NONFINITE
    assert op.run(x, lab, off, ref_logp=gpu([-1e15, 0], torch.float32))[0].isfinite().all() and op.flags() == 0


def test_preference_sum_beyond_float32_is_flagged(Q):
    """Pairs whose losses are finite and whose sum is not."""
    x, lab, off = torch.zeros(8, 8, device="cuda"), gpu(np.arange(8)), gpu(np.arange(9), torch.int32)
    op = Q.PreferenceLoss(8, 4, 8, "f32", kind="squared")
    ref = gpu([-1.4e19] * 4 + [0.0] * 4, torch.float32)
    stats = op.run(x, lab, off, ref_logp=ref, pair_weight=torch.ones(4, device="cuda"))[0]
    assert stats[0].isinf() and op.flags() == K.FLAG_NONFINITE


@pytest.mark.parametrize("tokens,E", [(40, 16), (9000, 256)])
def test_balance_beyond_float32_is_flagged(Q, tokens, E):
    """A z loss, a gradient of it and a gradient of the balance loss that float32 does not hold, in one launch and in
    three; masked tokens that would are not looked at."""
    ids = torch.zeros(tokens, 1, dtype=torch.int64, device="cuda")
    for fill, kw in ((1e25, dict(z_coef=1e-3)), (100.0, dict(z_coef=1e3, grad_scale=2e34 * tokens)),
                     (0.0, dict(coef=1e30, grad_scale=1e20))):
        x = torch.full((tokens, E), fill, device="cuda")
        op = Q.BalanceLoss(tokens, E, 1, "f32", **kw)
        stats, _, _, grad = op.run(x, ids)
        assert not (stats.isfinite().all() and grad.isfinite().all()) and op.flags(clear=True) == K.FLAG_NONFINITE, kw
        stats, _, _, grad = op.run(x, ids, mask=torch.zeros(tokens, dtype=torch.bool, device="cuda"))
        assert not stats.any() and not grad.any() and op.flags() == 0, kw


@pytest.mark.parametrize("vocab", [8, 3001])
def test_zero_advantage_with_a_ratio_beyond_float32(Q, vocab):
    """A term of 0 and a gradient of 0, not 0 times infinity; a positive advantage there is clipped."""
    x = torch.zeros(2, vocab, device="cuda")
    x[:, 0] = 200.0
    adv, old = np.array([0.0, 1.0]), np.array([-100.0, -100.0])
    op = Q.PolicyLoss(2, vocab, "f32")
    stats, _, grad = op.run(x, gpu([0, 0]), gpu(adv, torch.float32), old_logp=gpu(old, torch.float32))
    want = O.policy_loss(x.cpu().numpy(), [0, 0], adv, None, old, hi=float(np.float32(0.2)))[0]
    near(stats, want, 4 * U * np.abs(want))
    assert not grad.any() and op.flags() == 0


def test_policy_logp_has_no_bias_from_the_rounded_scale(Q):
    """bf16 rows multiply by s log2(e) in float32.  At s = 0.85 the nearest float32 is 0.04 u from it, its lower
    neighbour 1.6 u: over the mean exponent of 8.5 here that one would bias log S by 13 u.  The roundings of the
    products (64 values of the logits, up to 11 u each, of either sign) leave less than 3 u of their mean, log S of
    1.8 and its float32 another 2 u."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = (-10 - 4 * torch.rand(64, 131072, generator=gen, device="cuda")).bfloat16()
    x[:, 0] = 0
    op = Q.PolicyLoss(64, 131072, logit_scale=0.85)
    logp = op.run(x, torch.zeros(64, dtype=torch.int64, device="cuda"), torch.ones(64, device="cuda"))[1]
    want = -torch.logsumexp(x.double() * float(np.float32(0.85)), 1)
    assert abs((logp.double() - want).mean()) <= 5 * U

