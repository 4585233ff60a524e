"""The objectives' kernels that only large inputs reach, on the GPU, against the definitions in 64 bits: passes
past the memory-side cache, teams that walk from one row (or round of tokens) to the next, and rows longer than a
team's registers.

The definitions are evaluated here in torch float64, some rows at a time; the scalars of a row and the statistics
come from the oracle.  Tolerances are those that tests/test_gpu_objectives.py derives.
"""
import numpy as np
import pytest
import torch

from oracle import objectives as O
from tests.test_gpu_objectives import DT, HALF, U, check_balance, gpu, near

pytestmark = pytest.mark.gpu


@pytest.fixture()
def Q(gpu_lib):
    from second_order_optimizer_amd import objectives
    return objectives


def pieces(rows, cols):
    step = max(1, (1 << 23) // cols)
    return [slice(i, min(rows, i + step)) for i in range(0, rows, step)]


def softmax64(x, s):
    """3 t of every logit (t = s |x - max|), its softmax, log of the sum of exponentials past the maximum."""
    d = (x.double() - x.double().amax(1, keepdim=True)) * s
    total = torch.exp(d).sum(1, keepdim=True)
    return -3 * d, torch.exp(d) / total, torch.log(total)


def score(x, labels, s):
    """(logp, its tolerance) of every row, 0 for rows without a label."""
    logp, tol = np.zeros(x.shape[0]), np.zeros(x.shape[0])
    for at in pieces(*x.shape):
        t, p, log_sum = softmax64(x[at], s)
        tl = t.gather(1, labels[at, None].clamp(min=0))
        lp = -tl / 3 - log_sum
        e = 2 * U * (tl + (t * p).sum(1, keepdim=True) + 3 * log_sum + 6)
        live = labels[at, None] >= 0
        logp[at] = torch.where(live, lp, 0.0)[:, 0].cpu().numpy()
        tol[at] = torch.where(live, e, 0.0)[:, 0].cpu().numpy()
    return logp, tol


def check_gradient(grad, x, labels, coef, coef_err, tol, s, dtype):
    """Every entry of coef s (onehot - softmax)."""
    coef, coef_err, tol = (torch.as_tensor(a, device="cuda") for a in (coef, coef_err, tol))
    for at in pieces(*x.shape):
        t, p, _ = softmax64(x[at], s)
        hot = torch.zeros_like(p).scatter_(1, labels[at, None].clamp(min=0), (labels[at, None] >= 0).double())
        c = (coef[at] * s)[:, None]
        want = torch.where(c != 0, c * (hot - p), 0.0)
        T = (t * p).sum(1, keepdim=True)
        lim = (c.abs() * p * ((t + T + 10) * U + hot * tol[at, None]) +
               ((coef_err[at] * s)[:, None] + 4 * U * c.abs()) * (hot - p).abs() + HALF[dtype] * want.abs() + 1e-36) * 1.01
        bad = ~((grad[at].double() - want).abs() <= lim)
        assert not bad.any(), (at, int(bad.sum()), bad.nonzero()[:4].tolist(), grad[at][bad][:4], want[bad][:4])


def token_rows(seed, rows, vocab, dtype, pad, unlabelled):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (2 * torch.randn(rows, vocab + pad, generator=gen, device="cuda")).to(DT[dtype])[:, :vocab]
    labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    labels[torch.rand(rows, generator=gen, device="cuda") < unlabelled] = -100
    return x, labels


f32 = lambda a: np.asarray(a, np.float32).astype(np.float64)


# a pass over more than 256 MB of logits and gradients, at each team that can hold its rows, and rows beyond the
# registers with more of them than workgroups
@pytest.mark.parametrize("rows,vocab,dtype,kl,s", [
    (140001, 500, "bf16", 0.02, 1.0), (34003, 1001, "f32", 0.0, 1.25), (13501, 5003, "bf16", 0.05, 1.0),
    (8009, 4999, "f32", 0.0, 1.0), (3001, 24001, "bf16", 0.0, 0.7), (1101, 61003, "bf16", 0.02, 1.0),
    (1101, 33001, "f32", 0.02, 1.0), (600, 140003, "bf16", 0.02, 1.0), (520, 70001, "f32", 0.0, 1.25)])
def test_policy(Q, rows, vocab, dtype, kl, s):
    x, labels = token_rows(rows, rows, vocab, dtype, vocab % 4, 0.15)
    rng = np.random.default_rng(rows)
    logp, tol = score(x, labels, s)
    old, ref = f32(logp + 0.2 * rng.normal(size=rows)), f32(logp + 0.3 * rng.normal(size=rows))
    for edge in (0.8, 1.28):                     # no ratio so near a border that rounding could choose its side
        old = np.where(np.abs(np.exp(logp - old) - edge) < 1e-3, f32(old - 0.01), old)
    adv, w = f32(rng.normal(size=rows)), f32(rng.random(rows) * (rng.random(rows) < 0.8) / rows)
    op = Q.PolicyLoss(rows, vocab, dtype, clip_low=0.2, clip_high=0.28, kl_coef=kl, logit_scale=s, grad_scale=float(rows))
    t = lambda a: gpu(a, torch.float32)
    stats, got, grad = op.run(x, labels, t(adv), t(w), t(old), t(ref))
    near(got, logp, tol, "logp")
    lab = labels.cpu().numpy()
    wstats, coef = O.policy_terms(logp, lab, adv, w, old, ref, 0.2, 0.28, kl)
    live = (lab >= 0) & (w != 0)
    ratio, ed = np.exp(logp - old), np.exp(ref - logp)
    err = np.where(live, rows * w * ((np.abs(adv) * ratio + kl * ed) * (tol + 12 * U) + 6 * U), 0)
    check_gradient(grad, x, labels, coef * rows, err, tol, s, dtype)
    a = (w * live * (np.abs(adv) * ratio + 1) * (tol + 12 * U)).sum()
    k = (w * live * (ed + 1) * (tol + 12 * U)).sum()
    near(stats, wstats, np.array([a + kl * k, a, k, 1e-30]) + 2 * U * np.abs(wstats), "stats")
    assert op.flags() == 0


# several wavefronts a row with many rows; passes past the cache (256 MB) whose first rows are read past it too
# (logits over 192 MB), with one wavefront a row and with four
@pytest.mark.parametrize("rows,pairs,vocab,dtype,kind,eps,average", [
    (700, 2, 5003, "bf16", "sigmoid", 0.1, False), (1300, 5, 2501, "f32", "squared", 0.0, True),
    (2601, 4, 50001, "bf16", "sigmoid", 0.0, False), (45001, 9, 3001, "bf16", "sigmoid", 0.1, True),
    (8009, 3, 9001, "f32", "squared", 0.0, True), (1501, 2, 50001, "bf16", "sigmoid", 0.1, False)])
def test_preference(Q, rows, pairs, vocab, dtype, kind, eps, average):
    x, labels = token_rows(rows, rows, vocab, dtype, vocab % 4, 0.1)
    rng = np.random.default_rng(rows)
    inner = np.sort(rng.choice(np.arange(2, rows - 1), 2 * pairs - 1, replace=False))
    offsets = np.concatenate([[1], inner, [rows - 1]]).astype(np.int32)      # the first and the last row are in none
    logp, tol = score(x, labels, 1.0)
    ref, w = f32(logp + 0.02 * rng.normal(size=rows)), f32(rng.random(pairs) + 0.1)
    beta, e = float(np.float32(0.1)), float(np.float32(eps))
    op = Q.PreferenceLoss(rows, pairs, vocab, dtype, 0.1, kind, eps, average, grad_scale=3.0)
    t = lambda a: gpu(a, torch.float32)
    stats, seq, got, grad = op.run(x, labels, gpu(offsets), t(ref), t(w))
    near(got, logp, tol, "logp")
    wstats, wseq, coef = O.preference_terms(logp, labels.cpu().numpy(), offsets, ref, w, beta, kind, e, average)
    st = np.array([tol[offsets[i]:offsets[i + 1]].sum() for i in range(2 * pairs)])
    near(seq, wseq, st + 2 * U * np.abs(wseq) + 1e-30, "seq")
    eh = st[:pairs] + st[pairs:]
    h = wseq[:pairs] - wseq[pairs:]
    first = np.full(pairs, beta) if kind == "sigmoid" else 2 * np.abs(h - 0.5 / beta) + 2 * eh
    second = beta * beta / 4 if kind == "sigmoid" else 2.0
    near(stats, wstats, np.array([(w * eh * first).sum(), 0, (w * eh * beta).sum(), 0]) + 4 * U * (np.abs(wstats) + 1), "stats")
    cerr = np.zeros(rows)
    for i in range(2 * pairs):
        cerr[offsets[i]:offsets[i + 1]] = 3.0 * w[i % pairs] * eh[i % pairs] * second
    cerr = (cerr + 2 * U * np.abs(3.0 * coef)) * (coef != 0)
    check_gradient(grad, x, labels, 3.0 * coef, cerr, tol, 1.0, dtype)
    assert op.flags() == 0


@pytest.mark.parametrize("tokens,E,k,dtype,z", [
    (2000, 8, 8, "bf16", 1e-3), (4096, 8, 2, "bf16", 0.0), (4096, 3, 3, "f32", 1e-3),      # one launch, slots past the first
    (70000, 16, 8, "bf16", 1e-3),                                                         # slots past the first, many workgroups
    (20000, 512, 2, "f32", 1e-3), (40001, 256, 3, "bf16", 0.0)])                          # tokens past the first round
def test_balance(Q, tokens, E, k, dtype, z):
    check_balance(Q, np.random.default_rng(tokens), tokens, E, k, dtype, z, pad=E % 2)


@pytest.mark.parametrize("rows,cols,dtype,residual", [(3000, 4099, "bf16", True), (4300, 4100, "bf16", False),
                                                      (1500, 4099, "f32", True), (2101, 4097, "f32", False)])
def test_dropout(Q, rows, cols, dtype, residual):
    """More than 64 MB of inputs and output: the kept elements exactly, their values to the roundings."""
    from perf import operators as P
    seed, off, p = 3 << 40 | 11, (1 << 50) + 7, 0.25
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols + 3, generator=gen, device="cuda").to(DT[dtype])[:, 1:cols + 1]
    res = torch.randn(rows, cols + 1, generator=gen, device="cuda").to(DT[dtype])[:, :cols] if residual else None
    op = Q.Dropout(rows, cols, dtype, p)
    y, dx = op.run(x, seed, off, residual=res), op.backward(x, seed, off)
    keep = P._keep(rows, cols, seed, off, p, x.device)
    part = torch.where(keep, x.double() / 0.75, 0.0)
    assert ((dx.double() - part).abs() <= (HALF[dtype] + 2 * U) * part.abs()).all()
    want = part + res.double() if residual else part
    lim = HALF[dtype] * want.abs() * (1 + 4 * U) + 3 * U * (part.abs() + (res.double().abs() if residual else 0.0))
    assert ((y.double() - want).abs() <= lim).all()
