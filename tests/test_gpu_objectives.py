"""The objectives and dropout on the GPU against the float64 oracle.

Tolerances, from the roundings on the way (u = 2^-24, half a step of
float32): a term exp(s (x - M)) has its argument rounded three times and the
hardware's 2^x within one step, so with t = s |x - M| it is off by at most
(3 t + 2) u relatively; terms are added as trees of at most three float32
additions and then in 64 bits, so S is off by (T + 5) u with T the mean of 3 t
under the softmax, and log S by as much plus 2 u |log S|.  logp adds the
rounding of its own two terms.  LOGP(...) below is that sum, doubled.  A
gradient entry is coef p: p is off by (3 t + T + 8) u relatively, coef by what
logp's error makes of it (exp of it) plus a few u, and the result is rounded
once to its type (2^-9 of a value in a bf16 gradient has its half step at most
2^-8).
"""
import numpy as np
import pytest
import torch

from oracle import objectives as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture()
def Q(gpu_lib):
    from second_order_optimizer_amd import objectives
    return objectives


def gpu(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def wide(t):
    return t.double().cpu().numpy()


def matrix(rng, rows, cols, dtype, pad=0, lead=0, scale=2.0):
    """(tensor on the GPU, its values in 64 bits): N(0, scale), a slice of rows with `pad` more columns, `lead` of
    them in front."""
    whole = torch.from_numpy(rng.normal(size=(rows, cols + pad)).astype(np.float32) * scale).to(DT[dtype]).cuda()
    t = whole[:, lead:lead + cols]
    return t, wide(t)


def spread(x, s):
    """3 t of every logit, and its mean under the softmax, [rows, vocab] and [rows, 1]."""
    t = 3 * s * np.abs(x - x.max(axis=1, keepdims=True))
    p = np.exp(O.log_softmax(x, s))
    return t, p, (np.where(p > 0, t, 0) * p).sum(axis=1, keepdims=True)


def logp_tolerance(x, labels, s):
    t, p, T = spread(x, s)
    tl = np.take_along_axis(t, np.clip(labels, 0, x.shape[1] - 1)[:, None], 1)[:, 0]
    logS = np.abs(np.log(np.exp((x - x.max(axis=1, keepdims=True)) * s).sum(axis=1)))
    return 2 * U * (tl + T[:, 0] + 3 * logS + 6)


def near(got, want, tol, what=""):
    got = wide(got) if torch.is_tensor(got) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, bad.shape)[bad][:4])


def grad_tolerance(x, labels, coef, coef_err, s, dtype, want):
    """|grad| is |coef s| (onehot + p) at most in its parts."""
    t, p, T = spread(x, s)
    hot = np.zeros(x.shape)
    hot[np.arange(labels.size), np.clip(labels, 0, None)] = labels >= 0
    c = np.abs(coef * s)[:, None]
    lp = logp_tolerance(x, labels, s)[:, None]
    return (c * p * (t + T + 10) * U + c * hot * p * lp + (coef_err * s)[:, None] * np.abs(hot - p) +
            4 * U * c * np.abs(hot - p) + HALF[dtype] * np.abs(want) + 1e-36) * 1.01


# team sizes and register counts change at 4, 16, 32, 64, 128 and 256 KB a row
VOCABS = [1, 2, 3, 7, 8, 9, 63, 257, 1000, 2048, 2049, 8191, 16387, 33001, 65536, 70001, 131072, 140003]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_logp(Q, vocab, dtype):
    rng = np.random.default_rng(vocab)
    rows = 1 if vocab % 3 == 0 else 5
    x, xd = matrix(rng, rows, vocab, dtype, pad=vocab % 4, lead=vocab % 2 if vocab % 4 else 0)
    labels = rng.integers(0, vocab, rows)
    labels[-1] = vocab - 1
    for s in (1.0, 0.7):
        got = Q.TokenLogp(rows, vocab, dtype, logit_scale=s).run(x, gpu(labels))
        near(got, O.token_logp(xd, labels, s), logp_tolerance(xd, labels, s), s)


@pytest.mark.parametrize("rows", [1, 3, 511, 513, 2500])
def test_logp_many_rows(Q, rows):
    rng = np.random.default_rng(rows)
    for vocab, dtype in ((129, "bf16"), (3001, "f32"), (5003, "bf16")):
        x, xd = matrix(rng, rows, vocab, dtype)
        labels = rng.integers(-1, vocab, rows).astype(np.int32)
        got = Q.TokenLogp(rows, vocab, dtype).run(x, gpu(labels))
        near(got, O.token_logp(xd, labels), logp_tolerance(xd, labels, 1.0))


@pytest.mark.parametrize("rows,vocab,dtype", [(20011, 40, "bf16"), (20011, 700, "f32"), (600001, 9, "bf16"),
                                              (530000, 5, "f32")])
def test_logp_rows_beyond_the_teams(Q, rows, vocab, dtype):
    """Each team walks several rows; short ones are finished up to 64 at a time, and 8192 teams of them are resident."""
    rng = np.random.default_rng(rows)
    x, xd = matrix(rng, rows, vocab, dtype)
    labels = rng.integers(-1, vocab, rows).astype(np.int32)
    got = Q.TokenLogp(rows, vocab, dtype).run(x, gpu(labels))
    near(got, O.token_logp(xd, labels), np.where(labels >= 0, logp_tolerance(xd, labels, 1.0), 0))


def policy_inputs(rng, xd, labels, s):
    logp = O.token_logp(xd, labels, s)
    n = labels.size
    f = lambda a: np.asarray(a, np.float32).astype(np.float64)
    old, ref = f(logp + 0.2 * rng.normal(size=n)), f(logp + 0.3 * rng.normal(size=n))
    for edge in (0.8, 1.28):                     # no ratio so near a border that rounding could choose its side
        old = np.where(np.abs(np.exp(logp - old) - edge) < 1e-3, f(old - 0.01), old)
    return f(rng.normal(size=n)), f(rng.random(n) * (rng.random(n) < 0.8)), old, ref


def check_policy(Q, rng, rows, vocab, dtype, kl, s, pad=0, lead=0, in_place=False, few=False):
    x, xd = matrix(rng, rows, vocab, dtype, pad, lead)
    labels = rng.integers(0, vocab, rows)
    labels[rng.random(rows) < 0.15] = -100
    adv, w, old, ref = policy_inputs(rng, xd, labels, s)
    if few:
        w, old, ref = None, None, None
    op = Q.PolicyLoss(rows, vocab, dtype, clip_low=0.2, clip_high=0.28, kl_coef=kl, logit_scale=s, grad_scale=float(rows))
    t = lambda a: None if a is None else gpu(a, torch.float32)
    stats, logp, grad = op.run(x, gpu(labels), t(adv), weight=t(w), old_logp=t(old), ref_logp=t(ref),
                               grad=x if in_place else None)
    wstats, wlogp, wgrad = O.policy_loss(xd, labels, adv, w, old, ref, 0.2, 0.28, kl, s, float(rows))
    tol = logp_tolerance(xd, labels, s)
    near(logp, wlogp, np.where(labels >= 0, tol, 0), "logp")
    full = np.full(rows, 1.0 / rows) if w is None else w
    ratio = np.ones(rows) if old is None else np.exp(wlogp - old)
    d = np.zeros(rows) if ref is None else ref - wlogp
    # what logp's error makes of the coefficient and of the two terms, and their own roundings
    err = rows * full * ((np.abs(adv) * ratio + kl * np.exp(d)) * (tol + 12 * U) + 6 * U)
    live = (labels >= 0) & (full != 0)
    coef = np.where(live, rows * O.policy_terms(wlogp, labels, adv, full, old, ref, .2, .28, kl)[1], 0)
    near(grad, wgrad, grad_tolerance(xd, labels, coef, np.where(live, err, 0), s, dtype, wgrad), "grad")
    st = (full * live * ((np.abs(adv) * ratio + 1) * (tol + 12 * U))).sum() + 2 * U * np.abs(wstats)
    sk = (full * live * ((np.exp(d) + 1) * (tol + 12 * U))).sum()
    near(stats, wstats, np.array([st[0] + kl * sk, st[1], sk + st[2], st[3]]) + 1e-30, "stats")
    assert op.flags() == 0
    # ignored rows are exactly 0
    assert not grad[torch.from_numpy(~live).cuda()].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy(Q, vocab, dtype):
    rng = np.random.default_rng(vocab + 1)
    check_policy(Q, rng, 1 + vocab % 6, vocab, dtype, kl=0.05 * (vocab % 2), s=1.25 if vocab % 3 else 1.0,
                 pad=vocab % 5, lead=vocab % 3 if vocab % 5 > 2 else 0)


@pytest.mark.parametrize("rows,vocab,dtype", [(1500, 100, "bf16"), (1600, 333, "f32"), (1537, 2100, "bf16"),
                                              (1300, 2500, "f32"), (700, 12000, "f32"), (300, 40000, "bf16")])
def test_policy_more_rows_than_teams(Q, rows, vocab, dtype):
    """Rows beyond the resident teams: each team walks several, the next row's loads in flight."""
    check_policy(Q, np.random.default_rng(rows), rows, vocab, dtype, 0.02, 1.0, pad=3)


@pytest.mark.parametrize("rows,vocab,dtype", [(1, 90, "bf16"), (130, 90, "f32"), (7001, 90, "bf16"), (3100, 1200, "f32")])
def test_policy_statistics_over_many_workgroups(Q, rows, vocab, dtype):
    """From one workgroup to all that are resident, counted in groups; the same object again gives the same."""
    rng = np.random.default_rng(rows + vocab)
    check_policy(Q, rng, rows, vocab, dtype, 0.02, 1.0)
    x = torch.randn(rows, vocab, device="cuda").to(DT[dtype])
    lab, adv = torch.randint(0, vocab, (rows,), device="cuda"), torch.randn(rows, device="cuda")
    op = Q.PolicyLoss(rows, vocab, dtype)
    first = op.run(x, lab, adv)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, op.run(x, lab, adv)))


@pytest.mark.parametrize("vocab,dtype", [(9, "bf16"), (3001, "bf16"), (70001, "f32"), (140003, "bf16")])
def test_policy_in_place_and_defaults(Q, vocab, dtype):
    rng = np.random.default_rng(5)
    check_policy(Q, rng, 5, vocab, dtype, 0.02, 1.0, pad=1, in_place=True)
    check_policy(Q, rng, 5, vocab, dtype, 0.0, 1.0, few=True)


@pytest.mark.parametrize("vocab,dtype", [(40, "f32"), (300, "bf16"), (5000, "bf16"), (70000, "f32")])
def test_policy_gradient_against_differences(Q, vocab, dtype):
    """The gradient's product with a direction against differences of the oracle's loss along it: the
    difference quotient errs by h^2 of the third derivative, below 1e-6 here; the gradient's own rounding adds at
    most its half step times sum |g d|."""
    rng = np.random.default_rng(vocab)
    x, xd = matrix(rng, 6, vocab, dtype)
    labels = rng.integers(0, vocab, 6)
    adv, w, old, ref = policy_inputs(rng, xd, labels, 1.0)
    w = w + 0.1
    op = Q.PolicyLoss(6, vocab, dtype, clip_high=0.28, kl_coef=0.1)
    t = lambda a: gpu(a, torch.float32)
    g = wide(op.run(x, gpu(labels), t(adv), t(w), t(old), t(ref))[2])
    dirn = rng.normal(size=xd.shape)
    dirn[np.arange(6), labels] = 1.0
    w = w.astype(np.float32).astype(np.float64)
    loss = lambda h: O.policy_loss(xd + h * dirn, labels, adv, w, old, ref, 0.2, 0.28, 0.1)[0][0]
    want = (loss(1e-4) - loss(-1e-4)) / 2e-4
    assert abs((g * dirn).sum() - want) <= 1e-5 + 2 * HALF[dtype] * np.abs(g * dirn).sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [13, 1000, 9001, 70001])
def test_masked_columns_and_rows(Q, vocab, dtype):
    """Columns of -inf and of the type's lowest value are probability 0; a row all at the lowest value is
    uniform; NaN and infinities in rows left out (negative label, weight 0) reach nothing."""
    rng = np.random.default_rng(3)
    low = torch.finfo(DT[dtype]).min
    x, _ = matrix(rng, 6, vocab, dtype)
    x[0, 1:vocab // 2] = -float("inf")
    x[1, 1:vocab // 2] = low
    x[2, :] = low
    x[3, ::2] = float("nan")
    x[4, 1] = float("inf")
    x[4, 2] = -float("inf")
    labels = np.array([0, vocab - 1, 5, -1, 3, 7])
    adv = np.array([1.0, -0.5, 0.25, np.nan, np.nan, 2.0])
    w = np.array([0.5, 0.25, 0.125, 1.0, 0.0, 0.5])
    op = Q.PolicyLoss(6, vocab, dtype, kl_coef=0.1, grad_scale=2.0)
    ref = np.array([-1.0, -2.0, -3.0, np.nan, np.inf, -1.0])
    t = lambda a: gpu(a, torch.float32)
    stats, logp, grad = op.run(x, gpu(labels), t(adv), t(w), None, t(ref))
    keep = [0, 1, 2, 5]
    xd = wide(x)[keep]
    wstats, wlogp, wgrad = O.policy_loss(xd, labels[keep], adv[keep], w[keep], None, ref[keep], kl=0.1, grad_scale=2.0)
    # the reference is up to ~12 away from logp, so the KL terms are large: relative to them
    xt = np.where(np.isfinite(xd) & (xd > -1e30), xd, 0.0)      # columns of probability 0 carry no error
    lt = logp_tolerance(xt, labels[keep], 1.0)
    near(logp[keep], wlogp, lt + 1e-6)
    big = 1 + np.exp(np.abs(ref[keep] - wlogp))
    near(stats, wstats, 1e-5 * (w[keep] * big).sum())
    near(grad[keep], wgrad, HALF[dtype] * np.abs(wgrad) + 1e-5 * (w[keep] * big)[:, None])
    assert wide(logp)[3] == 0 and not grad[3].any() and not grad[4].any()
    assert op.flags() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [13, 1000, 9001, 70001])
def test_masked_columns_in_sequences(Q, vocab, dtype):
    """The same columns in the log-probabilities and the preference loss, at several scales."""
    rng = np.random.default_rng(4)
    x, _ = matrix(rng, 4, vocab, dtype)
    x[0, 1:vocab // 2] = -float("inf")
    x[1, 1:vocab // 2] = torch.finfo(DT[dtype]).min
    x[2, :] = torch.finfo(DT[dtype]).min
    labels = np.array([0, vocab - 1, 5, 3])
    xd = wide(x)
    xt = np.where(np.isfinite(xd) & (xd > -1e30), xd, 0.0)
    for s in (1.0, 0.7, 2.0):
        want = O.token_logp(xd, labels, s)
        near(Q.TokenLogp(4, vocab, dtype, logit_scale=s).run(x, gpu(labels)), want, logp_tolerance(xt, labels, s) + 1e-6)
        op = Q.PreferenceLoss(4, 1, vocab, dtype, logit_scale=s)
        stats, seq, logp, grad = op.run(x, gpu(labels), gpu([0, 2, 4], torch.int32))
        wstats, wseq, _, wgrad = O.preference_loss(xd, labels, [0, 2, 4], beta=float(np.float32(0.1)), s=s)
        near(seq, wseq, 2 * (logp_tolerance(xt, labels, s).sum() + 1e-6))
        near(stats, wstats, 1e-5)
        near(grad, wgrad, HALF[dtype] * np.abs(wgrad) + 1e-5)
        assert op.flags() == 0


def test_nonfinite_and_bad_labels_are_flagged(Q):
    x = torch.zeros(4, 50, device="cuda")
    x[1, 3] = float("nan")
    f = torch.ones(4, device="cuda")
    op = Q.PolicyLoss(4, 50, "f32")
    g = op.run(x, gpu([1, 2, 3, 4]), f)[2]
    assert g[1].isnan().all() and not g[[0, 2, 3]].isnan().any()
    assert op.flags(clear=True) == 2 and op.flags() == 0
    x[1, 3] = 0
    for big in (50, 1 << 40):
        stats, logp, g = op.run(x, gpu([1, big, 3, -5]), f, weight=f)
        assert op.flags(clear=True) == Q.FLAG_BAD_INDEX
        assert not g[1].any() and not g[3].any() and logp[1] == 0 and g[0].any()
    op = Q.TokenLogp(4, 50, "f32")
    assert op.run(x, gpu([1, 50, 3, 4], torch.int32)).tolist()[1] == 0 and op.flags() == Q.FLAG_BAD_INDEX


def test_no_rows(Q):
    e = torch.empty(0, device="cuda")
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 9, device="cuda")
    assert Q.TokenLogp(0, 9, "f32").run(x, lab).shape == (0,)
    stats, logp, grad = Q.PolicyLoss(0, 9, "f32").run(x, lab, e)
    assert stats.tolist() == [0, 0, 0, 0] and grad.shape == (0, 9)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    stats, seq, _, _ = Q.PreferenceLoss(0, 1, 9, "f32").run(x, lab, off)
    near(stats, np.array([np.log(2), 0, 0, 1]), 2 * U)
    assert seq.tolist() == [0, 0]
    stats, counts, prob, _ = Q.BalanceLoss(0, 9, 2, "f32").run(x, torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    assert stats.tolist() == [0, 0, 0, 0] and not counts.any() and not prob.any()
    assert Q.Dropout(0, 9, "f32").run(x, 1).shape == (0, 9)


# -- preference ------------------------------------------------------------------------------

def check_preference(Q, rng, lengths, vocab, dtype, beta, kind, eps, average, ref=True, weight=True, before=0, after=0,
                     pad=0, in_place=False, s=1.0):
    pairs = len(lengths) // 2
    rows = before + sum(lengths) + after
    offsets = (before + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32)
    x, xd = matrix(rng, rows, vocab, dtype, pad)
    labels = rng.integers(0, vocab, rows)
    labels[rng.random(rows) < 0.2] = -1
    f = lambda a: np.asarray(a, np.float32).astype(np.float64)
    wlp = O.token_logp(xd, labels, s)
    r = f(wlp + 0.3 * rng.normal(size=rows)) if ref else None
    w = f(rng.random(pairs) * (np.arange(pairs) != 1)) if weight else None
    op = Q.PreferenceLoss(rows, pairs, vocab, dtype, beta, kind, eps, average, logit_scale=s, grad_scale=3.0)
    t = lambda a: None if a is None else gpu(a, torch.float32)
    stats, seq, logp, grad = op.run(x, gpu(labels), gpu(offsets), t(r), t(w), grad=x if in_place else None)
    beta = float(np.float32(beta))
    eps = float(np.float32(eps))
    wstats, wseq, wlogp, wgrad = O.preference_loss(xd, labels, offsets, r, w, beta, kind, eps, average, s, 3.0)
    tol = np.where(labels >= 0, logp_tolerance(xd, labels, s), 0)
    near(logp, wlogp, tol, "logp")
    st = np.array([tol[offsets[i]:offsets[i + 1]].sum() for i in range(2 * pairs)])
    near(seq, wseq, st + 2 * U * np.abs(wseq) + 1e-30, "seq")
    eh = st[:pairs] + st[pairs:]
    h = wseq[:pairs] - wseq[pairs:]
    wt = np.full(pairs, 1.0 / pairs) if w is None else w
    # |d loss / dh| and |d slope / dh|: at most beta and beta^2 / 4, or 2 |h - 1 / 2 beta| and 2
    first = np.full(pairs, beta) if kind == "sigmoid" else 2 * np.abs(h - 0.5 / beta) + 2 * eh
    second = beta * beta / 4 if kind == "sigmoid" else 2.0
    e = (wt * eh * first).sum()
    near(stats, wstats, np.array([e, 0, (wt * eh * beta).sum(), 0]) + 4 * U * (np.abs(wstats) + 1) + 1e-30, "stats")
    coef = 3.0 * O.preference_terms(wlogp, labels, offsets, r, w, beta, kind, eps, average)[2]
    cerr = np.zeros(rows)
    for i in range(2 * pairs):
        cerr[offsets[i]:offsets[i + 1]] = 3.0 * wt[i % pairs] * eh[i % pairs] * second
    cerr = (cerr + 2 * U * np.abs(coef)) * (coef != 0)
    near(grad, wgrad, grad_tolerance(xd, labels, coef, cerr, s, dtype, wgrad), "grad")
    assert op.flags() == 0


@pytest.mark.parametrize("kind,eps,average", [("sigmoid", 0.0, False), ("sigmoid", 0.1, True), ("squared", 0.0, False),
                                              ("squared", 0.0, True)])
@pytest.mark.parametrize("vocab,dtype", [(1, "f32"), (37, "bf16"), (1000, "f32"), (9001, "bf16"), (70001, "f32")])
def test_preference(Q, vocab, dtype, kind, eps, average):
    rng = np.random.default_rng(vocab)
    few = vocab > 9000
    check_preference(Q, rng, [3, 0, 5, 1, 4, 2] if few else [30, 0, 7, 1, 300, 22], vocab, dtype, 0.5, kind, eps, average,
                     before=2, after=1, pad=vocab % 3)
    check_preference(Q, rng, [1, 1], vocab, dtype, 0.1, kind, eps, average, ref=False, weight=False,
                     in_place=True, s=0.8)


def test_preference_impossible_rejected_token(Q):
    """A rejected sequence of probability 0: the pair is won outright, its loss and gradients are 0 without
    smoothing; a preferred one of probability 0 is an infinite loss, which is flagged, with its gradient at the
    limit, beta (p - onehot) on that side."""
    x = torch.zeros(2, 8, device="cuda")
    x[1, 3] = -float("inf")
    lab = gpu([2, 3])
    off = gpu([0, 1, 2], torch.int32)
    op = Q.PreferenceLoss(2, 1, 8, "f32", beta=0.5)
    stats, seq, logp, grad = op.run(x, lab, off)
    assert stats[0] == 0 and stats[1] == 1 and stats[3] == 1 and seq[1] == -float("inf") and not grad.any()
    assert op.flags(clear=True) == 0
    stats, _, _, grad = op.run(x.flip(0).contiguous(), lab.flip(0).contiguous(), off)
    assert stats[0] == float("inf") and op.flags() == 2
    want = np.full(8, 0.5 / 7)
    want[3] = -0.5
    near(grad[0], want, 8 * U)
    near(grad[1], np.where(np.arange(8) == 2, 0.5 * 7 / 8, -0.5 / 8), 8 * U)


def test_preference_gradient_overflow_is_flagged(Q):
    x = torch.zeros(2, 8, device="cuda")
    op = Q.PreferenceLoss(2, 1, 8, "f32", beta=1e3, grad_scale=1e38)
    stats = op.run(x, gpu([2, 3]), gpu([0, 1, 2], torch.int32))[0]
    assert stats.isfinite().all() and op.flags() == 2


def test_preference_many_rows(Q):
    check_preference(Q, np.random.default_rng(0), [400, 350, 600, 500, 300, 450], 513, "bf16", 0.1, "sigmoid", 0.1, False)


def test_preference_weightless_pair_and_bad_offsets(Q):
    """A pair of weight 0 counts for nothing, NaN logits and all; offsets that decrease or pass the rows are
    flagged and their sequences are empty; rows of no sequence get gradient 0."""
    x = torch.randn(8, 20, device="cuda")
    x[2:4] = float("nan")
    lab = torch.arange(8, device="cuda")
    w = torch.tensor([1.0, 0.0], device="cuda")
    op = Q.PreferenceLoss(8, 2, 20, "f32")
    stats, seq, logp, grad = op.run(x, lab, gpu([0, 2, 4, 6, 8], torch.int32), pair_weight=w)
    assert stats.isfinite().all() and stats[3] == 1 and not grad[2:4].any() and not grad[6:].any()
    assert grad[:2].any() and grad[4:6].any() and op.flags() == 0
    x = torch.randn(8, 20, device="cuda")
    for off in ([0, 2, 1, 6, 8], [0, 2, 4, 6, 9], [-1, 2, 4, 6, 8]):
        _, seq, _, grad = op.run(x, lab, gpu(off, torch.int32))
        assert op.flags(clear=True) == Q.FLAG_BAD_INDEX and grad.isfinite().all() and seq.isfinite().all()
    _, _, _, grad = op.run(x, lab, gpu([1, 2, 4, 6, 7], torch.int32))
    assert op.flags() == 0 and not grad[0].any() and not grad[7].any() and grad[1:7].any(1).all()


# -- balance -----------------------------------------------------------------------------------

def check_balance(Q, rng, tokens, E, k, dtype, z, mask="some", pad=0, index=np.int32, in_place=False):
    x, xd = matrix(rng, tokens, E, dtype, pad, scale=1.0)
    chosen = np.stack([rng.permutation(E)[:k] for _ in range(tokens)]).astype(index)
    chosen[rng.random(chosen.shape) < 0.1] = -1
    m = None if mask is None else (rng.random(tokens) < 0.7 if mask == "some" else np.zeros(tokens, bool))
    if m is not None:
        x[torch.from_numpy(~m).cuda()] = float("nan")
        xd[~m] = np.nan
    op = Q.BalanceLoss(tokens, E, k, dtype, coef=0.01, z_coef=z, grad_scale=float(tokens))
    stats, counts, prob, grad = op.run(x, gpu(chosen), None if m is None else gpu(m), grad=x if in_place else None)
    c, zc = float(np.float32(0.01)), float(np.float32(z))
    wstats, wcounts, wprob, wgrad = O.balance_loss(xd, chosen, m, c, zc, float(tokens))
    assert counts.tolist() == wcounts.tolist()
    live = np.ones(tokens, bool) if m is None else m
    xl = xd[live]
    if xl.size:
        t, p, T = spread(xl, 1.0)
        # a softmax entry: its argument's and the sum's roundings, sums of at most 16 + 6 float32 additions
        rel = (t + T + 40) * U
        # column sums: at most 64 tokens a lane in float32, then 3 + 8 additions, then 64 bits
        near(prob, wprob, (p * rel).sum(0) / max(1, live.sum()) + 80 * U * wprob + 1e-36, "prob")
        n = max(1, live.sum())
        f = c * E * wcounts / (k * n) / n * tokens
        lse = np.abs(xl.max(1) + np.log(np.exp(xl - xl.max(1, keepdims=True)).sum(1)))[:, None]
        zt = 2 * zc / n * tokens * lse
        lerr = (T + 40 + 4 * lse) * U
        # g = p (f - sum p f) + p zt
        tol = p * (np.abs(f) + (p * f).sum(1, keepdims=True) + zt) * (rel + (p * rel).sum(1, keepdims=True) + 30 * U)
        tol += p * 2 * zc / n * tokens * lerr + HALF[dtype] * np.abs(wgrad[live]) + 1e-36
        near(grad[torch.from_numpy(live).cuda()], wgrad[live], tol, "grad")
        near(stats, wstats, np.abs(wstats) * 200 * U + zc * (2 * lse * lerr).sum() / n + 1e-30, "stats")
    else:
        assert stats.tolist() == [0, 0, 0, 0] and not prob.any()
    assert not grad[torch.from_numpy(~live).cuda()].any()
    assert op.flags() == 0


EXPERTS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 100, 128, 129, 255, 256, 257, 300, 512, 513, 777, 1024]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", EXPERTS)
def test_balance(Q, E, dtype):
    rng = np.random.default_rng(E)
    check_balance(Q, rng, 1 + E % 90, E, min(E, 1 + E % 4), dtype, 1e-3 * (E % 2), pad=E % 3)


@pytest.mark.parametrize("tokens,E,k,dtype", [(1, 8, 2, "f32"), (5000, 6, 6, "bf16"), (3001, 100, 8, "bf16"),
                                              (20011, 16, 2, "f32"), (2000, 1000, 4, "f32")])
def test_balance_tokens(Q, tokens, E, k, dtype):
    rng = np.random.default_rng(tokens)
    check_balance(Q, rng, tokens, E, k, dtype, 1e-3, index=np.int64)
    check_balance(Q, rng, tokens, E, k, dtype, 0.0, mask=None, pad=5)


def test_balance_in_place_masked_and_bad_index(Q):
    rng = np.random.default_rng(9)
    check_balance(Q, rng, 70, 37, 3, "bf16", 1e-3, pad=2, in_place=True)
    check_balance(Q, rng, 70, 37, 3, "bf16", 1e-3, mask="none")
    op = Q.BalanceLoss(3, 5, 2, "f32")
    _, counts, _, grad = op.run(torch.zeros(3, 5, device="cuda"), gpu([[0, 5], [1, 1 << 40], [4, -7]]))
    assert counts.tolist() == [1, 1, 0, 0, 1] and op.flags() == Q.FLAG_BAD_INDEX and grad.isfinite().all()


def test_balance_masked_experts(Q):
    """An expert switched off by -inf or the lowest value has probability 0 and gradient 0."""
    for dtype in ("bf16", "f32"):
        x = torch.zeros(9, 20, dtype=DT[dtype], device="cuda")
        x[:, 3] = -float("inf")
        x[:, 17] = torch.finfo(DT[dtype]).min
        chosen = gpu(np.tile([0, 5], (9, 1)))
        stats, counts, prob, grad = Q.BalanceLoss(9, 20, 2, dtype, z_coef=1e-3).run(x, chosen)
        assert prob[3] == 0 and prob[17] == 0 and not grad[:, [3, 17]].any() and grad.isfinite().all()
        near(prob[[0, 5, 19]], np.full(3, 1 / 18), 20 * U / 18)


# -- dropout -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 8), (5, 9), (1, 64), (17, 65), (9, 1025), (130, 100)])
def test_dropout(Q, rows, cols, dtype):
    """The kept elements exactly, their values to the roundings of the product and of the result."""
    rng = np.random.default_rng(cols)
    x, xd = matrix(rng, rows, cols, dtype, pad=3, lead=1)
    res, rd = matrix(rng, rows, cols, dtype, pad=1)
    seed, off = 0xDEADBEEF12345678, (1 << 33) + 5
    for p in (0.0, 0.1, 0.5, 1.0):
        op = Q.Dropout(rows, cols, dtype, p)
        keep = O.dropout_keep(rows, cols, seed, off, p)
        assert ((op.run(torch.ones_like(x), seed, off) != 0).cpu().numpy() == keep).all()
        want = O.dropout(xd, seed, off, p)
        near(op.backward(x, seed, off), want, (HALF[dtype] + 2 * U) * np.abs(want))
        both = want + rd
        near(op.run(x, seed, off, residual=res), both, HALF[dtype] * np.abs(both) * (1 + 4 * U) + 3 * U * (np.abs(want) + np.abs(rd)))
        y = x.clone()
        assert torch.equal(op.run(y, seed, off, residual=res, out=y), op.run(x, seed, off, residual=res))
        r = res.clone()
        assert torch.equal(op.run(x, seed, off, residual=r, out=r), op.run(x, seed, off, residual=res))


def test_dropout_dropped_values_reach_nothing(Q):
    x = torch.full((4, 33), float("nan"), device="cuda")
    keep = torch.from_numpy(O.dropout_keep(4, 33, 3, 4, 0.5)).cuda()
    assert torch.equal(Q.Dropout(4, 33, "f32", 0.5).run(x, 3, 4).isnan(), keep)


def test_dropout_many_blocks(Q):
    """Every workgroup of a larger tensor against the generator in tensor operations."""
    from perf import operators as P
    for rows, cols, dtype in ((3000, 1003, "bf16"), (257, 4096, "f32")):
        x = torch.ones(rows, cols, dtype=DT[dtype], device="cuda")
        keep = P._keep(rows, cols, 11 << 40, 1 << 50, 0.25, x.device)
        assert torch.equal(Q.Dropout(rows, cols, dtype, 0.25).run(x, 11 << 40, 1 << 50) != 0, keep)


def test_gradient_rows_lie_as_the_logits_do(Q):
    """A new gradient has every row at the same place within 16 bytes as the logits' row, at the least width."""
    op = Q.PolicyLoss(4, 9, dtype="bf16")
    lab, adv = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    for ld in (9, 10, 16, 17, 64):
        g = op.run(torch.zeros(4, ld, dtype=torch.bfloat16, device="cuda")[:, :9], lab, adv)[2]
        assert g.shape == (4, 9) and g.stride(1) == 1 and (g.stride(0) - ld) % 8 == 0 and 9 <= g.stride(0) <= 16


# -- strides beyond 32 bits, streams, graphs, repeatability -----------------------------------

def test_row_strides_past_32_bits(Q):
    """Rows 2^31 + 24 elements apart: byte offsets past 32 bits in the logits, the gradient and dropout."""
    far = (1 << 31) + 24
    whole = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    x = whole.as_strided((2, 3001), (far, 1))
    small = torch.randn(2, 3001, device="cuda").bfloat16()
    x.copy_(small)
    lab, f = gpu([5, 3000]), torch.ones(2, device="cuda")
    a = Q.PolicyLoss(2, 3001, "bf16").run(small, lab, f)
    b = Q.PolicyLoss(2, 3001, "bf16").run(x, lab, f, grad=x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    x.copy_(small)
    off = gpu([0, 1, 2], torch.int32)
    a = Q.PreferenceLoss(2, 1, 3001, "bf16").run(small, lab, off)
    b = Q.PreferenceLoss(2, 1, 3001, "bf16").run(x, lab, off, grad=x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    x.copy_(small)
    d = Q.Dropout(2, 3001, "bf16", 0.3)
    assert torch.equal(d.run(small, 1, 2, residual=small), d.run(x, 1, 2, residual=x, out=x))
    y = whole.as_strided((2, 300), (far, 1))
    y.copy_(small[:, :300])
    ids = gpu([[0, 1], [2, 299]])
    a = Q.BalanceLoss(2, 300, 2, "bf16").run(small[:, :300], ids)
    b = Q.BalanceLoss(2, 300, 2, "bf16").run(y, ids, grad=y)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_another_stream(Q):
    """Calls on a given stream, outputs made there; the caller's events order them."""
    s = torch.cuda.Stream()
    x = torch.randn(300, 5000, device="cuda")
    lab, f = torch.randint(0, 5000, (300,), device="cuda"), torch.randn(300, device="cuda")
    op = Q.PolicyLoss(300, 5000, "f32")
    want = op.run(x, lab, f)
    s.wait_stream(torch.cuda.current_stream())
    got = op.run(x, lab, f, stream=s)
    y = Q.Dropout(300, 5000, "f32").run(x, 1, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(y, Q.Dropout(300, 5000, "f32").run(x, 1))


def test_workspace_outlives_its_object_on_another_stream(Q):
    """An operator dropped while its call still runs on another stream: its workspace is not handed out again
    before that call has ended."""
    s = torch.cuda.Stream()
    x = torch.randn(2000, 30000, device="cuda")
    lab, off = torch.randint(0, 30000, (2000,), device="cuda"), gpu([0, 1000, 2000], torch.int32)
    want = Q.PreferenceLoss(2000, 1, 30000, "f32").run(x, lab, off)
    torch.cuda.synchronize()
    for _ in range(3):
        op = Q.PreferenceLoss(2000, 1, 30000, "f32")
        n = op.ws_bytes + 256
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = op.run(x, lab, off)
        del op
        spoiled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del spoiled


def test_graph_replays(Q):
    """All operators captured into one graph and replayed on changing inputs, eager work and synchronisation
    between the replays; dropout draws another mask at each through offset_tensor."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, vocab, E = 200, 3001, 37
    x = torch.randn(rows, vocab, device="cuda").bfloat16()
    router = torch.randn(rows, E, device="cuda")
    lab, adv = torch.randint(0, vocab, (rows,), device="cuda"), torch.randn(rows, device="cuda")
    ids = torch.randint(0, E, (rows, 2), device="cuda")
    off = gpu(np.arange(0, rows + 1, 50), torch.int32)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    make = lambda: (Q.TokenLogp(rows, vocab), Q.PolicyLoss(rows, vocab), Q.PreferenceLoss(rows, 2, vocab),
                    Q.BalanceLoss(rows, E, 2, "f32"), Q.Dropout(rows, vocab, p=0.3))

    def everything(ops):
        logp, pol, pref, bal, drop = ops
        return (logp.run(x, lab), *pol.run(x, lab, adv), *pref.run(x, lab, off), *bal.run(router, ids),
                drop.run(x, 5, 9, offset_tensor=step))
    captured, eager = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(captured)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything(captured)
    for i in range(4):
        x.copy_(torch.randn(rows, vocab, device="cuda", generator=g))
        router.copy_(torch.randn(rows, E, device="cuda", generator=g))
        step.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, everything(eager)):
            assert torch.equal(a, b), i
        assert torch.equal(outs[-1], eager[-1].run(x, 5, 9 + i))


def test_results_repeat_bit_for_bit(Q):
    x = torch.randn(1200, 7001, device="cuda").bfloat16()
    lab, adv = torch.randint(0, 7001, (1200,), device="cuda"), torch.randn(1200, device="cuda")
    off = gpu(np.linspace(0, 1200, 9), torch.int32)
    router, ids = torch.randn(9000, 60, device="cuda"), torch.randint(0, 60, (9000, 4), device="cuda")
    ops = Q.PolicyLoss(1200, 7001), Q.PreferenceLoss(1200, 4, 7001), Q.BalanceLoss(9000, 60, 4, "f32")
    run = lambda: (*ops[0].run(x, lab, adv), *ops[1].run(x, lab, off), *ops[2].run(router, ids))
    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
