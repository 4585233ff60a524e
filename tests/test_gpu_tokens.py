"""Sampling and the embedding on the GPU against the float64 oracle.

Sampling: weights are whole multiples of 2^-44 of the largest, each off by half
of one and by 2^-46 of itself, so that sums of V of them, and with them the
draw and top_p's border, are off by at most V 2^-45 + 2^-46 of the kept sum.
The oracle says how far each decision was from another answer; rows nearer
than MARGIN may keep one column more or less, and are not asked for their token.
Drawn rows hardly ever are; equal weights may be by design (0.4501 of 70000
equal columns are 31507 exactly: the border of top_p is an edge).
logp: the tolerance of tests/test_gpu_objectives.py, whose terms these are.

Embedding: a row is scaled in float32 and rounded, u + HALF of itself; a sum of
n terms in float32 is off by at most n u of the sum of their sizes, whatever
the order, and rounded once.
"""
import numpy as np
import pytest
import torch

from oracle import tokens as O
from tests.test_gpu_objectives import DT, HALF, U, gpu, logp_tolerance, matrix, near, wide

pytestmark = pytest.mark.gpu
MARGIN = 2e-8


@pytest.fixture()
def T(gpu_lib):
    from second_order_optimizer_amd import tokens
    return tokens


def check(got, x, u, t=1.0, k=0, p=1.0, m=0.0, clear_rows=0.9):
    """Token, log-probability and count of every row against the oracle."""
    token, logp, kept = (v.cpu().numpy() for v in got)
    want, wlogp, wkept, margin = O.sample(x, u.cpu().numpy(), t, k, p, m)
    clear = margin > MARGIN
    assert clear.mean() >= clear_rows and (np.abs(kept - wkept) <= 1).all()
    assert (token[clear] == want[clear]).all(), (np.flatnonzero(clear & (token != want))[:4], token[:8], want[:8])
    assert (kept[clear] == wkept[clear]).all(), (np.flatnonzero(clear & (kept != wkept))[:4], kept[:8], wkept[:8])
    ts = np.broadcast_to(np.asarray(t, np.float64), (len(want),))
    for r in np.flatnonzero(clear & (want >= 0)):
        s = 1.0 if ts[r] < 1e-6 else 1.0 / ts[r]
        live = x[r:r + 1][:, x[r] > -np.inf]
        label = np.array([(x[r][:want[r]] > -np.inf).sum()])
        near(logp[r:r + 1], wlogp[r:r + 1], logp_tolerance(live, label, s) + 2e-14, r)
    assert (logp[want < 0] == 0).all()


# registers and workgroups change at 4, 16, 64, 128 and 256 KB a row
VOCABS = [1, 2, 7, 8, 9, 255, 1000, 2049, 4100, 8191, 16387, 33001, 65536, 70001, 131072, 140003]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_sample(T, vocab, dtype):
    rng = np.random.default_rng(vocab)
    rows = 3
    x, xd = matrix(rng, rows, vocab, dtype, pad=vocab % 4, lead=vocab % 2 if vocab % 4 else 0)
    u = gpu(rng.random(rows).astype(np.float32))
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05),
                       (0.8, 50, 0.8, 0.02), (0.0, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.0), (2.0, 3000, 0.99, 0.0)):
        op = T.Sampler(rows, vocab, dtype, temperature=t, top_k=k, top_p=p, min_p=m)
        check(op.run(x, u), xd, u, t, k, p, m)
        assert op.flags() == 0


@pytest.mark.parametrize("rows,vocab,dtype", [(700, 1000, "f32"), (2000, 50, "bf16"), (300, 5003, "bf16")])
def test_sample_many_rows_with_their_own_settings(T, rows, vocab, dtype):
    rng = np.random.default_rng(rows)
    x, xd = matrix(rng, rows, vocab, dtype, pad=3)
    u = gpu(rng.random(rows).astype(np.float32))
    t, p, m = (rng.choice(np.float32(v), rows).astype(np.float32) for v in
               ([0.0, 0.5, 1.0, 2.0], [0.0, 0.3, 0.9, 1.0, 1.5], [-1.0, 0.0, 0.1, 1.0, 2.0]))
    k = rng.choice([-3, 0, 1, 7, 40, 10 * vocab], rows).astype(np.int32)
    got = T.Sampler(rows, vocab, dtype).run(x, u, gpu(t), gpu(k), gpu(p), gpu(m))
    check(got, xd, u, t, np.maximum(k, 0), np.clip(p, 0, 1), np.clip(m, 0, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 700, 5000, 70000])
def test_sample_ties(T, vocab, dtype):
    """Equal logits, in all of a row and in runs: taken by rising number, where a border lies among them too."""
    rng = np.random.default_rng(vocab)
    x = np.zeros((5, vocab), np.float32)
    x[1] = -3.0
    x[2] = rng.integers(-1, 2, vocab)
    x[3] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)
    x[4] = rng.integers(0, 3, vocab) * 0.25
    xg = gpu(x).to(DT[dtype])
    xd = wide(xg)
    u = gpu(np.float32([0.0, 0.31, 0.72, 0.11, 0.999]))
    for k, p in ((13, 1.0), (0, 0.4501), (vocab // 2 + 1, 0.7003), (vocab - 1, 1.0)):
        check(T.Sampler(5, vocab, dtype, top_k=k, top_p=p).run(xg, u), xd, u, 1.0, k, p, clear_rows=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_masks_and_extremes(T, dtype):
    """Columns of minus infinity, of the type's lowest value, a row without any column, huge and equal logits."""
    rng = np.random.default_rng(5)
    vocab = 3001
    x, _ = matrix(rng, 8, vocab, dtype)
    low = torch.finfo(DT[dtype]).min
    x[0, torch.from_numpy(rng.random(vocab) < 0.9).cuda()] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, 2999] = low
    x[3, 1:] = low
    x[4] = low
    x[5] *= 1e30
    x[6] = torch.finfo(DT[dtype]).max
    x[6, ::2] = low
    xd = wide(x)
    u = gpu(np.float32([0.2, 0.5, 0.5, 0.9999, 0.5001, 0.3, 0.7002, 0.1]))
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.9, 20, 0.9, 0.0), (1.0, 0, 0.7777, 0.01), (0.0, 0, 1.0, 0.0),
                       (1e-5, 0, 1.0, 0.0), (1e9, 0, 1.0, 0.0)):
        op = T.Sampler(8, vocab, dtype, temperature=t, top_k=k, top_p=p, min_p=m)
        with np.errstate(over="ignore", invalid="ignore"):
            # rows 4 and 6 are equal columns: 0.9 of 20 of them is an edge
            check(op.run(x, u), xd, u, t, k, p, m, clear_rows=0.75)
        assert op.flags() == 0


def test_sample_flags(T, gpu_lib):
    """Rows that are no numbers, draws outside [0, 1) and settings that are none: token -1, and nothing else."""
    rng = np.random.default_rng(6)
    x, xd = matrix(rng, 8, 500, "f32")
    u = torch.rand(8, device="cuda")
    op = T.Sampler(8, 500, "f32", top_k=20)
    y = x.clone()
    y[1, 3], y[2, 499] = np.nan, np.inf
    token, logp, kept = op.run(y, u)
    assert op.flags(clear=True) == gpu_lib.FLAG_NONFINITE
    assert token[[1, 2]].tolist() == [-1, -1] and kept[[1, 2]].tolist() == [0, 0] and logp[[1, 2]].tolist() == [0, 0]
    same = op.run(x, u)[0]
    keep = [0, 3, 4, 5, 6, 7]
    assert op.flags() == 0 and (same[keep] == token[keep]).all() and (same >= 0).all()
    bad = u.clone()
    bad[0], bad[1], bad[2] = 1.0, -0.5, np.nan
    assert (op.run(x, bad)[0][:3] == -1).all() and op.flags(clear=True) == 4
    t = torch.ones(8, device="cuda")
    t[4], t[5] = -1.0, np.nan
    assert (op.run(x, u, temperature=t)[0][4:6] == -1).all() and op.flags(clear=True) == 4
    assert (op.run(x, u, top_p=t)[0] == -1).tolist() == [False] * 5 + [True] + [False] * 2 and op.flags(clear=True) == 4


def test_sample_draws_the_distribution(T):
    """Evenly spread draws of one row take every kept column as often as its probability says, to one draw."""
    n = 1 << 14
    x = torch.linspace(-2, 2, 37, device="cuda").flip(0).expand(n, 37).contiguous()
    u = (torch.arange(n, device="cuda").float() + 0.5) / n
    token, _, kept = T.Sampler(n, 37, "f32", top_p=0.9).run(x, u)
    w = np.exp(wide(x[0]))
    k = int(kept[0])
    p = np.where(np.arange(37) < k, w, 0) / w[:k].sum()
    assert np.abs(np.bincount(token.cpu().numpy(), minlength=37) - n * p).max() <= 1.01


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 65536), (2, 65541), (5, 80003), (16, 131072), (17, 65600), (3, 65535)])
def test_sample_rows_in_parts(T, rows, vocab, dtype):
    """Few rows, several workgroups each, and what sends a row back to one: settings of its own, ties, masks by the
    part, values that are no numbers."""
    rng = np.random.default_rng(vocab)
    x, xd = matrix(rng, rows, vocab, dtype, pad=vocab % 4)
    u = gpu(rng.random(rows).astype(np.float32))
    for t, k, p, m in ((0.8, 50, 0.95, 0.0), (1.0, 64, 1.0, 0.0), (1.0, 65, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.5, 1, 0.5, 0.1),
                       (1.0, 7, 1.0, 0.3), (1e4, 33, 0.8, 0.0)):
        op = T.Sampler(rows, vocab, dtype, temperature=t, top_k=k, top_p=p, min_p=m)
        check(op.run(x, u), xd, u, t, k, p, m)
        assert op.flags() == 0
    t, p, m = (rng.choice(np.float32(v), rows).astype(np.float32) for v in
               ([0.0, 0.5, 1.0, 2.0], [0.0, 0.3, 0.9, 1.0, 1.5], [-1.0, 0.0, 0.1, 1.0, 2.0]))
    k = rng.choice([-3, 0, 1, 7, 40, 64, 65, 10 * vocab], rows).astype(np.int32)
    op = T.Sampler(rows, vocab, dtype)
    check(op.run(x, u, gpu(t), gpu(k), gpu(p), gpu(m)), xd, u, t, np.maximum(k, 0), np.clip(p, 0, 1), np.clip(m, 0, 1))
    op = T.Sampler(rows, vocab, dtype, top_k=40)
    check(op.run(x, u, gpu(t), None, gpu(p), gpu(m)), xd, u, t, 40, np.clip(p, 0, 1), np.clip(m, 0, 1))
    # all but a few columns masked: parts without any, and fewer left than top_k
    y = torch.full_like(x, float("-inf"))
    y[:, 3:vocab:vocab // 7] = x[:, 3:vocab:vocab // 7]
    few = T.Sampler(rows, vocab, dtype, top_k=50, top_p=0.9)
    check(few.run(y, u), wide(y), u, 1.0, 50, 0.9)
    y[:, vocab // 2:] = float("-inf")
    y[:, :9] = 2.0                                                     # equal ones, all in the first part
    check(few.run(y, u), wide(y), u, 1.0, 50, 0.9)
    y.fill_(1.0)                                                       # more equal ones than a list holds
    token, _, kept = T.Sampler(rows, vocab, dtype, top_k=40).run(y, u)
    assert kept.tolist() == [40] * rows and token.tolist() == [int(float(v) * 40) for v in u.cpu().numpy().astype(np.float64)]
    y[0] = float("-inf")
    y[-1, vocab - 1] = float("nan")
    token, logp, kept = few.run(y, u)
    bad = sorted({0, rows - 1})
    assert (token[bad] == -1).all() and (logp[bad] == 0).all() and (kept[bad] == 0).all() and (token[1:-1] >= 0).all()
    assert few.flags() != 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_of_the_most_equal_columns(T, dtype):
    """2^20 - 1 columns of the largest weight fill the 64 bits of their sum."""
    vocab = (1 << 20) - 1
    with pytest.raises(RuntimeError):
        T.Sampler(3, vocab + 1, dtype)
    x = torch.zeros(3, vocab, dtype=DT[dtype], device="cuda")
    u = gpu(np.array([0.0, 0.61803, 1 - 2.0 ** -24], np.float32))
    token, logp, kept = T.Sampler(3, vocab, dtype).run(x, u)
    assert token.tolist() == [int(float(v) * vocab) for v in u.cpu().numpy().astype(np.float64)] and (kept == vocab).all()
    near(logp, np.full(3, -np.log(vocab)), 2 * U * np.log(vocab))
    token, _, kept = T.Sampler(3, vocab, dtype, top_p=0.7001).run(x, u)
    n = int(np.ceil(0.7001 * vocab))
    assert kept.tolist() == [n] * 3 and token.tolist() == [int(float(v) * n) for v in u.cpu().numpy().astype(np.float64)]


def test_sample_of_no_rows_and_repeats(T):
    assert [v.numel() for v in T.Sampler(0, 9, "f32").run(torch.empty(0, 9, device="cuda"), torch.empty(0, device="cuda"))] == [0, 0, 0]
    x = torch.randn(64, 9000, device="cuda").bfloat16()
    u = torch.rand(64, device="cuda")
    op = T.Sampler(64, 9000, top_p=0.9)
    first = op.run(x, u)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, op.run(x, u)))


# -- embedding -----------------------------------------------------------------

def ids_of(rng, n, vocab, kind):
    if kind == "one":
        return np.full(n, vocab // 2)
    ids = rng.integers(0, vocab, n) if kind == "even" else np.minimum(np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    return np.where(rng.random(n) < 0.05, -1 - rng.integers(0, 9, n), ids)


def check_embedding(T, rng, tokens, vocab, width, dtype, table_dtype, kind, scale=1.0, int64=True, pad=0):
    table, td = matrix(rng, vocab, width, table_dtype, pad=pad)
    dy, dyd = matrix(rng, tokens, width, dtype, pad=2 * pad, lead=pad)
    ids = ids_of(rng, tokens, vocab, kind)
    op = T.Embedding(tokens, vocab, width, dtype, table_dtype, scale)
    idg = gpu(ids.astype(np.int64 if int64 else np.int32))
    want = O.lookup(td, ids, scale)
    near(op.run(table, idg), want, (HALF[dtype] + 2 * U) * np.abs(want), "rows")
    grad, counts = op.backward(dy, idg)
    want, size, n = O.lookup_grad(dyd, ids, vocab, scale)
    assert grad.dtype == DT[table_dtype] and (counts.cpu().numpy() == n).all()
    tol = (n[:, None] + 2) * U * size + (HALF[table_dtype] + U) * np.abs(want)
    near(grad, want, tol, "grad")
    again = op.backward(dy, idg)[0]
    assert torch.equal(grad, again)
    old, oldd = matrix(rng, vocab, width, table_dtype, pad=pad)
    out = old.clone() if pad == 0 else old
    op.backward(dy, idg, grad=out, accumulate=True)
    near(out, want + oldd, tol + (HALF[table_dtype] + 2 * U) * np.abs(want + oldd), "accumulated")
    assert (wide(out)[n == 0] == oldd[n == 0]).all()
    assert op.flags() == 0


@pytest.mark.parametrize("tokens", [1, 2, 63, 128, 129, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("vocab", [1, 2, 64, 65, 511, 512, 3001])
def test_embedding_lengths(T, tokens, vocab):
    rng = np.random.default_rng(tokens * 7919 + vocab)
    check_embedding(T, rng, tokens, vocab, 9, "f32", "f32", rng.choice(["even", "falling", "one"]), 1.5, tokens % 2 == 0)


@pytest.mark.parametrize("width", [1, 3, 4, 7, 8, 64, 255, 256, 257, 511, 1025, 2049, 4100])
@pytest.mark.parametrize("dtype,table_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_embedding_widths_and_types(T, width, dtype, table_dtype):
    rng = np.random.default_rng(width)
    check_embedding(T, rng, 300, 70, width, dtype, table_dtype, "falling", 8.0, pad=width % 3)


@pytest.mark.parametrize("tokens,vocab,kind", [(70000, 50, "even"), (300000, 300000, "falling"), (40000, 5, "one"),
                                               (263000, 1000, "falling"), (20000, 150000, "even")])
def test_embedding_large(T, tokens, vocab, kind):
    """Tokens with thousands of rows, joined from tiles; more tiles than a sort has; three digits."""
    check_embedding(T, np.random.default_rng(vocab), tokens, vocab, 5, "f32", "f32", kind)


def test_embedding_order_of_sums(T):
    """A token's rows are added by their positions: a value that only the order saves is there."""
    dy = torch.zeros(400, 8, device="cuda")
    dy[0], dy[1], dy[2] = 2.0 ** 30, -2.0 ** 30, 1.0
    dy[300:] = 0.25
    ids = torch.full((400,), 3, device="cuda")
    grad, counts = T.Embedding(400, 7, 8, "f32").backward(dy, ids)
    assert (grad[3] == 26.0).all() and counts.tolist() == [0, 0, 0, 400, 0, 0, 0]


def test_embedding_bad_ids(T):
    """Tokens past the table: rows of zeros, nothing added, flagged."""
    table = torch.randn(10, 20, device="cuda")
    ids = torch.tensor([3, 10, -1, 1 << 40, 9], device="cuda")
    op = T.Embedding(5, 10, 20, "f32")
    y = op.run(table, ids)
    assert op.flags(clear=True) == 4 and (y[[1, 2, 3]] == 0).all() and torch.equal(y[[0, 4]], table[[3, 9]])
    grad, counts = op.backward(torch.ones(5, 20, device="cuda"), ids)
    assert op.flags(clear=True) == 4 and counts.sum() == 2 and grad.sum() == 40


def test_embedding_of_nothing(T):
    op = T.Embedding(0, 6, 9, "f32")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert op.run(torch.ones(6, 9, device="cuda"), none).shape == (0, 9)
    grad, counts = op.backward(torch.empty(0, 9, device="cuda"), none)
    assert (grad == 0).all() and (counts == 0).all()


def test_embedding_autograd(T):
    """The node's gradient is the formula's, adds up over uses of one table, and agrees with differences."""
    table = torch.randn(30, 12, device="cuda", requires_grad=True)
    ids = torch.tensor([4, 4, 0, -1, 29], device="cuda")
    op = T.Embedding(5, 30, 12, "f32", scale=2.0)
    w = torch.randn(5, 12, device="cuda")
    y = op.run(table, ids)
    ((op.run(table, ids) * w).sum() + y.square().sum()).backward()
    want = torch.zeros(30, 12, dtype=torch.float64)
    for t, v in enumerate(ids.tolist()):
        if v >= 0:
            want[v] += 2 * w[t].double().cpu() + 8 * table[v].detach().double().cpu()
    near(table.grad, want.numpy(), 16 * U * (np.abs(want.numpy()) + 40))
    with torch.no_grad():
        step = torch.zeros_like(table)
        step[4, 5] = 1 / 64
        diff = (op.run(table + step, ids) - op.run(table - step, ids)).double().mul(32)[:, 5] * w[:, 5].double()
    assert abs(float(diff.sum()) - 2 * float(w[0, 5] + w[1, 5])) < 1e-4
    with pytest.raises(Exception):
        op.run(table, ids, out=torch.empty(5, 12, device="cuda"))
    with torch.no_grad():
        out = torch.empty(5, 12, device="cuda")
        assert op.run(table, ids, out=out) is not None and torch.equal(out, y)


def test_captured_and_replayed(T):
    """Both operators in one graph, replayed on other inputs with eager work in between."""
    rng = np.random.default_rng(9)
    rows, vocab, width = 300, 1003, 96
    logits, u = torch.empty(rows, vocab, device="cuda"), torch.empty(rows, device="cuda")
    table = torch.randn(vocab, width, device="cuda")
    dy = torch.randn(rows, width, device="cuda")
    sampler, emb = T.Sampler(rows, vocab, "f32", top_k=30, top_p=0.9), T.Embedding(rows, vocab, width, "f32")

    def go(s, e):
        token, logp, kept = s.run(logits, u)
        return (token, logp, kept, e.run(table, token), *e.backward(dy, token))

    logits.normal_(), u.uniform_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(sampler, emb)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(sampler, emb)
    other = T.Sampler(rows, vocab, "f32", top_k=30, top_p=0.9), T.Embedding(rows, vocab, width, "f32")
    for _ in range(4):
        logits.copy_(gpu(rng.normal(size=(rows, vocab)).astype(np.float32)) * 3)
        u.copy_(gpu(rng.random(rows).astype(np.float32)))
        graph.replay()
        want = go(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_on_another_stream(T):
    x, u = torch.randn(50, 2000, device="cuda"), torch.rand(50, device="cuda")
    op = T.Sampler(50, 2000, "f32", top_p=0.8)
    want = op.run(x, u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = op.run(x, u, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
