"""Kernels of sampling, the embedding and the orthogonalised update that only large inputs reach.

Sampling: 512 threads a row, of more rows than compute units, each more than 1024 vectors of 16 bytes.  Embedding: past
the memory-side cache, for lookups of more than 128 MiB of rows and gradients of more than 256 MiB of rows and table.
Orthogonalised updates: X X^T, d x d products, X products, the last one and the one into the weight in tiles of 256,
with sides that end inside a tile; shares of such tiles; two steps a product.
"""
import numpy as np
import pytest
import torch

from oracle import orthogonal as O
from tests.test_gpu_objectives import DT, HALF, U, gpu, matrix, near, wide
from tests.test_gpu_tokens import check

pytestmark = pytest.mark.gpu


# -- sampling --------------------------------------------------------------------

@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 300, 9001), ("f32", 257, 5003), ("f32", 300, 20011), ("bf16", 400, 32768)])
def test_sample_rows_of_512_threads(gpu_lib, dtype, rows, vocab):
    from second_order_optimizer_amd import tokens
    rng = np.random.default_rng(rows + vocab)
    x, xd = matrix(rng, rows, vocab, dtype, pad=vocab % 5)
    u = gpu(rng.random(rows).astype(np.float32))
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 40, 0.9, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 0.95, 0.05), (0.0, 0, 1.0, 0.0),
                       (2.0, 3000, 0.99, 0.0)):
        op = tokens.Sampler(rows, vocab, dtype, temperature=t, top_k=k, top_p=p, min_p=m)
        got = op.run(x, u)
        check(got, xd, u, t, k, p, m)
        assert op.flags() == 0 and all(torch.equal(a, b) for a, b in zip(got, op.run(x, u)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_settings_ties_and_masks_of_512_threads(gpu_lib, dtype):
    """Rows of their own settings; equal logits, columns that are not allowed, rows without any and of no numbers among
    them.  The others' tokens are what they are without those rows."""
    from second_order_optimizer_amd import tokens
    rows, vocab = 320, 10007
    rng = np.random.default_rng(7)
    x, _ = matrix(rng, rows, vocab, dtype)
    x[torch.from_numpy(rng.random((rows, vocab)) < 0.3).cuda()] = -np.inf
    x[5] = gpu((rng.integers(0, 3, vocab) * 0.25).astype(np.float32)).to(DT[dtype])
    x[6] = 1.5
    x[7] = -np.inf
    xd = wide(x)
    u = gpu(rng.random(rows).astype(np.float32))
    t, p, m = (rng.choice(np.float32(v), rows).astype(np.float32) for v in
               ([0.0, 0.5, 1.0, 2.0], [0.0, 0.3, 0.9, 1.0, 1.5], [-1.0, 0.0, 0.1, 1.0, 2.0]))
    k = rng.choice([-3, 0, 1, 7, 40, 300, 10 * vocab], rows).astype(np.int32)
    op = tokens.Sampler(rows, vocab, dtype)
    got = op.run(x, u, gpu(t), gpu(k), gpu(p), gpu(m))
    check(got, xd, u, t, np.maximum(k, 0), np.clip(p, 0, 1), np.clip(m, 0, 1))
    assert op.flags() == 0 and got[0][7] == -1 and got[2][7] == 0
    x[8, vocab - 1], x[9, 0] = np.nan, np.inf
    again = op.run(x, u, gpu(t), gpu(k), gpu(p), gpu(m))
    assert op.flags() == gpu_lib.FLAG_NONFINITE and (again[0][8:10] == -1).all()
    keep = [r for r in range(rows) if r not in (8, 9)]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(3, 700), (3, 5000), (3, 70000), (300, 9001)])
def test_sample_tokens_among_equal_logits(gpu_lib, rows, vocab, dtype):
    """Rows of equal logits, and of a run of equal ones above the others: kept is a whole number n that the settings
    say, and the token column floor(u n) of the run.  The draws lie in the middle between two columns."""
    from second_order_optimizer_amd import tokens
    rng = np.random.default_rng(vocab)
    run = np.sort(rng.choice(vocab, vocab // 3, replace=False))
    for columns, below in ((np.arange(vocab), 0.0), (run, -60.0)):
        x = np.full((rows, vocab), below, np.float32)
        x[:, columns] = 0.0
        for k, p in ((13, 1.0), (0, 0.40001), (len(columns) // 2 + 1, 0.70003), (len(columns) - 1, 1.0)):
            n = min(k, len(columns)) if k else len(columns)
            n = int(np.ceil(p * n)) if p < 1 else n
            at = np.floor(rng.random(rows) * n).astype(np.int64)
            u = ((at + 0.5) / n).astype(np.float32)
            token, logp, kept = tokens.Sampler(rows, vocab, dtype, top_k=k, top_p=p).run(gpu(x).to(DT[dtype]), gpu(u))
            assert kept.tolist() == [n] * rows and token.tolist() == columns[at].tolist(), (k, p, below)
            near(logp, np.full(rows, -np.log(len(columns))), 2 * U * np.log(vocab))


# -- embedding -------------------------------------------------------------------

@pytest.mark.parametrize("dtype,table_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_embedding_past_the_cache(gpu_lib, dtype, table_dtype):
    """Rows and table of more than either kernel's share of the cache; the last columns are no whole vector."""
    from second_order_optimizer_amd import tokens
    gen = torch.Generator(device="cuda").manual_seed(3)
    width, scale = 1029, 1.5
    n, vocab = (70000, 70001) if dtype == "bf16" else (35000, 100003)
    rand = lambda *s, dt: torch.randn(*s, generator=gen, device="cuda").to(DT[dt])  # noqa: E731
    table, dy = rand(vocab, width + 3, dt=table_dtype)[:, 1:width + 1], rand(n, width + 2, dt=dtype)[:, 2:]
    ids = (torch.rand(n, generator=gen, device="cuda") ** 3 * vocab).long().clamp(max=vocab - 1)
    ids[::50] = -1
    there = ids >= 0
    assert n * width * DT[dtype].itemsize > 1 << 27
    assert n * width * DT[dtype].itemsize + vocab * width * DT[table_dtype].itemsize > 1 << 28
    op = tokens.Embedding(n, vocab, width, dtype, table_dtype, scale)
    y = op.run(table, ids)
    want = torch.where(there[:, None], table[ids.clamp(min=0)].float() * scale, 0.0).to(DT[dtype])      # one product, one rounding
    assert torch.equal(y, want)
    room = torch.full((n, width + 5), 7.0, device="cuda").to(DT[dtype])
    op.run(table, ids, out=room[:, 2:width + 2])
    assert torch.equal(room[:, 2:width + 2], want) and (room[:, :2] == 7).all() and (room[:, width + 2:] == 7).all()
    del room, y, want
    grad, counts = op.backward(dy, ids)
    assert torch.equal(counts.long(), torch.bincount(ids[there], minlength=vocab))
    old = rand(vocab, width + 1, dt=table_dtype)
    into = old.clone()
    op.backward(dy, ids, grad=into[:, :width], accumulate=True)
    assert torch.equal(into[:, width], old[:, width])
    for c in range(0, width, 129):                        # the exact sums of some columns at a time
        part = slice(c, min(c + 129, width))
        sums, sizes = (torch.zeros(vocab, part.stop - c, dtype=torch.float64, device="cuda") for _ in range(2))
        d = dy[there, part].double() * scale
        sums.index_add_(0, ids[there], d)
        sizes.index_add_(0, ids[there], d.abs())
        # n terms in float32, the scale and one rounding to the table's type
        tol = (counts[:, None] + 3).double() * U * sizes + HALF[table_dtype] * sums.abs()
        assert ((grad[:, part].double() - sums).abs() <= tol).all(), c
        total = sums + old[:, part].double()
        tol = tol - HALF[table_dtype] * sums.abs() + (HALF[table_dtype] + 2 * U) * total.abs() + U * sizes
        assert ((into[:, part].double() - total).abs() <= tol).all(), c
        none = counts == 0
        assert torch.equal(into[none, part], old[none, part])
    assert op.flags() == 0


# -- orthogonalised update ---------------------------------------------------------

def iterated(x, steps=5, eps=1e-7, dtype=torch.float64):
    """O of a matrix in 64 bits (or in float32 products) on the GPU, from the side that keeps its products small."""
    x = (x.double() / (x.double().norm() + eps)).to(dtype)
    right = x.shape[0] > x.shape[1]
    for a, b, c in O.triples(O.COEFS, steps).tolist():
        g = x.t().contiguous() @ x if right else x @ x.t().contiguous()
        q = b * g + c * (g @ g)
        x = a * x + (x @ q if right else q @ x)
    return x.double()


def close(got, x, products, extra=0.0):
    """Off by no more than documented: HALF 1.2e-3 for noise; FULL what float32 products are, of sums of another order
    (3 times those, and 1e-6).

    Single rows and columns: one that goes with a row of X X^T is off mostly along itself, by one number, the rounding
    of its diagonal sums.  These are random walks of that many additions: of the rows (their mean square is the whole's)
    the farthest of 6000 is 6 deviations out with a chance of 10^-5, and a deviation is up to sqrt(2) of the rms, as the
    additions that follow the largest term of (A A)_ii, whose roundings weigh the most, are all d for the first row and
    none for the last: 8.5 times the whole's.
    """
    want = iterated(x)
    tol = O.DOCUMENTED["noise"][0]
    if products == "full":
        tol = 3 * float((iterated(x, dtype=torch.float32) - want).norm() / want.norm()) + 1e-6
    tol += extra
    off = got.double() - want
    whole = float(off.norm() / want.norm())
    print(tuple(x.shape), products, f"{whole:.2e} of {tol:.2e}")
    assert whole <= tol
    for d in (0, 1):
        assert float((off.norm(dim=d) / want.norm(dim=d)).max()) <= 8.5 * tol, d
    return want


@pytest.mark.parametrize("products", ["half", "full"])
@pytest.mark.parametrize("rows,cols", [(4000, 4090), (4090, 4000), (4096, 6000), (6000, 4096), (2570, 20001)])
def test_update_in_tiles_of_256(gpu_lib, rows, cols, products):
    from second_order_optimizer_amd import orthogonal as M
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    op = M.Orthogonal(rows, cols, dtype="f32", products=products)
    got = op.run(x)
    close(got, x, products)
    assert op.flags() == 0 and torch.equal(got, op.run(x))
    xb = x.bfloat16()
    close(M.Orthogonal(rows, cols, dtype="bf16", products=products).run(xb), xb, products, HALF["bf16"])


@pytest.mark.parametrize("products", ["half", "full"])
def test_step_in_tiles_of_256(gpu_lib, products):
    """Two layers in one launch, one way round and the other, from weights of zeros with a rate of 1 (the update alone),
    and then a step of weights that are there."""
    from second_order_optimizer_amd import orthogonal as M
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    shapes = [(4090, 3990), (2559, 4091)]
    g, bg = [rand(*s) for s in shapes], [rand(s[0]) for s in shapes]
    w, m, b, bm = ([torch.zeros_like(t) for t in v] for v in (g, g, bg, bg))
    op = M.OrthogonalStep(w, m, b, bm, products=products, scale="none")
    op.run(g, bg, lr=1.0, momentum=0.5)
    for i in range(2):
        close(-w[i], 1.5 * g[i], products, U)                # U = g + mu m with m = g
        assert torch.equal(m[i], g[i]) and torch.equal(b[i], -bg[i]) and torch.equal(bm[i], bg[i])
    old = [t.clone() for t in w]
    op.run(g, bg, lr=0.25, momentum=0.0, weight_decay=0.5)
    for i in range(2):
        # the weight's part: decay, product and sum are rounded, against an update of at most the weight's size
        close((0.875 * old[i].double() - w[i].double()) / 0.25, g[i], products, 16 * U)
    assert op.flags() == 0


@pytest.mark.parametrize("rows,cols,dtype", [(130, 300, "bf16"), (130, 300, "f32"), (2047, 1000, "f32"), (1024, 8192, "f32"), (50, 900, "f32"),
                                             (4000, 4090, "bf16"), (16384, 4096, "bf16"), (4096, 6000, "f32")])
def test_update_after_others(gpu_lib, rows, cols, dtype):
    """What a workspace holds of earlier calls, of numbers and of none, is in no later result."""
    from second_order_optimizer_amd import orthogonal as M
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, other = (torch.randn(rows, cols, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    op = M.Orthogonal(rows, cols, dtype=dtype)
    want = M.Orthogonal(rows, cols, dtype=dtype).run(x)
    for before in (other, torch.full_like(other, np.nan), torch.full_like(other, 3e38)):
        op.run(before)
        assert torch.equal(op.run(x), want)


def test_rows_after_others(gpu_lib):
    """The same of the embedding's gradient and of sampling in parts."""
    from second_order_optimizer_amd import tokens
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n in (5000, 70000):
        emb, fresh = (tokens.Embedding(n, 3001, 130, "f32") for _ in range(2))
        sets = [(torch.randn(n, 130, generator=gen, device="cuda"), (torch.rand(n, generator=gen, device="cuda") ** 2 * 3001).long()) for _ in range(2)]
        want = fresh.backward(*sets[0])
        for before in (sets[1], (torch.full_like(sets[1][0], np.nan), torch.full_like(sets[1][1], 7)), (sets[1][0], torch.full_like(sets[1][1], -1))):
            emb.backward(*before)
            assert all(torch.equal(a, b) for a, b in zip(emb.backward(*sets[0]), want))
    sampler, fresh = (tokens.Sampler(3, 70000, top_k=50, top_p=0.9) for _ in range(2))
    x, other = (torch.randn(3, 70000, generator=gen, device="cuda").bfloat16() * 3 for _ in range(2))
    u = torch.rand(3, generator=gen, device="cuda")
    want = fresh.run(x, u)
    for before in (other, torch.full_like(other, np.nan), torch.full_like(other, -np.inf), torch.zeros_like(other)):
        sampler.run(before, u)
        assert all(torch.equal(a, b) for a, b in zip(sampler.run(x, u), want))
