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


def test_outputs_on_memory_that_is_read():
    """What is written may lie beside what is read, between its rows as well, and nowhere on it."""
    op = T.Embedding(4, 8, 16, dtype="f32", device="cpu")
    room, ids = torch.zeros(4000), torch.zeros(4, dtype=torch.int64)
    table, wide, dy = room[:128].view(8, 16), room[1000:1000 + 8 * 40].view(8, 40), torch.zeros(4, 16)
    at = lambda n: room[n:n + 64].view(4, 16)  # noqa: E731
    for out in (at(0), at(64), at(16), at(127), at(3), wide[:4, :16], wide[4:, 8:24], wide[:4, 0:16]):
        base = table if out.data_ptr() < wide.data_ptr() else wide[:, 0:16]
        refused(A, op.run, base, ids, out=out)
    for out in (at(128), at(500), wide[:4, 16:32], wide[4:, 24:40]):
        refused(U, op.run, wide[:, 0:16] if out.data_ptr() >= wide.data_ptr() else table, ids, out=out)
    refused(U, op.run, wide[:, 24:40], ids, out=wide[:4, 0:16])
    refused(A, op.run, table, room[2000:2008].view(torch.int64), out=at(2005))
    for bad, ok in ((at(0), at(128)), (at(64), at(900))):
        refused(A, op.backward, bad, ids, grad=table)
        refused(U, op.backward, ok, ids, grad=table)
    refused(A, op.backward, wide[:4, 10:26], ids, grad=wide[:, 0:16], accumulate=True)
    refused(U, op.backward, wide[:4, 16:32], ids, grad=wide[:, 0:16], accumulate=True)
    refused(A, op.backward, dy, room[2000:2008].view(torch.int64), grad=room[1900:2028].view(8, 16))
    none = T.Embedding(0, 8, 16, dtype="f32", device="cpu")
    refused(U, none.run, table, ids[:0], out=table[:0])


@pytest.mark.parametrize("fn,over", [("lookup", dict(y=0x10000 + 508)), ("lookup", dict(y=0x30000 + 30)), ("lookup", dict(y=0x10020, table_ld=24, y_ld=48)),
                                     ("grad", dict(y=0x10000 + 500)), ("grad", dict(counts=0x10000)), ("grad", dict(counts=0x20000)),
                                     ("grad", dict(counts=0x30000)), ("grad", dict(ids=0x10000))])
def test_shared_memory_at_the_c_entries(lib, fn, over):
    from tests.test_tokens_abi import call, embedding
    assert call(getattr(lib, "kfac_embedding_" + fn), embedding(**over)) == A


def test_update_beside_and_on_its_input(lib):
    """out: x itself with its strides, or memory that it has no part of."""
    op = M.Orthogonal(4, 8, batch=2, dtype="f32", device="cpu")
    room = torch.zeros(3, 10, 20)
    x = room[:2, 2:6, 4:12]
    for out in (x, room[:2, 2:6, 12:20], room[:2, 6:10, 4:12], torch.zeros(2, 4, 8)):
        refused(U, op.run, x, out=out)
    for out in (room[:2, 3:7, 4:12], room[:2, 2:6, 5:13], room[1:, 2:6, 4:12], room[:2, 2:6, 0:8], room.view(-1)[44:108].view(2, 4, 8)):
        refused(A, op.run, x, out=out)
    one = M.Orthogonal(4, 8, dtype="f32", device="cpu")
    refused(A, one.run, room[0, :4, :8], out=room[0, 1:5, :8])
    refused(U, one.run, room[0, :4, :8], out=room[0, 4:8, :8])
    refused(U, one.run, room[0, :4, :8], out=room[:1, :4, :8])              # itself, as a batch of one
    from tests.test_tokens_abi import how, matrix, orthogonalize
    for over in (dict(y=0x10004), dict(y=0x10000 + 4 * (70 * 200 - 1)), dict(y=0x10000 - 4 * (70 * 200 - 1)), dict(y=0x10000 + 4 * 7000)):
        assert orthogonalize(lib, matrix(**over), how()) == A, over


def test_overlap_against_every_byte(tmp_path):
    """csrc/overlap.h on small matrices says what their bytes say."""
    import itertools
    import shutil
    import subprocess
    if not shutil.which("g++"):
        pytest.skip("g++ not installed")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text('#include <cstdio>\n#include <set>\n#include "%s"\n' % os.path.join(root, "second_order_optimizer_amd", "csrc", "overlap.h") + """
int main() {
  long long at, run, rows, ld, mats, stride;
  kfac::Lines l[2];
  for (;;) {
    std::set<long long> bytes;
    bool shared = false;
    for (int i = 0; i < 2; ++i) {
      if (std::scanf("%lld %lld %lld %lld %lld %lld", &at, &run, &rows, &ld, &mats, &stride) != 6) return 0;
      l[i] = kfac::lines_of(reinterpret_cast<void*>(at), run, rows, ld, mats, stride);
      for (long long m = 0; m < mats; ++m)
        for (long long r = 0; r < rows; ++r)
          for (long long c = 0; c < run; ++c) {
            const long long b = at + m * stride + r * ld + c;
            if (i) shared |= bytes.count(b) != 0;
            else bytes.insert(b);
          }
    }
    std::printf("%d %d\\n", shared, kfac::overlap(l[0], l[1]));
  }
}
""")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    rng = np.random.default_rng(0)
    cases = []
    for _ in range(4000):
        pair = []
        for _ in range(2):
            run, rows, mats = (int(rng.integers(0, n)) for n in (7, 5, 3))
            ld = run + int(rng.integers(0, 9))
            pair.append((1000 + int(rng.integers(0, 60)), run, rows, ld, mats, rows * ld + int(rng.integers(0, 9))))
        cases.append(pair)
    for a, b, at in itertools.product(range(1, 5), range(1, 5), range(0, 80, 3)):      # of one matrix of 11 columns
        cases.append([(1000, a, 4, 11, 1, 0), (1000 + at, b, 3, 11, 1, 0)])
    text = "\n".join(" ".join(map(str, v)) for pair in cases for v in pair)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for pair, line in zip(cases, out):
        shared, said = line.split()
        assert said == shared, pair
    assert any(line == "0 0" for line in out) and any(line == "1 1" for line in out)


@pytest.mark.gpu
def test_capture_beside_a_graph_of_another_stream(gpu_lib):
    """What the refusal of a captured lookup advises: an eager graph of the same table, made on a stream of its own, may
    live while a lookup and its backward pass are captured; replays with eager work between them."""
    op, other = (T.Embedding(5, 9, 16, "f32") for _ in range(2))
    table, ids = torch.randn(9, 16, device="cuda", requires_grad=True), torch.tensor([0, 3, 3, -1, 8], device="cuda")
    counts = torch.tensor([1.0, 0, 0, 2, 0, 0, 0, 0, 1], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = other.run(table, ids)
    torch.cuda.synchronize()
    table.grad = torch.zeros_like(table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        table.grad.zero_()
        y = op.run(table, ids)
        y.backward(torch.full_like(y, 2.0))
    for i in range(3):
        with torch.no_grad():
            table.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[[0, 1, 2, 4]], table.detach()[ids[[0, 1, 2, 4]]]) and (y[3] == 0).all()
        assert torch.equal(table.grad, 2 * counts[:, None].expand(9, 16)), i
    with torch.cuda.stream(side):
        table.grad.zero_()
        eager.backward(torch.ones_like(eager))
    torch.cuda.synchronize()
    assert torch.equal(table.grad, counts[:, None].expand(9, 16))


@pytest.mark.gpu
@pytest.mark.parametrize("again", [False, True])
def test_capture_refused_while_another_operator_holds_the_table(gpu_lib, again):
    """Tied weights: the table is a projection's weight too, whose eager graph on the default stream still lives."""
    op = T.Embedding(5, 9, 16, "f32")
    table, ids = torch.randn(9, 16, device="cuda", requires_grad=True), torch.arange(5, device="cuda")
    loss = torch.nn.functional.linear(torch.randn(4, 16, device="cuda"), table).sum()
    if again:
        loss = loss + op.run(table, ids).sum()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = torch.ones(3, device="cuda")                # (a graph of something)
        with pytest.raises(K.KfacError) as e:
            op.run(table, ids)
    assert e.value.status == U and kept is not None
    del loss
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = op.run(table, ids)
        y.backward(torch.ones_like(y))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, table.detach()[:5]) and float(table.grad.sum()) == 5 * 16
