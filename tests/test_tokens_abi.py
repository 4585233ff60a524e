"""The C ABI and binding of sampling, the embedding and the orthogonalised update on the host: exports, struct
layout, and every refusal, at the C entry points (well-formed addresses that are never read) and at the Python
classes (CPU tensors, which are never used)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import second_order_optimizer_amd as K
from second_order_optimizer_amd import objectives as Q
from second_order_optimizer_amd import orthogonal as M
from second_order_optimizer_amd import tokens as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = {"kfac_tokens.h": (T, {"kfac_sample_t": T.Sample, "kfac_embedding_t": T.EmbeddingArgs}),
           "kfac_orthogonal.h": (M, {"kfac_orthogonal_t": M.How, "kfac_orthogonal_matrix_t": M.Matrix})}
WS = 0x100000
A, D, U = K.KFAC_ERR_ARG, K.KFAC_ERR_DTYPE, K.KFAC_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from second_order_optimizer_amd import build
        build.build()
    M._library()
    return T._library()


@pytest.mark.parametrize("header", HEADERS)
def test_exports_every_declared_function(lib, header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(kfac_[a-z_]+)\s*\(", src))
    assert names == set(HEADERS[header][0].EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("header", HEADERS)
def test_struct_layout_matches_header(tmp_path, header):
    lines, want = [], []
    for name, mirror in HEADERS[header][1].items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(mirror))
        for f, _ in mirror._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(mirror, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(["#include <stdio.h>", "#include <stddef.h>",
                            f'#include "{os.path.join(ROOT, "include", header)}"', "int main(void){", *lines, "return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(c), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want


def call(fn, s, ws=WS, n=1 << 60):
    return fn(None if s is None else ctypes.byref(s), ws, n, None)


def sample(**over):
    v = dict(logits=0x10000, u=0x20000, token=0x30000, logp=0x40000, kept=0x50000, rows=4, ld=16, temperature=1.0,
             top_p=1.0, min_p=0.0, top_k=0, vocab=16, dtype=K.BF16, reserved=0)
    v.update(over)
    return T.Sample(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=1), A), (dict(dtype=2), D), (dict(rows=-1), A), (dict(vocab=0), A), (dict(ld=15), A),
    (dict(temperature=-1.0), A), (dict(temperature=NAN), A), (dict(temperature=INF), A), (dict(top_p=-0.1), A),
    (dict(top_p=1.5), A), (dict(top_p=NAN), A), (dict(min_p=-0.1), A), (dict(min_p=1.1), A), (dict(top_k=-1), A),
    (dict(vocab=1 << 20, ld=1 << 21), U), (dict(rows=1 << 40, ld=1 << 40), U), (dict(logits=None), A),
    (dict(u=None), A), (dict(token=None), A), (dict(logp=None), A), (dict(kept=None), A),
    (dict(logits=0x10001), K.KFAC_ERR_ALIGN), (dict(token=0x30004), K.KFAC_ERR_ALIGN),
    (dict(row_top_p=0x60002), K.KFAC_ERR_ALIGN), (dict(row_top_k=0x60001), K.KFAC_ERR_ALIGN),
])
def test_sample_refusals(lib, bad, code):
    """Every refusal comes before any HIP call (a call that got through would give KFAC_ERR_HIP here)."""
    assert call(lib.kfac_sample_tokens, sample(**bad)) == code


def embedding(**over):
    v = dict(table=0x10000, y=0x20000, ids=0x30000, counts=0x40000, tokens=4, table_ld=16, y_ld=16, vocab=8, width=16,
             dtype=K.BF16, table_dtype=K.F32, id_type=Q.I64, scale=1.0, accumulate=0, reserved=0)
    v.update(over)
    return T.EmbeddingArgs(**v)


@pytest.mark.parametrize("bad,code", [
    (dict(reserved=1), A), (dict(dtype=2), D), (dict(table_dtype=-1), D), (dict(id_type=2), D), (dict(tokens=-1), A),
    (dict(vocab=0), A), (dict(width=0), A), (dict(table_ld=15), A), (dict(y_ld=15), A), (dict(scale=INF), A),
    (dict(scale=NAN), A), (dict(accumulate=2), A), (dict(vocab=(1 << 29) + 1), U), (dict(tokens=(1 << 30) + 1), U),
    (dict(width=(1 << 24) + 1, table_ld=1 << 25, y_ld=1 << 25), U), (dict(table_ld=1 << 60), U), (dict(y_ld=1 << 60), U),
    (dict(table=None), A), (dict(y=None), A), (dict(ids=None), A), (dict(table=0x10002), K.KFAC_ERR_ALIGN),
    (dict(y=0x20001), K.KFAC_ERR_ALIGN), (dict(ids=0x30004), K.KFAC_ERR_ALIGN),
])
def test_embedding_refusals(lib, bad, code):
    assert call(lib.kfac_embedding_lookup, embedding(**bad)) == code
    assert call(lib.kfac_embedding_grad, embedding(**bad)) == code


def test_embedding_counts_alignment(lib):
    assert call(lib.kfac_embedding_grad, embedding(counts=0x40002)) == K.KFAC_ERR_ALIGN


def test_workspaces(lib):
    for op, args in ((T.TOK_SAMPLE, (4, 16)), (T.TOK_EMBEDDING, (4, 8, 16)), (T.TOK_EMBEDDING, (100000, 8, 16))):
        n = T.workspace_size(op, *args)
        assert n >= 256 and n % 256 == 0
    for args, code in (((2, 1, 1, 1), A), ((0, -1, 1, 1), A), ((0, 1, 0, 1), A), ((0, 1, 1 << 20, 1), U), ((1, 1, 1, 0), A),
                       ((1, 1 << 31, 1, 1), U), ((1, 1, 1 << 30, 1), U), ((1, 1, 1, 1 << 25), U)):
        with pytest.raises(K.KfacError) as e:
            T.workspace_size(*args)
        assert e.value.status == code, args
    for fn, s, need in ((lib.kfac_sample_tokens, sample(), T.workspace_size(T.TOK_SAMPLE, 4, 16)),
                        (lib.kfac_embedding_grad, embedding(), T.workspace_size(T.TOK_EMBEDDING, 4, 8, 16)),
                        (lib.kfac_embedding_lookup, embedding(), 256)):
        assert call(fn, s, ws=None) == K.KFAC_ERR_WORKSPACE
        assert call(fn, s, n=need - 1) == K.KFAC_ERR_WORKSPACE
        assert call(fn, s, ws=WS + 16) == K.KFAC_ERR_ALIGN
        assert call(fn, None) == A


COEFS = (ctypes.c_float * 48)(*([1.5, -0.5, 0.0] * 16))


def how(coefs=COEFS, **over):
    v = dict(coefs=ctypes.addressof(coefs) if coefs is not None else None, eps=1e-7, steps=5, products=0, nesterov=1, scale=1)
    v.update(over)
    return M.How(**v)


def matrix(**over):
    v = dict(x=0x10000, y=0x20000, ld=70, stride=70 * 100, y_ld=70, y_stride=70 * 100, rows=100, cols=70, batch=2, dtype=K.F32)
    v.update(over)
    return M.Matrix(**v)


def orthogonalize(lib, m, h, ws=WS, n=1 << 60):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return lib.kfac_orthogonalize(ref(m), ref(h), ws, n, None)


HOW_BAD = [
    (dict(coefs=None), A), (dict(steps=0), A), (dict(steps=17), A), (dict(eps=-1.0), A), (dict(eps=NAN), A), (dict(eps=INF), A),
    (dict(products=2), A), (dict(nesterov=2), A), (dict(scale=3), A), (dict(coefs=(ctypes.c_float * 15)(65.0)), A),
    (dict(coefs=(ctypes.c_float * 15)(NAN)), A), (dict(coefs=(ctypes.c_float * 15)(*([10.0, 0.0, 0.0] * 5))), U),
]


@pytest.mark.parametrize("bad,code", HOW_BAD)
def test_iteration_refusals(lib, bad, code):
    assert orthogonalize(lib, matrix(), how(**bad)) == code
    assert step(lib, [layer()], how=how(**bad)) == code
    n = ctypes.c_size_t(0)
    assert lib.kfac_orthogonal_workspace_size(ctypes.byref(matrix()), ctypes.byref(how(**bad)), ctypes.byref(n)) == code


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), D), (dict(rows=0), A), (dict(cols=0), A), (dict(batch=-1), A), (dict(ld=69), A), (dict(y_ld=69), A),
    (dict(stride=70 * 100 - 1), A), (dict(y_stride=5), A), (dict(rows=65537), U), (dict(cols=65537, ld=65537, y_ld=65537), U),
    (dict(batch=65536), U), (dict(rows=65536, cols=65536, ld=65536, y_ld=65536, batch=60000), U), (dict(stride=1 << 61), U),
    (dict(ld=1 << 60), U), (dict(x=None), A), (dict(y=None), A), (dict(x=0x10002), K.KFAC_ERR_ALIGN),
    (dict(y=0x20001), K.KFAC_ERR_ALIGN), (dict(y=0x10000, y_ld=71, y_stride=71 * 100), A), (dict(y=0x10000, y_stride=70 * 101), A),
])
def test_orthogonalize_refusals(lib, bad, code):
    assert orthogonalize(lib, matrix(**bad), how()) == code


def test_orthogonalize_workspace_refusals(lib):
    n = ctypes.c_size_t(0)
    for m in (matrix(), matrix(rows=3), matrix(rows=300, cols=200, ld=200, y_ld=200, stride=60000, y_stride=60000)):
        assert lib.kfac_orthogonal_workspace_size(ctypes.byref(m), ctypes.byref(how()), ctypes.byref(n)) == K.KFAC_OK
        assert orthogonalize(lib, m, how(), n=n.value - 1) == K.KFAC_ERR_WORKSPACE
        assert orthogonalize(lib, m, how(), ws=None) == K.KFAC_ERR_WORKSPACE
        assert orthogonalize(lib, m, how(), ws=WS + 8) == K.KFAC_ERR_ALIGN
    assert orthogonalize(lib, None, how()) == A and orthogonalize(lib, matrix(), None) == A
    assert lib.kfac_orthogonal_workspace_size(ctypes.byref(matrix()), ctypes.byref(how()), None) == A
    assert orthogonalize(lib, matrix(batch=0, x=None, y=None), how()) == K.KFAC_OK      # nothing to do


def layer(**over):
    L = K.Layer()
    v = dict(kind=K.LINEAR, has_bias=1, d_in=70, d_out=100, grad_w=0x10000, w=0x20000, mom_w=0x30000, grad_b=0x40000, b=0x50000,
             mom_b=0x60000)
    v.update(over)
    for k, x in v.items():
        setattr(L, k, x)
    return L


def step(lib, layers, hp=None, how=how(), ws=WS, n=1 << 60):
    hp = K.HParams(lr=0.1) if hp is None else hp
    arr = K.layer_array(layers) if layers else None
    return lib.kfac_step_orthogonal(arr, len(layers), ctypes.byref(hp), ctypes.byref(how), ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(kind=K.BATCHNORM), U), (dict(kind=7), A), (dict(has_bias=2), A), (dict(d_in=0), A), (dict(d_out=0), A),
    (dict(reserved=1), A), (dict(d_in=65537), U), (dict(grad_w=None), A), (dict(w=None), A), (dict(mom_w=None), A),
    (dict(grad_b=None), A), (dict(b=None), A), (dict(mom_b=None), A), (dict(w=0x20002), K.KFAC_ERR_ALIGN),
    (dict(b=0x50001), K.KFAC_ERR_ALIGN),
])
def test_step_refusals(lib, bad, code):
    assert step(lib, [layer(), layer(**bad)]) == code


def test_step_scalars_and_workspace(lib):
    for hp, code in ((K.HParams(lr=NAN), A), (K.HParams(momentum=INF), A), (K.HParams(weight_decay=NAN), A),
                     (K.HParams(reserved=1), A), (K.HParams(options=1), U), (K.HParams(phase_mask=1), U)):
        assert step(lib, [layer()], hp) == code
    assert step(lib, []) == A
    n = ctypes.c_size_t(0)
    arr = K.layer_array([layer(), layer(d_in=5)])
    assert lib.kfac_orthogonal_step_workspace_size(arr, 2, ctypes.byref(how()), ctypes.byref(n)) == K.KFAC_OK
    assert step(lib, [layer(), layer(d_in=5)], n=n.value - 1) == K.KFAC_ERR_WORKSPACE
    assert step(lib, [layer()], ws=WS + 16) == K.KFAC_ERR_ALIGN


# -- the Python classes -------------------------------------------------------------------------

def refused(status, fn, *a, **kw):
    with pytest.raises(K.KfacError) as e:
        fn(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_constructor_refusals(lib):
    cpu = dict(device="cpu")
    refused(D, T.Sampler, 4, 8, dtype="f64", **cpu)
    refused(A, T.Sampler, -1, 8, **cpu)
    refused(A, T.Sampler, 4, 0, **cpu)
    refused(U, T.Sampler, 4, (1 << 32) + 8, **cpu)
    for kw in (dict(temperature=-1.0), dict(temperature=NAN), dict(top_k=-1), dict(top_k=1 << 31), dict(top_p=1.5), dict(min_p=-0.5)):
        refused(A, T.Sampler, 4, 8, **kw, **cpu)
    refused(D, T.Embedding, 4, 8, 16, dtype="f16", **cpu)
    refused(D, T.Embedding, 4, 8, 16, table_dtype="f16", **cpu)
    refused(A, T.Embedding, -1, 8, 16, **cpu)
    refused(A, T.Embedding, 4, 0, 16, **cpu)
    refused(A, T.Embedding, 4, 8, 0, **cpu)
    refused(A, T.Embedding, 4, 8, 16, scale=INF, **cpu)
    refused(U, T.Embedding, 4, (1 << 32) + 8, 16, **cpu)
    refused(U, T.Embedding, 1 << 31, 8, 16, **cpu)
    refused(D, M.Orthogonal, 4, 8, dtype="f64", **cpu)
    refused(A, M.Orthogonal, 0, 8, **cpu)
    refused(A, M.Orthogonal, 4, 8, batch=-1, **cpu)
    refused(U, M.Orthogonal, 70000, 8, **cpu)
    for kw in (dict(steps=0), dict(steps=17), dict(coefs=(1.0, 2.0)), dict(coefs=((1.0, 0.0, 0.0),)), dict(coefs=(100.0, 0.0, 0.0)),
               dict(eps=-1.0), dict(eps=NAN), dict(products="quarter")):
        refused(A, M.Orthogonal, 4, 8, **kw, **cpu)
    w, m, b = torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4)
    refused(A, M.OrthogonalStep, [], [])
    refused(A, M.OrthogonalStep, [w], [m, m])
    refused(A, M.OrthogonalStep, [w], [w])                                    # one memory for two
    refused(A, M.OrthogonalStep, [w, w[1:]], [m, torch.zeros(3, 8)])
    refused(A, M.OrthogonalStep, [w], [torch.zeros(8, 4)])
    refused(A, M.OrthogonalStep, [w.t()], [torch.zeros(8, 4)])
    refused(D, M.OrthogonalStep, [w.bfloat16()], [m])
    refused(A, M.OrthogonalStep, [w], [m], [b], [None])
    refused(A, M.OrthogonalStep, [w], [m], [torch.zeros(5)], [torch.zeros(5)])
    refused(A, M.OrthogonalStep, [w], [m], scale="none of these")
    refused(A, M.OrthogonalStep, ["w"], [m])


def test_run_refusals(lib):
    x, u = torch.zeros(4, 8), torch.zeros(4)
    op = T.Sampler(4, 8, dtype="f32", device="cpu")
    refused(U, op.run, x, u)                                     # valid, but not on a GPU
    refused(D, op.run, x.bfloat16(), u)
    refused(A, op.run, torch.zeros(4, 9), u)
    refused(A, op.run, torch.zeros(8, 4).t(), u)
    refused(A, op.run, x, torch.zeros(5))
    refused(D, op.run, x, u.double())
    refused(D, op.run, x, u, top_k=torch.zeros(4, dtype=torch.int64))
    refused(A, op.run, x, u, temperature=torch.zeros(8)[::2])
    refused(A, op.run, None, u)
    e = T.Embedding(4, 8, 16, dtype="f32", table_dtype="bf16", device="cpu")
    table, ids, dy = torch.zeros(8, 16).bfloat16(), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 16)
    refused(U, e.run, table, ids)
    refused(D, e.run, table.float(), ids)
    refused(A, e.run, table[:7], ids)
    refused(D, e.run, table, ids.short())
    refused(A, e.run, table, ids[:3])
    refused(D, e.run, table, ids, out=torch.zeros(4, 16).bfloat16())
    refused(A, e.run, table.requires_grad_(), ids, out=dy)
    refused(U, e.backward, dy, ids)
    refused(D, e.backward, dy.bfloat16(), ids)
    refused(D, e.backward, dy, ids, grad=torch.zeros(8, 16))
    refused(A, e.backward, dy, ids, accumulate=True)
    same = T.Embedding(8, 8, 16, dtype="f32", device="cpu")
    square, eight = torch.zeros(8, 16), torch.zeros(8, dtype=torch.int64)
    refused(A, same.run, square, eight, out=square)
    refused(A, same.backward, square, eight, grad=square)
    o = M.Orthogonal(4, 8, batch=2, dtype="f32", device="cpu")
    y = torch.zeros(2, 4, 8)
    refused(U, o.run, y)
    refused(D, o.run, y.bfloat16())
    refused(A, o.run, y[0])
    refused(A, o.run, y.transpose(1, 2))
    refused(A, o.run, y, out=torch.zeros(4, 8).expand(2, 4, 8))
    w, m, b, bm = torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4), torch.zeros(4)
    s = M.OrthogonalStep([w], [m], [b], [bm])
    refused(U, s.run, [x], [u])
    refused(A, s.run, x, [u])
    refused(A, s.run, [x, x], [u])
    refused(A, s.run, [x])
    refused(A, s.run, [x], [None])
    refused(A, s.run, [torch.zeros(8, 4).t()], [u])
    refused(D, s.run, [x.double()], [u])
    refused(A, M.OrthogonalStep([w], [m]).run, [x], [u])
    for gw, gb in ((w, u), (m, u), (x, b), (x, bm)):
        refused(A, s.run, [gw], [gb])
    with pytest.raises(TypeError):
        s.run([x], [u], lr="fast")
