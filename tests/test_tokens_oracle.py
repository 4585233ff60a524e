"""Pins of the oracle for sampling, the embedding and the orthogonalised update: small cases by hand, and the
norm bounds that the library's host code derives for the iteration."""
import os
import subprocess

import numpy as np
import pytest

from oracle import orthogonal as O
from oracle import tokens as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sample_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.3])
    assert [T.sample_row(x, u)[0] for u in (0.0, 0.0999, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [T.sample_row(x, u, k=2)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]          # 0.4 and 0.3 of 0.7
    assert T.sample_row(x, 0.99, p=0.65)[2] == 2 and T.sample_row(x, 0.99, p=0.71)[2] == 3
    assert T.sample_row(x, 0.99, m=0.7)[2] == 2 and T.sample_row(x, 0.99, m=1.0)[2] == 1
    assert T.sample_row(x, 0.99, k=3, p=0.45)[2] == 2                                    # 0.45 of the 0.9 that top_k keeps
    assert T.sample_row(x, 0.5, t=0.0)[:2] == pytest.approx((1, np.log(0.4)))
    w = np.exp(x / 0.5)
    assert T.sample_row(x, 0.5, t=0.5)[1] == pytest.approx(np.log(w[T.sample_row(x, 0.5, t=0.5)[0]] / w.sum()))


def test_sample_ties_and_masks():
    assert [T.sample_row(np.zeros(5), u, k=2)[0] for u in (0.1, 0.9)] == [0, 1]          # equal ones: the first two
    assert T.sample_row([-np.inf, -np.inf], 0.5)[:3] == (-1, 0.0, 0)
    assert T.sample_row([-np.inf, 3.0, -np.inf], 0.99)[:3] == (1, 0.0, 1)


def test_sample_distribution():
    x = np.random.default_rng(0).normal(size=20)
    w = np.exp(x - x.max())
    draws = np.array([T.sample_row(x, (i + 0.5) / 4000)[0] for i in range(4000)])
    assert np.abs(np.bincount(draws, minlength=20) - 4000 * w / w.sum()).max() <= 1


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(1)
    table, ids, dy = rng.normal(size=(6, 4)), np.array([2, 0, 2, -1, 9]), rng.normal(size=(5, 4))
    grad, size, counts = T.lookup_grad(dy, ids, 6, 1.5)
    assert counts.tolist() == [1, 0, 2, 0, 0, 0] and (size >= np.abs(grad)).all()
    for v in range(6):
        for c in range(4):
            step = np.zeros_like(table)
            step[v, c] = 1e-3
            diff = ((T.lookup(table + step, ids, 1.5) - T.lookup(table - step, ids, 1.5)) * dy).sum() / 2e-3
            assert diff == pytest.approx(grad[v, c], abs=1e-9)


@pytest.mark.parametrize("shape", [(3, 3), (4, 9), (9, 4)])
def test_orthogonalize_by_products(shape):
    """The singular values' map is the products X <- a X + (b A + c A A) X."""
    x = np.random.default_rng(2).normal(size=shape)
    a, b, c = O.triples(O.COEFS, 1)[0]
    z = x / (np.linalg.norm(x) + 1e-7)
    for _ in range(5):
        g = z @ z.T
        z = a * z + (b * g + c * g @ g) @ z
    assert np.allclose(O.orthogonalize(x), z, atol=1e-12)
    assert (O.orthogonalize(np.zeros((2, 3))) == 0).all()
    cubic = O.orthogonalize(x, (1.5, -0.5, 0.0), steps=60)
    s = np.linalg.svd(cubic, compute_uv=False)
    assert np.allclose(s, 1.0, atol=1e-6)


def test_step_and_bias():
    rng = np.random.default_rng(3)
    w, m, g = (rng.normal(size=(5, 3)) for _ in range(3))
    w2, m2 = O.step(w, m, g, 0.1, 0.9, 0.01)
    assert np.allclose(m2, 0.9 * m + g)
    assert np.allclose(w2, w * (1 - 0.001) - 0.1 * (5 / 3) ** 0.5 * O.orthogonalize(g + 0.9 * m2))
    assert O.shape_factor(3, 5, "aspect") == 1.0 and O.shape_factor(3, 100, "rms") == 2.0


def test_error_bound_holds_for_rounded_products():
    """An iteration whose matrices are rounded to so many bits stays within the bound."""
    def rounded(v, bits):
        m, e = np.frexp(v)
        return np.ldexp(np.round(m * 2.0 ** bits) / 2.0 ** bits, e)
    a, b, c = O.triples(O.COEFS, 1)[0]
    for seed, shape in enumerate([(8, 8), (20, 50), (64, 33)]):
        x = np.random.default_rng(seed).normal(size=shape)
        for bits in (11, 16):
            z = rounded(x / np.linalg.norm(x), bits)
            z = z.T if shape[0] > shape[1] else z
            for _ in range(5):
                g = rounded(z @ z.T, bits)
                z = rounded(a * z + rounded(b * g + c * g @ g, bits) @ z, bits)
            off = np.linalg.norm((z.T if shape[0] > shape[1] else z) - O.orthogonalize(x))
            assert off <= O.error_bound(x, bits), (shape, bits)


def test_norm_bounds_of_the_host(tmp_path):
    """poly_of of csrc/orthogonal.h: the maxima of |b s^2 + c s^4| and |a s + b s^3 + c s^5| over 0 .. rho, plus 2%."""
    src = open(os.path.join(ROOT, "second_order_optimizer_amd", "csrc", "orthogonal.h")).read()
    body = src[src.index("struct PolyBound {"):src.index("// Matrices with a side of at most this")]
    cases = [(3.4445, -4.775, 2.0315, 1.0), (3.4445, -4.775, 2.0315, 1.3), (1.5, -0.5, 0.0, 1.0), (1.0, 0.0, 0.0, 2.0),
             (0.0, 0.0, 0.0, 1.0), (2.0, -1.5, 0.5, 1.1), (-1.0, 3.0, -2.0, 0.7), (3.0, -3.5, 1.4, 1e-3)]
    rows = ",".join("{%r,%r,%r,%r}" % c for c in cases)
    main = tmp_path / "poly.cpp"
    main.write_text("#include <algorithm>\n#include <cmath>\n#include <cstdio>\n" + body + f"""
int main() {{
  double c[][4] = {{{rows}}};
  for (auto& r : c) {{
    float f[3] = {{float(r[0]), float(r[1]), float(r[2])}};
    PolyBound p = poly_of(f, r[3]);
    std::printf("%.17g %.17g\\n", p.b, p.next);
  }}
}}""")
    exe = tmp_path / "poly"
    subprocess.run(["g++", "-std=c++17", "-Wall", str(main), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    for (a, b, c, rho), line in zip(cases, out):
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        s = np.linspace(0, rho, 200001)
        want = 1.02 * np.abs(b * s**2 + c * s**4).max(), 1.02 * np.abs(a * s + b * s**3 + c * s**5).max()
        assert [float(v) for v in line.split()] == pytest.approx(want, rel=1e-6, abs=1e-12)
