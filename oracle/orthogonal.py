"""Float64 CPU oracle of the orthogonalised update -- TEST INFRASTRUCTURE ONLY,
as the rest of this package.

Written from the singular values' point of view: every step maps them by
a s + b s^3 + c s^5 and leaves the singular vectors alone (Newton-Schulz
iteration for the polar factor).
"""
from __future__ import annotations

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def triples(coefs, steps):
    """float32 coefficients of each step."""
    c = np.asarray(coefs, np.float32).astype(np.float64)
    return np.broadcast_to(c, (steps, 3)) if c.ndim == 1 else c


def orthogonalize(x, coefs=COEFS, steps=5, eps=1e-7):
    x = np.asarray(x, np.float64)
    norm = np.sqrt((x * x).sum()) + eps
    if norm == 0:
        return np.zeros_like(x)
    left, s, right = np.linalg.svd(x / norm, full_matrices=False)
    for a, b, c in triples(coefs, steps):
        s = a * s + b * s**3 + c * s**5
    return (left * s) @ right


def shape_factor(rows, cols, scale):
    return {"none": 1.0, "aspect": max(1.0, rows / cols) ** 0.5, "rms": 0.2 * max(rows, cols) ** 0.5}[scale]


def step(w, mom, grad, lr, mu, wd, coefs=COEFS, steps=5, eps=1e-7, nesterov=True, scale="aspect"):
    """(weight, momentum) after a step."""
    w, mom, grad = (np.asarray(v, np.float64) for v in (w, mom, grad))
    mom = mu * mom + grad
    u = grad + mu * mom if nesterov else mom
    return (1 - lr * wd) * w - lr * shape_factor(*w.shape, scale) * orthogonalize(u, coefs, steps, eps), mom


def bias_step(b, mom, grad, lr, mu, wd):
    b, mom, grad = (np.asarray(v, np.float64) for v in (b, mom, grad))
    mom = mu * mom + grad + wd * b
    return b - lr * mom, mom


def error_bound(x, bits, coefs=COEFS, steps=5, eps=1e-7):
    """2-norm (Frobenius) bound on the error of O(x) where the matrices between products are held in `bits` bits.

    With h = 2^-bits, the half step relative to a value: a step's map has the
    Frobenius-norm Lipschitz constant max |p'(s)|, |p(s) / s| over the
    singular values up to the norm; to that come the roundings of A
    ((|b| + 2 |c| |A|) |X| h |A|_F), of B (h |B|_F |X|) and of the result
    (h |X'|_F).  A float32 sum is off by 2^-24 of each of its running sums; those
    of K terms added 16 at a time, of either sign, come to sqrt(K / 16) of
    sqrt(K) terms: K / 4 terms, a quarter of the terms' sizes together.  Times 8,
    for sums whose terms are mostly of one sign.
    """
    x = np.asarray(x, np.float64)
    if x.shape[0] > x.shape[1]:
        x = x.T
    h, u = 2.0 ** -bits, 2.0 ** -24
    norm = np.sqrt((x * x).sum()) + eps
    if norm == 0:
        return 0.0
    x = x / norm
    e = (h + 2 * u) * np.linalg.norm(x)
    for a, b, c in triples(coefs, steps):
        gram = x @ x.T
        poly = b * gram + c * gram @ gram
        top = np.sqrt(max(np.linalg.eigvalsh(gram)[-1], 0.0))
        s = np.linspace(0, top * 1.05, 2001)
        lip = max(np.abs(a + 3 * b * s**2 + 5 * c * s**4).max(), np.abs(a + b * s**2 + c * s**4).max())
        new = a * x + poly @ x
        sums = 2 * u * (np.linalg.norm(np.abs(x) @ np.abs(x).T) * (abs(b) + 2 * abs(c) * top**2) * top
                        + abs(c) * np.linalg.norm(np.abs(gram) @ np.abs(gram)) * top
                        + np.linalg.norm(np.abs(poly) @ np.abs(x)))
        local = h * ((abs(b) + 2 * abs(c) * top**2) * top * np.linalg.norm(gram) + np.linalg.norm(poly) * top
                     + np.linalg.norm(new)) + sums + 4 * u * np.linalg.norm(new)
        e = lip * e + local
        x = new
    return float(e)


# -- what the documented roundings alone make of it ------------------------------

def _in_bits(v, scale, planes):
    """v held in IEEE halves, one or two of them, at a power of two."""
    v = np.ldexp(v, scale)
    high = v.astype(np.float16).astype(np.float64)
    low = (v - high).astype(np.float16).astype(np.float64) if planes == 2 else 0.0
    return np.ldexp(high + low, -scale)


def _single(v):
    return v.astype(np.float32).astype(np.float64)


def half_products(x, coefs=COEFS, steps=5, eps=1e-7, mistake=None):
    """O(x) with the matrices between the products held as `products` HALF documents: A, B and X as an operand in 11
    bits, B's diagonal and X in the term a X apart, everything else exact.

    The error of sums in float32 is a hundredth of these roundings'.  `mistake` plants one: "x_low" (a X from 11 bits),
    "diagonal" (B's in 11 bits with the rest), "row" (the last product leaves one out), "zeros".
    """
    x = np.asarray(x, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    rho = 1.0
    bits = lambda bound: 15 - int(np.ceil(np.log2(max(bound, 1e-30))))  # noqa: E731
    for a, b, c in triples(coefs, steps):
        s = np.linspace(0, rho, 4001)
        top = 1.02 * np.abs(b * s**2 + c * s**4).max()
        operand, kept = _in_bits(x, bits(rho), 1), _in_bits(x, bits(rho), 2)
        if mistake == "x_low":
            kept = operand
        gram = _in_bits(_single(operand @ operand.T), bits(rho * rho), 1)
        poly = _single(b * gram + c * gram @ gram)
        d = np.diag(poly).copy()
        rest = _in_bits(poly - np.diag(d), bits(top), 1)
        if mistake == "diagonal":
            rest, d = _in_bits(poly, bits(top), 1), 0 * d
        x = _single((a + d[:, None]) * kept + rest @ operand)
        rho = 1.02 * np.abs(a * s + b * s**3 + c * s**5).max()
    if mistake == "row":
        x[len(x) // 2] = 0
    if mistake == "zeros":
        x = 0 * x
    return x.T if tall else x


def single_products(x, coefs=COEFS, steps=5, eps=1e-7):
    """O(x) with every product, sum and matrix in float32."""
    f = np.float32
    x = np.asarray(x, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = (x.T if tall else x) / (np.sqrt((x * x).sum()) + eps)
    x = np.ascontiguousarray(x).astype(f)
    for a, b, c in triples(coefs, steps).astype(f):
        gram = x @ np.ascontiguousarray(x.T)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.T if tall else x).astype(np.float64)


def small_bound(x, coefs=COEFS, steps=5, eps=1e-7):
    """2-norm bound on the error where Q of O(x) = Q X0 is formed in 64 bits (sides of at most 64).

    Q and X0 are rounded to float32 (u each), the d products of an element are summed in float32 (at most d u of their
    sizes, whatever the order), the result is rounded (u).  Q's own errors are 2^-53 of R, which a step's factors raise
    by at most a^2 each: 10^-10 of Q after sixteen.
    """
    x = np.asarray(x, np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    norm = np.sqrt((x * x).sum()) + eps
    x = x / (norm if norm else 1.0)
    r, q = x @ x.T, np.eye(len(x))
    for a, b, c in triples(coefs, steps):
        p = a * np.eye(len(x)) + b * r + c * r @ r
        q, r = p @ q, p @ r @ p
    return (len(x) + 4) * 2.0 ** -24 * np.linalg.norm(np.abs(q) @ np.abs(x)) + 1e-10 * np.linalg.norm(q @ x)


def kinds(rng, rows, cols):
    """(name, matrix) of the kinds whose accuracy is documented."""
    noise = rng.normal(size=(rows, cols))
    d = min(rows, cols)
    left, right = np.linalg.qr(rng.normal(size=(rows, d)))[0], np.linalg.qr(rng.normal(size=(cols, d)))[0].T
    few = lambda k: rng.normal(size=(rows, k)) @ rng.normal(size=(k, cols))  # noqa: E731
    yield "noise", noise
    yield "directions", noise + 2 * few(3)
    yield "strong", noise + 10 * few(8)
    yield "decades", (left * 10 ** -np.linspace(0, 2, d)) @ right
    yield "rows", noise * np.exp(2 * rng.normal(size=(rows, 1)))
    yield "sparse", noise * (rng.random((rows, cols)) < 0.02)
    yield "equal", left @ right
    yield "identity", np.eye(rows, cols)
    yield "dominated", noise + 100 * few(8)
    yield "one", few(1)


# Documented: off by at most so much of the result's 2-norm, with HALF and with FULL.
DOCUMENTED = {"noise": (1.2e-3, 5e-6), "directions": (1.2e-3, 5e-6), "strong": (1.2e-3, 1e-5), "decades": (1.2e-3, 5e-6),
              "rows": (1.2e-3, 5e-6), "sparse": (4e-3, 5e-6), "equal": (1e-2, 5e-6), "identity": (1e-2, 5e-6),
              "dominated": (1.2e-2, 3e-4), "one": (1.2e-2, 3e-4)}
