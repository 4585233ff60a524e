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
