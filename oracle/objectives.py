"""Float64 CPU oracle of the training objectives and of dropout -- TEST
INFRASTRUCTURE ONLY, as the rest of this package.

Written from the definitions, plainly, in float64:
  * logp = log softmax of the scaled logits at the label;
  * the clipped policy loss with the estimator exp(d) - d - 1 of the KL
    divergence from a reference;
  * the logistic (with label smoothing) and squared losses on the difference
    of two sequences' log ratios;
  * the router balance loss E sum_e f_e P_e with f_e the share of the slots
    and P_e the mean probability of expert e, and the squared log-sum-exp;
  * Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel Random
    Numbers: As Easy as 1, 2, 3"), eight 16-bit draws a block.
"""
from __future__ import annotations

import numpy as np


def log_softmax(x, s=1.0):
    x = np.asarray(x, np.float64)
    z = (x - x.max(axis=1, keepdims=True)) * s
    return z - np.log(np.exp(z).sum(axis=1, keepdims=True))


def token_logp(x, labels, s=1.0):
    """Label log-probabilities; 0 for negative labels (their rows are not looked at)."""
    labels = np.asarray(labels)
    out = np.zeros(labels.size)
    at = np.flatnonzero(labels >= 0)
    if at.size:
        out[at] = log_softmax(np.asarray(x)[at], s)[np.arange(at.size), labels[at]]
    return out


def logit_rows(x, labels, coef, s=1.0):
    """d/dx of sum coef logp: coef s (onehot - softmax), 0 where coef is 0."""
    x = np.asarray(x)
    out = np.zeros(x.shape)
    at = np.flatnonzero((np.asarray(labels) >= 0) & (np.asarray(coef) != 0))
    if at.size:
        g = -np.exp(log_softmax(x[at], s))
        g[np.arange(at.size), np.asarray(labels)[at]] += 1.0
        out[at] = g * (np.asarray(coef)[at] * s)[:, None]
    return out


def policy_terms(logp, labels, adv, weight, old, ref, lo, hi, kl):
    """(stats [4], coef [rows]): the loss as a function of the log-probabilities and its derivative."""
    n = logp.size
    coef = np.zeros(n)
    loss_a = loss_k = share = 0.0
    for r in range(n):
        if labels[r] < 0 or weight[r] == 0:
            continue
        ratio = 1.0 if old is None else np.exp(logp[r] - old[r])
        first, second = ratio * adv[r], min(max(ratio, 1.0 - lo), 1.0 + hi) * adv[r]
        slope = 0.0 if second < first else -first
        loss_a -= weight[r] * min(first, second)
        share += weight[r] * (second < first)
        if ref is not None:
            d = ref[r] - logp[r]
            loss_k += weight[r] * (np.expm1(d) - d)
            if kl:
                slope -= kl * np.expm1(d)
        coef[r] = weight[r] * slope
    return np.array([loss_a + (kl * loss_k if kl else 0.0), loss_a, loss_k, share]), coef


def policy_loss(x, labels, adv, weight=None, old=None, ref=None, lo=0.2, hi=0.2, kl=0.0, s=1.0, grad_scale=1.0):
    labels = np.asarray(labels)
    weight = np.full(labels.size, 1.0 / max(1, labels.size)) if weight is None else np.asarray(weight, np.float64)
    logp = token_logp(x, labels, s)
    stats, coef = policy_terms(logp, labels, np.asarray(adv, np.float64), weight, old, ref, lo, hi, kl)
    return stats, logp, logit_rows(x, labels, coef * grad_scale, s)


def preference_terms(logp, labels, offsets, ref, weight, beta, kind, eps, average):
    """(stats [4], seq [2 pairs], coef [rows]) from the log-probabilities."""
    pairs = (len(offsets) - 1) // 2
    seq, share = np.zeros(2 * pairs), np.zeros(2 * pairs)
    for i in range(2 * pairs):
        rows = [r for r in range(offsets[i], offsets[i + 1]) if labels[r] >= 0]
        share[i] = (1.0 / len(rows) if rows else 0.0) if average else 1.0
        seq[i] = sum(logp[r] - (0.0 if ref is None else ref[r]) for r in rows) * share[i]
    stats, coef = np.zeros(4), np.zeros(logp.size)
    for i in range(pairs):
        w = 1.0 / pairs if weight is None else float(weight[i])
        if w == 0:
            continue
        h = seq[i] - seq[pairs + i]
        if kind == "sigmoid":
            x = beta * h
            loss = (1 - eps) * np.logaddexp(0.0, -x) + (eps * np.logaddexp(0.0, x) if eps else 0.0)
            slope = beta * (eps - 1.0 / (1.0 + np.exp(x)) if x >= 0 else 1.0 / (1.0 + np.exp(-x)) - (1.0 - eps))
        else:
            loss, slope = (h - 0.5 / beta) ** 2, 2.0 * (h - 0.5 / beta)
        stats += [w * loss, w * (h > 0), w * beta * h, w]
        for j, sign in ((i, 1.0), (pairs + i, -1.0)):
            for r in range(offsets[j], offsets[j + 1]):
                if labels[r] >= 0:
                    coef[r] = sign * w * slope * share[j]
    return stats, seq, coef


def preference_loss(x, labels, offsets, ref=None, weight=None, beta=0.1, kind="sigmoid", eps=0.0, average=False,
                    s=1.0, grad_scale=1.0):
    logp = token_logp(x, labels, s)
    stats, seq, coef = preference_terms(logp, labels, offsets, ref, weight, beta, kind, eps, average)
    return stats, seq, logp, logit_rows(x, labels, coef * grad_scale, s)


def balance_loss(x, chosen, mask=None, coef=0.01, z_coef=0.0, grad_scale=1.0):
    """(stats [4], counts [E], prob [E], grad [tokens, E])."""
    x, chosen = np.asarray(x, np.float64), np.asarray(chosen)
    tokens, E = x.shape
    k = chosen.shape[1]
    live = np.flatnonzero(np.ones(tokens, bool) if mask is None else np.asarray(mask, bool))
    n = max(1, live.size)
    counts = np.zeros(E, np.int64)
    for e in chosen[live].ravel():
        if 0 <= e < E:
            counts[e] += 1
    grad, prob, z = np.zeros(x.shape), np.zeros(E), 0.0
    f = coef * E * counts / (k * n)
    if live.size:
        m = x[live].max(axis=1, keepdims=True)
        lse = m[:, 0] + np.log(np.exp(x[live] - m).sum(axis=1))
        p = np.exp(x[live] - lse[:, None])
        prob = p.sum(axis=0) / n
        z = z_coef * (lse ** 2).sum() / n
        grad[live] = p * (f - (p * f).sum(axis=1, keepdims=True)) / n + p * (2.0 * z_coef / n * lse)[:, None]
    balance = (f * prob).sum()
    return np.array([balance + z, balance, z, live.size]), counts, prob, grad * grad_scale


def philox(counter, key):
    """Philox 4x32-10: four 32-bit words from four and a key of two (python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_threshold(p):
    return int(round(p * 65536))


def dropout_keep(rows, cols, seed, offset, p):
    """Which elements stay, [rows, cols] bool."""
    per_row = -(-cols // 8)
    out = np.zeros((rows, per_row * 8), bool)
    key = (seed & 0xFFFFFFFF, seed >> 32)
    for b in range(rows * per_row):
        w = philox((b & 0xFFFFFFFF, b >> 32, offset & 0xFFFFFFFF, offset >> 32), key)
        draws = [h for x in w for h in (x & 0xFFFF, x >> 16)]
        out[b // per_row, b % per_row * 8:][:8] = [d >= dropout_threshold(p) for d in draws]
    return out[:, :cols]


def dropout(x, seed, offset, p, residual=None):
    x = np.asarray(x, np.float64)
    t = dropout_threshold(p)
    keep = dropout_keep(x.shape[0], x.shape[1], seed, offset, p)
    y = np.zeros(x.shape)
    y[keep] = x[keep] * (65536.0 / (65536 - t)) if t < 65536 else 0.0
    return y if residual is None else y + np.asarray(residual, np.float64)
