"""What is measured of the training-objective operators, and their plain forms.

The operators stand on either side of an optimizer step: they make the rows that it reads.
Dropout makes a layer's input rows, the losses make the output-gradient rows of the head and of
a router, token log-probabilities are what the losses compare with.

    logp     log-probability of each row's label under the softmax of its logits
    policy   clipped policy loss with a KL term: per-row log-probabilities, loss, logit gradients
    pref     preference loss over pairs of sequences (paired log ratios), likewise
    balance  router balance loss with per-expert counts, logit gradients
    dropout  dropout from a counter-based generator with a residual, forward and backward

Where `own` is false, run() computes them with elementary torch operations; where it is true, it
calls the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# -- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # scoring the tokens one decoding step proposed for 64 sequences: the smallest call
        dict(name="logp_step", op="logp", rows=64, vocab=32768, pad=0, dtype="bf16", scale=1.0),
        # scoring whole prompts, as the reference and the old policy are scored before training
        dict(name="logp_prompts", op="logp", rows=8192, vocab=32768, pad=0, dtype="bf16", scale=1.0),
        # a small policy head (1000 actions) on a minibatch of 256 states, float32
        dict(name="policy_actions", op="policy", rows=256, vocab=1000, pad=0, dtype="f32", kl=0.0, scale=1.0),
        # a minibatch of token rows over a vocabulary of odd size whose head is padded to 64 columns
        dict(name="policy_odd", op="policy", rows=2047, vocab=50001, pad=47, dtype="bf16", kl=0.05, scale=1.25),
        # a minibatch over a large vocabulary: the largest case
        dict(name="policy_wide", op="policy", rows=4096, vocab=131072, pad=0, dtype="bf16", kl=0.02, scale=1.0),
        # two short preference pairs, float32 logits
        dict(name="pref_short", op="pref", pairs=2, longest=48, vocab=16384, pad=0, dtype="f32", beta=0.1,
             kind="sigmoid", smooth=0.0, average=False),
        # a training batch of eight pairs of ragged lengths
        dict(name="pref_batch", op="pref", pairs=8, longest=600, vocab=32768, pad=0, dtype="bf16", beta=0.1,
             kind="sigmoid", smooth=0.1, average=False),
        # the router of a small mixture on one short sequence
        dict(name="balance_short", op="balance", tokens=256, experts=16, top_k=2, dtype="f32", z=0.0),
        # the router of a wide mixture on a training batch
        dict(name="balance_batch", op="balance", tokens=65536, experts=256, top_k=8, dtype="bf16", z=1e-3),
        # one row of 4096 with its residual: where the launch counts
        dict(name="dropout_row", op="dropout", rows=1, cols=4096, dtype="bf16", p=0.1, residual=True),
        # the residual stream of a training batch
        dict(name="dropout_batch", op="dropout", rows=8192, cols=4096, dtype="bf16", p=0.1, residual=True),
        # rows of odd width, no residual, float32
        dict(name="dropout_odd", op="dropout", rows=16384, cols=1025, dtype="f32", p=0.25, residual=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logp", "policy", "policy", "pref", "balance", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    scale = rng.choice([1.0, 1.0, 1.25, 0.7])
    cap = 200_000_000                           # logits of a drawn case: under half of the largest listed one
    if op in ("logp", "policy"):
        vocab = _log_int(rng, 500, 131072)
        rows = _log_int(rng, 1 if op == "logp" else 16, max(16, min(32768, cap // vocab)))
        case = dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, -vocab % 64, 8]), dtype=dtype, scale=scale)
        if op == "policy":
            case["kl"] = rng.choice([0.0, 0.02, 0.1])
        return case
    if op == "pref":
        vocab = _log_int(rng, 1000, 65536)
        pairs = _log_int(rng, 1, 32)
        longest = _log_int(rng, 16, max(16, min(2048, cap // (2 * pairs * vocab))))
        return dict(op=op, pairs=pairs, longest=longest, vocab=vocab, pad=rng.choice([0, -vocab % 64]), dtype=dtype,
                    beta=rng.choice([0.05, 0.1, 0.5]), kind=rng.choice(["sigmoid", "sigmoid", "squared"]),
                    smooth=rng.choice([0.0, 0.1]), average=rng.choice([False, False, True]))
    if op == "balance":
        experts = _log_int(rng, 4, 512)
        tokens = _log_int(rng, 64, 65536)
        return dict(op=op, tokens=tokens, experts=experts, top_k=min(experts, rng.choice([1, 2, 4, 8])), dtype=dtype,
                    z=rng.choice([0.0, 1e-3]))
    cols = _log_int(rng, 64, 16384)
    return dict(op=op, rows=_log_int(rng, 1, max(1, min(65536, 33_000_000 // cols))), cols=cols, dtype=dtype,
                p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.choice([False, True]))


def work(case):
    op, el = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("logp", "policy", "pref"):
        rows = sum(_lengths(case)) if op == "pref" else case["rows"]
        n = rows * case["vocab"]
        grad = op != "logp"
        return {"bytes": n * el * (2 if grad else 1) + rows * 28, "flops": n * (9 if grad else 4)}
    if op == "balance":
        n = case["tokens"] * case["experts"]
        return {"bytes": 2 * n * el + case["tokens"] * (4 * case["top_k"] + 1) + 8 * case["experts"], "flops": 10 * n}
    n = case["rows"] * case["cols"]             # forward x (and residual) -> y, backward dy -> dx
    return {"bytes": n * el * (5 if case["residual"] else 4), "flops": 4 * n}


# -- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape, dtype="f32"):
    """N(0, 1) in `dtype`, drawn in float32 by pieces of at most 2^27 values."""
    out = torch.empty(shape, dtype=_DT[dtype], device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        piece = flat[i:i + (1 << 27)]
        piece.copy_(torch.randn(piece.numel(), generator=gen, device="cuda"))
    return out


def _lengths(case):
    """Tokens of each sequence (the chosen ones, then the rejected ones): ragged, fixed by the case alone."""
    n = 2 * case["pairs"]
    return [max(1, case["longest"] - (i * 37 + 11 * (i % 3)) % max(1, case["longest"] * 3 // 5)) for i in range(n)]


def _token_rows(case, gen, rows):
    """Logits [rows, vocab] (a slice of padded rows where the case has padding) and labels that the model finds likely."""
    vocab, pad = case["vocab"], case["pad"]
    whole = _randn(gen, rows, vocab + pad, dtype=case["dtype"])
    whole.mul_(2.0)
    labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    at = labels.unsqueeze(1)
    likely = 6.0 + 4.0 * torch.rand(rows, 1, generator=gen, device="cuda")
    whole.scatter_(1, at, (whole.gather(1, at).float() + likely).to(whole.dtype))
    return whole[:, :vocab], labels


def _score(logits, labels, scale):
    """Label log-probabilities in 64 bits, some rows at a time: what the old policy and the reference said is near it."""
    out = torch.empty(labels.numel(), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // logits.shape[1])
    for i in range(0, labels.numel(), step):
        z = logits[i:i + step].double() * scale
        out[i:i + step] = z.gather(1, labels[i:i + step, None])[:, 0] - torch.logsumexp(z, 1)
    return out


def prepare(case, seed):
    gen = _generator(seed)
    op, s = case["op"], {"case": case}
    if op == "logp":
        s["logits"], s["labels"] = _token_rows(case, gen, case["rows"])
    elif op == "policy":
        rows = case["rows"]
        s["logits"], s["labels"] = _token_rows(case, gen, rows)
        logp = _score(s["logits"], s["labels"], case["scale"])
        old = (logp + 0.15 * torch.randn(rows, generator=gen, device="cuda").double()).float()
        # the two sides of a clip border are different gradients, and rounding alone may choose between them:
        # no ratio is left within 1e-4 of one
        ratio = torch.exp(logp - old.double())
        for border in (1.0 - _CLIP[0], 1.0 + _CLIP[1]):
            old = torch.where((ratio - border).abs() < 1e-4, old - 1e-3, old)
        s["old"] = old
        s["ref"] = (logp + 0.2 * torch.randn(rows, generator=gen, device="cuda").double()).float()
        s["advantage"] = torch.randn(rows, generator=gen, device="cuda")
        keep = torch.rand(rows, generator=gen, device="cuda") < 0.85          # the other rows are prompt or padding
        s["weight"] = keep.float() / keep.sum().clamp(min=1)
        s["labels"] = torch.where(keep | (s["labels"] % 2 == 0), s["labels"], -100)
    elif op == "pref":
        lengths = _lengths(case)
        rows = sum(lengths)
        s["logits"], labels = _token_rows(case, gen, rows)
        logp = _score(s["logits"], labels, 1.0)
        s["ref"] = (logp + 0.1 * torch.randn(rows, generator=gen, device="cuda").double()).float()
        s["labels"] = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.9, labels, -100)
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
        s["weight"] = torch.full((case["pairs"],), 1.0 / case["pairs"], device="cuda")
    elif op == "balance":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        bias = torch.randn(e, generator=gen, device="cuda")                     # some experts are liked better
        s["logits"] = (_randn(gen, t, e) + 0.5 * bias).to(_DT[case["dtype"]])
        s["experts"] = torch.topk(s["logits"].float(), k, dim=1).indices.int()
        drop = torch.rand(t, k, generator=gen, device="cuda") < 0.02            # slots over an expert's capacity
        s["experts"] = torch.where(drop, -1, s["experts"])
        s["mask"] = torch.rand(t, generator=gen, device="cuda") < 0.9
    else:
        shape = (case["rows"], case["cols"])
        s["x"] = _randn(gen, *shape, dtype=case["dtype"])
        s["dy"] = _randn(gen, *shape, dtype=case["dtype"])
        s["residual"] = _randn(gen, *shape, dtype=case["dtype"]) if case["residual"] else None
        s["seed"] = int(seed) * 0x9E3779B97F4A7C15 % (1 << 64)
        s["offset"] = (1 << 33) + int(seed) % 1000
    s["plan"] = _plan(case) if own else None
    return s


_CLIP = (0.2, 0.28)


# -- the operators of the library ------------------------------------------------------------

def _plan(case):
    from second_order_optimizer_amd import objectives as O
    op, dt = case["op"], case["dtype"]
    if op == "logp":
        return O.TokenLogp(case["rows"], case["vocab"], dtype=dt, logit_scale=case["scale"])
    if op == "policy":
        return O.PolicyLoss(case["rows"], case["vocab"], dtype=dt, clip_low=_CLIP[0], clip_high=_CLIP[1],
                            kl_coef=case["kl"], logit_scale=case["scale"], grad_scale=float(case["rows"]))
    if op == "pref":
        return O.PreferenceLoss(sum(_lengths(case)), case["pairs"], case["vocab"], dtype=dt, beta=case["beta"],
                                kind=case["kind"], label_smoothing=case["smooth"], average=case["average"])
    if op == "balance":
        return O.BalanceLoss(case["tokens"], case["experts"], case["top_k"], dtype=dt, coef=0.01, z_coef=case["z"])
    return O.Dropout(case["rows"], case["cols"], dtype=dt, p=case["p"])


def _run_own(s):
    op, plan = s["case"]["op"], s["plan"]
    if op == "logp":
        return plan.run(s["logits"], s["labels"])
    if op == "policy":
        return plan.run(s["logits"], s["labels"], s["advantage"], weight=s["weight"], old_logp=s["old"],
                        ref_logp=s["ref"])
    if op == "pref":
        return plan.run(s["logits"], s["labels"], s["offsets"], ref_logp=s["ref"], pair_weight=s["weight"])
    if op == "balance":
        return plan.run(s["logits"], s["experts"], mask=s["mask"])
    y = plan.run(s["x"], s["seed"], s["offset"], residual=s["residual"])
    return y, plan.backward(s["dy"], s["seed"], s["offset"])


# -- the plain forms --------------------------------------------------------------------------

def _softmax_rows(logits, labels, scale):
    """Per row, in 32 bits: e^(z - max), its sum and the label's log-probability in 64 bits; labels below 0 score as 0."""
    z = logits.float()
    z = (z - z.amax(1, keepdim=True)).mul_(scale)
    at = labels.clamp(min=0).long().unsqueeze(1)
    z_label = z.gather(1, at)[:, 0].double()
    e = z.exp_()
    total = e.sum(1, dtype=torch.float64)
    return e, total, torch.where(labels >= 0, z_label - torch.log(total), 0.0)


def _logit_grad(e, total, labels, coef, dtype):
    """coef (onehot(label) - softmax), rounded once."""
    scaled = (coef / total).float().unsqueeze(1)
    at = labels.clamp(min=0).long().unsqueeze(1)
    p_label = e.gather(1, at)
    g = e.mul_(-scaled)
    g.scatter_(1, at, coef.float().unsqueeze(1) - p_label * scaled)
    return g.to(dtype)


def _run_logp(s):
    return _softmax_rows(s["logits"], s["labels"], s["case"]["scale"])[2].float()


def _run_policy(s):
    case, a = s["case"], s["advantage"].double()
    e, total, logp = _softmax_rows(s["logits"], s["labels"], case["scale"])
    w = torch.where(s["labels"] >= 0, s["weight"].double(), 0.0)
    ratio = torch.exp(logp - s["old"].double())
    held = ratio.clamp(1.0 - _CLIP[0], 1.0 + _CLIP[1])
    surrogate = torch.minimum(ratio * a, held * a)
    clipped = held * a < ratio * a
    d = s["ref"].double() - logp
    kl = torch.exp(d) - d - 1.0
    slope = torch.where(clipped, 0.0, -a * ratio) + case["kl"] * (1.0 - torch.exp(d))
    coef = w * slope * case["scale"] * float(case["rows"])
    loss_a, loss_k = (w * -surrogate).sum(), (w * kl).sum()
    stats = torch.stack([loss_a + case["kl"] * loss_k, loss_a, loss_k, (w * clipped).sum()]).float()
    return stats, logp.float(), _logit_grad(e, total, s["labels"], coef, s["logits"].dtype)


def _segment_sums(x, offsets):
    run = torch.cat([x.new_zeros(1), torch.cumsum(x, 0)])
    at = offsets.long()
    return run[at[1:]] - run[at[:-1]]


def _run_pref(s):
    case, n = s["case"], s["case"]["pairs"]
    e, total, logp = _softmax_rows(s["logits"], s["labels"], 1.0)
    valid = s["labels"] >= 0
    ratio = torch.where(valid, logp - s["ref"].double(), 0.0)
    seq = _segment_sums(ratio, s["offsets"])
    count = _segment_sums(valid.double(), s["offsets"])
    share = torch.where(count > 0, 1.0 / count.clamp(min=1.0), 0.0) if case["average"] else torch.ones_like(seq)
    seq = seq * share
    h = seq[:n] - seq[n:]
    w, beta, eps = s["weight"].double(), case["beta"], case["smooth"]
    if case["kind"] == "sigmoid":
        x = beta * h
        loss = (1.0 - eps) * torch.log1p(torch.exp(-x.abs())) + (1.0 - eps) * (-x).clamp(min=0.0) \
            + eps * torch.log1p(torch.exp(-x.abs())) + eps * x.clamp(min=0.0)
        slope = beta * (1.0 / (1.0 + torch.exp(-x)) - (1.0 - eps))
    else:
        x = h - 1.0 / (2.0 * beta)
        loss, slope = x * x, 2.0 * x
    stats = torch.stack([(w * loss).sum(), (w * (h > 0)).sum(), (w * beta * h).sum(), w.sum()]).float()
    per_seq = torch.cat([w * slope, -w * slope]) * share
    rows = torch.arange(logp.numel(), device=logp.device)
    which = (rows.unsqueeze(1) >= s["offsets"][1:].unsqueeze(0)).sum(1)
    coef = torch.where(valid, per_seq[which], 0.0)
    return stats, seq.float(), logp.float(), _logit_grad(e, total, s["labels"], coef, s["logits"].dtype)


def _run_balance(s):
    case, x, ids = s["case"], s["logits"].float(), s["experts"]
    experts, k = case["experts"], case["top_k"]
    live = s["mask"].double()
    n = live.sum().clamp(min=1.0)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = (top + torch.log(total))[:, 0].double()
    picked = (ids.unsqueeze(-1) == torch.arange(experts, device=ids.device)) & s["mask"][:, None, None]
    counts = picked.sum((0, 1))
    prob = (p * s["mask"].unsqueeze(1)).sum(0, dtype=torch.float64) / n
    share = counts.double() / (k * n)
    balance, z = 0.01 * experts * (share * prob).sum(), case["z"] * (live * lse * lse).sum() / n
    stats = torch.stack([balance + z, balance, z, live.sum()]).float()
    f = (0.01 * experts / n * share).float()
    g = p * (f - (p * f).sum(1, keepdim=True)) + p * (2.0 * case["z"] / n * lse).float().unsqueeze(1)
    return stats, counts.int(), prob.float(), (g * s["mask"].unsqueeze(1)).to(s["logits"].dtype)


def _times(m, x):
    """(high, low) 32-bit halves of m x for 32-bit m, x held in int64."""
    low, high = m * (x & 0xFFFF), m * (x >> 16)
    return (high + (low >> 16)) >> 16, (low + ((high & 0xFFFF) << 16)) & 0xFFFFFFFF


def _keep(rows, cols, seed, offset, p, device):
    """Which elements stay: Philox 4x32-10, one block of eight 16-bit draws for eight neighbours of a row."""
    per_row = (cols + 7) // 8
    block = torch.arange(rows * per_row, dtype=torch.int64, device=device)
    c0, c1 = block & 0xFFFFFFFF, block >> 32
    c2, c3 = torch.full_like(block, offset & 0xFFFFFFFF), torch.full_like(block, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _times(0xD2511F53, c0)
        h1, l1 = _times(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    draws = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1)
    return draws.view(rows, per_row * 8)[:, :cols] >= int(round(p * 65536))


def _run_dropout(s):
    case, x = s["case"], s["x"]
    keep = _keep(case["rows"], case["cols"], s["seed"], s["offset"], case["p"], x.device)
    scale = 65536.0 / (65536 - int(round(case["p"] * 65536)))
    y = torch.where(keep, x.float() * scale, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype), torch.where(keep, s["dy"].float() * scale, 0.0).to(x.dtype)


_PLAIN = {"logp": _run_logp, "policy": _run_policy, "pref": _run_pref, "balance": _run_balance, "dropout": _run_dropout}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# -- the definitions in 64 bits, with automatic differentiation ------------------------------

def _by_rows(logits, labels, scale, coef_of):
    """Label log-probabilities and d/dlogits of sum(coef * logp), some rows at a time."""
    rows, vocab = logits.shape
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    grad = torch.empty(rows, vocab, dtype=torch.float64, device="cuda") if coef_of is not None else None
    step = max(1, (1 << 25) // vocab)
    for i in range(0, rows, step):
        x = logits[i:i + step].double().requires_grad_(coef_of is not None)
        scored = torch.log_softmax(x * scale, 1).gather(1, labels[i:i + step, None].clamp(min=0).long())[:, 0]
        scored = torch.where(labels[i:i + step] >= 0, scored, 0.0)
        logp[i:i + step] = scored.detach()
        if coef_of is not None:
            grad[i:i + step] = torch.autograd.grad((scored * coef_of[i:i + step]).sum(), x)[0]
    return logp, grad


def _exact_policy(s):
    case, labels, a = s["case"], s["labels"], s["advantage"].double()
    logp = _by_rows(s["logits"], labels, case["scale"], None)[0].requires_grad_()
    w = s["weight"].double() * (labels >= 0)
    ratio = torch.exp(logp - s["old"].double())
    first, second = ratio * a, torch.clamp(ratio, 1 - _CLIP[0], 1 + _CLIP[1]) * a
    gap = s["ref"].double() - logp
    kl = torch.expm1(gap) - gap
    loss_a, loss_k = -(w * torch.minimum(first, second)).sum(), (w * kl).sum()
    loss = loss_a + case["kl"] * loss_k
    coef = torch.autograd.grad(loss, logp)[0] * case["rows"]
    stats = torch.stack([loss, loss_a, loss_k, (w * (second < first)).sum()]).detach()
    return stats, logp.detach(), _by_rows(s["logits"], labels, case["scale"], coef)[1]


def _exact_pref(s):
    case, labels = s["case"], s["labels"]
    logp = _by_rows(s["logits"], labels, 1.0, None)[0].requires_grad_()
    at = s["offsets"].tolist()
    seq = []
    for i in range(2 * case["pairs"]):
        valid = labels[at[i]:at[i + 1]] >= 0
        x = (logp[at[i]:at[i + 1]] - s["ref"][at[i]:at[i + 1]].double())[valid]
        seq.append(x.sum() / (max(1, x.numel()) if case["average"] else 1))
    seq = torch.stack(seq)
    h = seq[:case["pairs"]] - seq[case["pairs"]:]
    w, beta, eps = s["weight"].double(), case["beta"], case["smooth"]
    if case["kind"] == "sigmoid":
        each = -(1 - eps) * torch.nn.functional.logsigmoid(beta * h) - eps * torch.nn.functional.logsigmoid(-beta * h)
    else:
        each = (h - 1 / (2 * beta)) ** 2
    loss = (w * each).sum()
    coef = torch.autograd.grad(loss, logp, retain_graph=True)[0]
    stats = torch.stack([loss, (w * (h > 0)).sum(), (w * beta * h).sum(), w.sum()]).detach()
    return stats, seq.detach(), logp.detach(), _by_rows(s["logits"], labels, 1.0, coef)[1]


def _exact_balance(s):
    case, mask = s["case"], s["mask"]
    x = s["logits"].double().requires_grad_()
    n = max(1, int(mask.sum()))
    prob = torch.softmax(x, 1)[mask].sum(0) / n
    chosen = s["experts"][mask].flatten().long()
    counts = torch.bincount(chosen[chosen >= 0], minlength=case["experts"])
    balance = 0.01 * case["experts"] * (counts.double() / (case["top_k"] * n) * prob).sum()
    z = case["z"] * torch.logsumexp(x, 1)[mask].square().sum() / n
    grad = torch.autograd.grad(balance + z, x)[0]
    stats = torch.stack([balance + z, balance, z, mask.sum().double()]).detach()
    return stats, counts.int(), prob.detach(), grad


def _exact_dropout(s):
    case, u64 = s["case"], np.uint64
    blocks = np.arange(case["rows"] * -(-case["cols"] // 8), dtype=u64)
    low32, shift = u64(0xFFFFFFFF), u64(32)
    c = [blocks & low32, blocks >> shift, np.full_like(blocks, s["offset"] % 2**32), np.full_like(blocks, s["offset"] // 2**32)]
    for r in range(10):
        k = [u64((s["seed"] + r * 0x9E3779B9) % 2**32), u64((s["seed"] // 2**32 + r * 0xBB67AE85) % 2**32)]
        a, b = c[0] * u64(0xD2511F53), c[2] * u64(0xCD9E8D57)
        c = [(b >> shift) ^ c[1] ^ k[0], b & low32, (a >> shift) ^ c[3] ^ k[1], a & low32]
    words = np.stack(c, 1).astype("<u4").view("<u2").reshape(case["rows"], -1)[:, :case["cols"]]
    threshold = round(case["p"] * 65536)
    factor = (words >= threshold) * (65536 / (65536 - threshold))
    y = s["x"].double().cpu().numpy() * factor
    if s["residual"] is not None:
        y = y + s["residual"].double().cpu().numpy()
    return y, s["dy"].double().cpu().numpy() * factor


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logp":
        return _by_rows(s["logits"], s["labels"], case["scale"], None)[0]
    return {"policy": _exact_policy, "pref": _exact_pref, "balance": _exact_balance, "dropout": _exact_dropout}[case["op"]](s)
