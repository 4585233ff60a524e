"""What is measured of the sampling, embedding and orthogonalisation operators, and their plain forms.

A round of training a policy over tokens: the tokens' embedding rows go through layers to logits, a token is
sampled from each row of them, the objectives make gradients, and the layers' weights and the embedding take
a step.

    sample  a token of each row of logits with temperature, top-k, top-p and min-p, from given random numbers
    embed   embedding lookup with scaling; its gradient, dense, with per-token counts
    orth    the nearest-to-orthogonal update of a matrix by Newton-Schulz products
    step    momentum, orthogonalised update and weight decay of a stack of layers, with their biases

Where `own` is false, run() computes them with elementary torch operations; where it is true, it calls the
library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_COEFS = (3.4445, -4.7750, 2.0315)      # of x -> a x + b x^3 + c x^5
_STEPS, _EPS = 5, 1e-7
_HP = dict(lr=0.02, momentum=0.9, weight_decay=5e-4)


# -- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one sequence's next token over a large vocabulary: the smallest call, where latency counts
        dict(name="sample_one", op="sample", rows=1, vocab=131072, pad=0, dtype="bf16", temperature=0.8, top_k=50,
             top_p=0.95, min_p=0.0, masked=0.0, per_row=False),
        # one decoding step of 64 sequences, each with settings of its own
        dict(name="sample_step", op="sample", rows=64, vocab=32768, pad=0, dtype="bf16", temperature=0.7, top_k=40,
             top_p=0.9, min_p=0.02, masked=0.0, per_row=True),
        # actions of a small policy head, float32, one in ten not allowed in a state
        dict(name="sample_actions", op="sample", rows=4096, vocab=1000, pad=0, dtype="f32", temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0, masked=0.1, per_row=False),
        # many rollouts at once over a large vocabulary of odd size, its head padded: nucleus only
        dict(name="sample_rollouts", op="sample", rows=1023, vocab=100257, pad=31, dtype="bf16", temperature=1.0,
             top_k=0, top_p=0.9, min_p=0.0, masked=0.0, per_row=False),
        # the input rows of one decoding step of 64 sequences
        dict(name="embed_step", op="embed", tokens=64, vocab=32768, width=4096, dtype="bf16", table="bf16", scale=64.0,
             grad=False),
        # a batch of odd sizes, float32 table and rows, both ways
        dict(name="embed_odd", op="embed", tokens=5003, vocab=50001, width=1025, dtype="f32", table="f32", scale=1.0,
             grad=True),
        # a training batch, bf16 rows of a float32 table, both ways
        dict(name="embed_batch", op="embed", tokens=32768, vocab=65536, width=4096, dtype="bf16", table="f32",
             scale=64.0, grad=True),
        # the projections of sixteen heads, a batch of small matrices
        dict(name="orth_heads", op="orth", batch=16, rows=64, cols=1024, dtype="bf16"),
        # one matrix of odd size, float32, taller than wide
        dict(name="orth_odd", op="orth", batch=1, rows=2047, cols=1000, dtype="f32"),
        # one matrix of a 4096 <-> 16384 pair: the largest case
        dict(name="orth_pair", op="orth", batch=1, rows=16384, cols=4096, dtype="bf16"),
        # a step of one small layer with its bias
        dict(name="step_fc", op="step", layers=1, d_in=64, d_out=32),
        # a step of four MLP blocks, each a 1024 -> 4096 and a 4096 -> 1024 layer with their biases
        dict(name="step_mlp", op="step", layers=8, d_in=1024, d_out=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "embed", "orth", "orth", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "sample":
        vocab = _log_int(rng, 500, 131072)
        rows = _log_int(rng, 1, max(1, min(16384, 100_000_000 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, -vocab % 64, 5]), dtype=dtype,
                    temperature=rng.choice([0.6, 0.8, 1.0, 1.3]), top_k=rng.choice([0, 0, 1, 20, 50, 400]),
                    top_p=rng.choice([1.0, 0.95, 0.9, 0.5]), min_p=rng.choice([0.0, 0.0, 0.05]),
                    masked=rng.choice([0.0, 0.0, 0.3]), per_row=rng.choice([False, True]))
    if op == "embed":
        width = _log_int(rng, 64, 8192)
        vocab = _log_int(rng, 500, max(500, min(131072, 250_000_000 // width)))
        tokens = _log_int(rng, 1, max(1, min(65536, 130_000_000 // width)))
        return dict(op=op, tokens=tokens, vocab=vocab, width=width, dtype=dtype,
                    table=rng.choice(["f32", dtype]), scale=rng.choice([1.0, 8.0, 0.5]), grad=rng.choice([True, True, False]))
    if op == "orth":
        small = _log_int(rng, 16, 2048)
        large = _log_int(rng, small, 8192)
        shape = rng.choice([(small, large), (large, small)])
        return dict(op=op, batch=rng.choice([1, 1, 2, 3]), rows=shape[0], cols=shape[1], dtype=dtype)
    small = _log_int(rng, 16, 1024)
    large = _log_int(rng, small, 4096)
    shape = rng.choice([(small, large), (large, small)])
    return dict(op=op, layers=rng.choice([1, 2, 3, 6]), d_in=shape[0], d_out=shape[1])


def _products(rows, cols):
    """Operations of the Newton-Schulz products of one matrix; of the symmetric ones (X X^T and its square) half."""
    d, n = min(rows, cols), max(rows, cols)
    return _STEPS * (3.0 * d * d * n + 1.0 * d * d * d)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * 20, "flops": 10 * n}
    if op == "embed":
        el, te = (2 if case[k] == "bf16" else 4 for k in ("dtype", "table"))
        t, w = case["tokens"], case["width"]
        size = t * w * (te + el) + 8 * t                    # (a token met twice may be read once)
        if case["grad"]:
            size += t * w * el + case["vocab"] * (w * te + 4)
        return {"bytes": size, "flops": 2 * t * w}
    if op == "orth":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4),
                "flops": case["batch"] * _products(case["rows"], case["cols"])}
    n = case["layers"] * case["d_out"] * (case["d_in"] + 1)
    return {"bytes": 20 * n, "flops": case["layers"] * _products(case["d_in"], case["d_out"])}


# -- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _logits(case, gen):
    """A slice of padded rows: a bulk of unlikely tokens, a few likely ones, some that are not allowed; a row without any."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn(rows, vocab, generator=gen, device="cuda").mul_(2.0)
    likely = torch.randint(0, vocab, (rows, 12), generator=gen, device="cuda")
    x.scatter_add_(1, likely, 5.0 + 4.0 * torch.rand(rows, 12, generator=gen, device="cuda"))
    if case["masked"]:
        x[torch.rand(rows, vocab, generator=gen, device="cuda") < case["masked"]] = -math.inf
        if rows > 8:
            x[7] = -math.inf
    whole = torch.empty(rows, vocab + case["pad"], dtype=_DT[case["dtype"]], device="cuda")
    whole[:, :vocab] = x
    return whole[:, :vocab]


def _matrix(gen, *shape):
    """What an optimizer orthogonalises: a few strong directions over a bulk of noise."""
    rows, cols = shape[-2:]
    k = max(1, min(8, rows // 2, cols // 2))
    left = torch.randn(*shape[:-2], rows, k, generator=gen, device="cuda")
    right = torch.randn(*shape[:-2], k, cols, generator=gen, device="cuda")
    return 1e-3 * (torch.randn(*shape, generator=gen, device="cuda") + torch.matmul(left, right))


def prepare(case, seed):
    gen = _generator(seed)
    op, s = case["op"], {"case": case}
    if op == "sample":
        rows = case["rows"]
        s["logits"] = _logits(case, gen)
        s["u"] = torch.rand(rows, generator=gen, device="cuda")
        if case["per_row"]:
            pick = lambda *v: torch.tensor(v, device="cuda")[torch.randint(0, len(v), (rows,), generator=gen, device="cuda")]  # noqa: E731
            t, p = case["temperature"], case["top_p"]
            s["temperature"] = pick(t, 1.0, 1.5 * t)
            s["top_k"] = pick(case["top_k"], 0, case["top_k"] + 3).int()
            s["top_p"] = pick(p, 1.0, 0.7 * p)
            s["min_p"] = pick(case["min_p"], 0.0, 0.1)
    elif op == "embed":
        t, vocab, width = case["tokens"], case["vocab"], case["width"]
        s["table"] = torch.randn(vocab, width, generator=gen, device="cuda").mul_(0.02).to(_DT[case["table"]])
        # a token's frequency falls with its number, as in text; one in fifty is padding
        u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(max=vocab - 1)
        s["ids"] = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.02, -1, ids)
        if case["grad"]:
            s["dy"] = torch.randn(t, width, generator=gen, device="cuda").mul_(1e-3).to(_DT[case["dtype"]])
    elif op == "orth":
        s["x"] = _matrix(gen, case["batch"], case["rows"], case["cols"]).to(_DT[case["dtype"]])
    else:
        n, d_in, d_out = case["layers"], case["d_in"], case["d_out"]
        shapes = [(d_out, d_in) if i % 2 == 0 else (d_in, d_out) for i in range(n)]
        f = lambda v: v.contiguous()  # noqa: E731
        s["w"] = [f(torch.randn(o, i, generator=gen, device="cuda").mul_(i ** -0.5)) for o, i in shapes]
        s["mom"] = [f(4.0 * _matrix(gen, o, i)) for o, i in shapes]
        s["grad"] = [f(_matrix(gen, o, i)) for o, i in shapes]
        s["b"], s["mom_b"], s["grad_b"] = ([c * torch.randn(o, generator=gen, device="cuda") for o, _ in shapes]
                                           for c in (0.1, 4e-3, 1e-3))
    s["plan"] = _plan(s) if own else None
    return s


# -- the operators of the library ------------------------------------------------------------

def _plan(s):
    case = s["case"]
    op = case["op"]
    if op == "sample":
        from second_order_optimizer_amd import tokens
        return tokens.Sampler(case["rows"], case["vocab"], dtype=case["dtype"], temperature=case["temperature"],
                              top_k=case["top_k"], top_p=case["top_p"], min_p=case["min_p"])
    if op == "embed":
        from second_order_optimizer_amd import tokens
        return tokens.Embedding(case["tokens"], case["vocab"], case["width"], dtype=case["dtype"],
                                table_dtype=case["table"], scale=case["scale"])
    from second_order_optimizer_amd import orthogonal
    if op == "orth":
        return orthogonal.Orthogonal(case["rows"], case["cols"], batch=case["batch"], dtype=case["dtype"], steps=_STEPS,
                                     coefs=_COEFS, eps=_EPS)
    return orthogonal.OrthogonalStep(s["w"], s["mom"], biases=s["b"], bias_momenta=s["mom_b"], steps=_STEPS,
                                     coefs=_COEFS, eps=_EPS, nesterov=True, scale="aspect")


def _run_own(s):
    op, plan = s["case"]["op"], s["plan"]
    if op == "sample":
        if s["case"]["per_row"]:
            return plan.run(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"])
        return plan.run(s["logits"], s["u"])
    if op == "embed":
        y = plan.run(s["table"], s["ids"])
        return (y, *plan.backward(s["dy"], s["ids"])) if s["case"]["grad"] else y
    if op == "orth":
        return plan.run(s["x"])
    plan.run(s["grad"], s["grad_b"], **_HP)
    return s["w"], s["mom"], s["b"], s["mom_b"]


# -- the plain forms --------------------------------------------------------------------------

def _setting(s, name):
    """[rows, 1] in 64 bits."""
    v = s[name].double() if s["case"]["per_row"] else torch.full((s["case"]["rows"],), float(s["case"][name]),
                                                                 dtype=torch.float64, device="cuda")
    return v.unsqueeze(1)


def _run_sample(s):
    z, place = s["logits"].double().sort(dim=1, descending=True, stable=True)       # equal ones: lowest index first
    top = z[:, :1]
    live = top[:, 0] > -math.inf
    z = (z - torch.where(top > -math.inf, top, 0.0)) / _setting(s, "temperature")
    w = torch.exp(z)
    rank = torch.arange(w.shape[1], device=w.device)
    k, p = _setting(s, "top_k"), _setting(s, "top_p")
    keep = (z > -math.inf) & ((k == 0) | (rank < k))
    some = w * keep
    run = torch.cumsum(some, 1)
    keep &= (p >= 1.0) | (run - some < p * run[:, -1:]) | (rank == 0)
    keep &= w >= _setting(s, "min_p")
    kept = torch.zeros_like(w).scatter_(1, place, w * keep)                        # back to the tokens' own order
    run = torch.cumsum(kept, 1)
    token = (run <= s["u"].double().unsqueeze(1) * run[:, -1:]).sum(1)
    at = torch.where(live, token, 0)
    chosen = (place == at.unsqueeze(1)).double()
    logp = torch.where(chosen > 0, z, 0.0).sum(1) - torch.log(w.sum(1).clamp(min=1e-300))
    return torch.where(live, token, -1), torch.where(live, logp, 0.0).float(), (keep.sum(1) * live).int()


def _run_embed(s):
    case, ids = s["case"], s["ids"]
    there = (ids >= 0).unsqueeze(1)
    rows = s["table"][ids.clamp(min=0)].float()
    y = torch.where(there, rows * case["scale"], 0.0).to(_DT[case["dtype"]])
    if not case["grad"]:
        return y
    at = torch.where(ids >= 0, ids, case["vocab"])
    grad = torch.zeros(case["vocab"] + 1, case["width"], device="cuda")
    grad.index_add_(0, at, s["dy"].float() * case["scale"])
    counts = torch.zeros(case["vocab"] + 1, dtype=torch.int32, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    return y, grad[:-1].to(_DT[case["table"]]), counts[:-1]


def _newton_schulz(x):
    """[batch, rows, cols] in 32 bits."""
    a, b, c = _COEFS
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x / (norm + _EPS)).float()
    for _ in range(_STEPS):
        g = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _run_orth(s):
    return _newton_schulz(s["x"].float()).to(s["x"].dtype)


def _run_step(s):
    lr, mu, wd = _HP["lr"], _HP["momentum"], _HP["weight_decay"]
    wide = s["w"][0].shape
    turn = lambda v, w: v if w.shape == wide else v.t()  # noqa: E731
    torch._foreach_mul_(s["mom"], mu)
    torch._foreach_add_(s["mom"], s["grad"])
    u = torch.stack([turn(g + mu * m, g) for g, m in zip(s["grad"], s["mom"])])
    o = _newton_schulz(u)
    scales = [max(1.0, w.shape[0] / w.shape[1]) ** 0.5 for w in s["w"]]
    torch._foreach_mul_(s["w"], 1.0 - lr * wd)
    torch._foreach_sub_(s["w"], [(lr * k) * turn(v, w) for k, v, w in zip(scales, o, s["w"])])
    torch._foreach_mul_(s["mom_b"], mu)
    torch._foreach_add_(s["mom_b"], [g + wd * b for g, b in zip(s["grad_b"], s["b"])])
    torch._foreach_add_(s["b"], s["mom_b"], alpha=-lr)
    return s["w"], s["mom"], s["b"], s["mom_b"]


_PLAIN = {"sample": _run_sample, "embed": _run_embed, "orth": _run_orth, "step": _run_step}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# -- the definitions in 64 bits -----------------------------------------------------------------

def _exact_sample(s):
    case = s["case"]
    token, logp, kept = [], [], []
    u = s["u"].double().tolist()
    for r in range(case["rows"]):
        x = s["logits"][r].double().cpu().numpy()
        get = lambda name: float(s[name][r]) if case["per_row"] else float(case[name])  # noqa: E731
        allowed = np.flatnonzero(x > -np.inf)
        if not allowed.size:
            token.append(-1), logp.append(0.0), kept.append(0)
            continue
        weight = np.exp((x - x[allowed].max()) / get("temperature"))
        order = allowed[np.lexsort((allowed, -x[allowed]))]
        if get("top_k"):
            order = order[:int(get("top_k"))]
        if get("top_p") < 1:
            order = order[:1 + int(np.searchsorted(np.cumsum(weight[order]), get("top_p") * weight[order].sum()))]
        order = np.sort(order[weight[order] >= get("min_p")])
        run_ = np.cumsum(weight[order])
        t = order[min(len(order) - 1, int(np.searchsorted(run_, u[r] * run_[-1], side="right")))]
        token.append(int(t)), kept.append(len(order))
        logp.append(float((x[t] - x[allowed].max()) / get("temperature") - np.log(weight.sum())))
    return torch.tensor(token), torch.tensor(logp, dtype=torch.float64), torch.tensor(kept, dtype=torch.int32)


def _exact_embed(s):
    case = s["case"]
    ids = s["ids"]
    y = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
    live = torch.nonzero(ids >= 0)[:, 0]
    y[live] = torch.index_select(s["table"], 0, ids[live]).double() * case["scale"]
    if not case["grad"]:
        return y
    grad = torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device="cuda")
    grad.index_put_((ids[live],), s["dy"][live].double(), accumulate=True)
    return y, grad.mul_(case["scale"]), torch.bincount(ids[live], minlength=case["vocab"]).int()


def _exact_orth(x):
    """One matrix, by products from the side that keeps them small."""
    a, b, c = _COEFS
    x = x.double()
    x = x / (torch.linalg.matrix_norm(x) + _EPS)
    right = x.shape[0] > x.shape[1]
    eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(_STEPS):
        q = x.mT @ x if right else x @ x.mT
        q = a * eye + (b * eye + c * q) @ q
        x = x @ q if right else q @ x
    return x


def _exact_step(s):
    lr, mu, wd = _HP["lr"], _HP["momentum"], _HP["weight_decay"]
    out = ([], [], [], [])
    for w, m, g, b, n, h in zip(s["w"], s["mom"], s["grad"], s["b"], s["mom_b"], s["grad_b"]):
        w, m, g, b, n, h = (v.double() for v in (w, m, g, b, n, h))
        m = mu * m + g
        o = _exact_orth(g + mu * m)
        n = mu * n + h + wd * b
        scale = max(1.0, w.shape[0] / w.shape[1]) ** 0.5
        for to, v in zip(out, (w - lr * wd * w - lr * scale * o, m, b - lr * n, n)):
            to.append(v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orth":
        return torch.stack([_exact_orth(x) for x in s["x"]])
    return {"sample": _exact_sample, "embed": _exact_embed, "step": _exact_step}[case["op"]](s)
