#!/usr/bin/env python3
"""A small routed policy trained by K-FAC steps on the library's objectives.

Contextual bandit: a state belongs to one of ten classes, an action a pays 1
when a % 10 is the state's class.  The network is

    h = dropout(relu(W1 s + b1)),   z = Wr h  (router),   logits = Wa ((1 + p_e u_e) h) + ba

with e the router's choice, p_e its probability and u_e a fixed gain per
expert.  Two phases share it:

  * policy: actions are sampled (Sampler, with their log-probabilities), scored
    under the starting policy (TokenLogp), and a few clipped steps (PolicyLoss
    with its KL term) are taken on them;
  * preference: pairs of short action sequences, the right class preferred to
    a wrong one (PreferenceLoss).

Both add the router's BalanceLoss and use Dropout with one mask per step.
The losses return gradient rows, autograd carries them through the layers,
and the rows each layer received are what its K-FAC factors are built from.
With --step orthogonal the layers take orthogonalised steps in place of K-FAC's.

    python examples/policy_kfac.py [--rounds 12] [--pref-steps 12] [--step kfac]
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from second_order_optimizer_amd import objectives as O      # noqa: E402
from second_order_optimizer_amd.orthogonal import OrthogonalStep      # noqa: E402
from second_order_optimizer_amd.stack import KfacStack      # noqa: E402
from second_order_optimizer_amd.tokens import Sampler       # noqa: E402

CLASSES, ACTIONS, EXPERTS, STATE, HIDDEN = 10, 1000, 4, 32, 128
ROWS, PAIRS, LENGTH = 512, 32, 8                   # 2 * PAIRS * LENGTH = ROWS: one stack serves both phases
HP = dict(lr=0.1, momentum=0.5, weight_decay=0.0, ema_decay=0.9, damping=1e-2)
ORTHOGONAL = dict(lr=0.05, momentum=0.5)


class RoutedPolicy:
    def __init__(self, seed, step="kfac"):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
        shapes = [(STATE, HIDDEN), (HIDDEN, EXPERTS), (HIDDEN, ACTIONS)]
        self.stack = KfacStack([SimpleNamespace(kind="linear", d_in=i, d_out=o, has_bias=True, rows=ROWS)
                                for i, o in shapes], "full")
        for st, (i, o) in zip(self.stack.state, shapes):
            st["w"].copy_(normal(o, i) / i ** 0.5)
        self.gain = 0.5 * normal(EXPERTS, HIDDEN)
        self.centres = normal(CLASSES, STATE)
        self.gen, self.seed, self.passes = gen, seed, 0
        self.drop = O.Dropout(ROWS, HIDDEN, "f32", p=0.1)
        self.balance = O.BalanceLoss(ROWS, EXPERTS, 1, "f32", coef=0.01, z_coef=1e-4, grad_scale=float(ROWS))
        self.score = O.TokenLogp(ROWS, ACTIONS, "f32")
        self.sampler = Sampler(ROWS, ACTIONS, "f32")
        self.orthogonal = None
        if step == "orthogonal":
            self.orthogonal = OrthogonalStep(*[[st[k] for st in self.stack.state] for k in ("w", "mom_w", "b", "mom_b")])

    def states(self, classes):
        return self.centres[classes] + 0.3 * torch.randn(classes.numel(), STATE, generator=self.gen, device="cuda")

    def forward(self, s, train=True):
        """(logits, router logits, chosen experts, inputs and outputs of the three layers)."""
        p = [(st["w"].detach().requires_grad_(train), st["b"].detach().requires_grad_(train))
             for st in self.stack.state]
        pre = torch.nn.functional.linear(s, *p[0])
        h = torch.relu(pre)
        if train:
            self.passes += 1
            h = self.drop.run(h, self.seed, self.passes)      # the mask is made again in the backward pass
        z = torch.nn.functional.linear(h, *p[1])
        prob, expert = torch.softmax(z, 1).max(1)
        y = h * (1 + prob[:, None] * self.gain[expert])
        logits = torch.nn.functional.linear(y, *p[2])
        return logits, z, expert, [(s, pre), (h, z), (y, logits)], p

    def step(self, out, logit_grad):
        """One step from the gradient rows of the logits and the router's balance loss."""
        logits, z, expert, layers, params = out
        stats, counts, _, z_grad = self.balance.run(z.detach(), expert[:, None])
        for _, o in layers:
            o.retain_grad()
        torch.autograd.backward([logits, z], [logit_grad, z_grad])
        for slot, (a, o), (w, b) in zip(self.stack.inputs[0], layers, params):
            slot["a"].copy_(a.detach())
            slot["g"].copy_(o.grad)                       # per-row gradients: the losses ran with grad_scale = rows
            slot["grad_w"].copy_(w.grad / ROWS)
            slot["grad_b"].copy_(b.grad / ROWS)
        if self.orthogonal:
            slots = self.stack.inputs[0]
            self.orthogonal.run([s["grad_w"] for s in slots], [s["grad_b"] for s in slots], **ORTHOGONAL)
        else:
            self.stack.step(KfacStack.hparams(HP))
        return stats, counts


def train(rounds=12, pref_steps=12, seed=0, log=print, step="kfac"):
    """Returns (mean reward of each policy round, preference loss of each step)."""
    net = RoutedPolicy(seed, step)
    classes = torch.arange(ROWS, device="cuda") % CLASSES
    policy = O.PolicyLoss(ROWS, ACTIONS, "f32", clip_low=0.2, clip_high=0.28, kl_coef=0.002, grad_scale=float(ROWS))
    start = [{k: v.clone() for k, v in st.items()} for st in net.stack.state]

    def starting_logp(s, actions):
        """What the untrained network said: the reference of both losses."""
        now = net.stack.state
        net.stack.state = start
        logits = net.forward(s, train=False)[0]
        net.stack.state = now
        return net.score.run(logits, actions)

    rewards, losses = [], []
    for r in range(rounds):
        s = net.states(classes)
        logits = net.forward(s, train=False)[0]
        actions, old, _ = net.sampler.run(logits, torch.rand(ROWS, generator=net.gen, device="cuda"))
        reward = (actions % CLASSES == classes).float()
        advantage = (reward - reward.mean()) / (reward.std() + 1e-3)
        ref = starting_logp(s, actions)
        for _ in range(4):
            out = net.forward(s)
            stats, _, grad = policy.run(out[0].detach(), actions, advantage, old_logp=old, ref_logp=ref)
            balance, counts = net.step(out, grad)
        rewards.append(float(reward.mean()))
        log(f"round {r}: reward {rewards[-1]:.3f}  loss {float(stats[0]):+.4f}  KL {float(stats[2]):.3f}  "
            f"clipped {float(stats[3]):.2f}  balance {float(balance[1]):.4f}  experts {counts.tolist()}")

    pref = O.PreferenceLoss(ROWS, PAIRS, ACTIONS, "f32", beta=0.1, grad_scale=float(ROWS))
    offsets = torch.arange(0, ROWS + 1, LENGTH, dtype=torch.int32, device="cuda")
    for r in range(pref_steps):
        cls = torch.randint(0, CLASSES, (PAIRS,), generator=net.gen, device="cuda")
        wrong = (cls + torch.randint(1, CLASSES, (PAIRS,), generator=net.gen, device="cuda")) % CLASSES
        tens = torch.randint(0, ACTIONS // CLASSES, (2, PAIRS, LENGTH), generator=net.gen, device="cuda")
        actions = (tens * CLASSES + torch.stack([cls, wrong])[:, :, None]).reshape(-1)
        s = net.states(cls.repeat_interleave(LENGTH).repeat(2))
        out = net.forward(s)
        stats, seq, _, grad = pref.run(out[0].detach(), actions, offsets, ref_logp=starting_logp(s, actions))
        net.step(out, grad)
        losses.append(float(stats[0]))
        log(f"preference {r}: loss {losses[-1]:.4f}  in order {float(stats[1]):.2f}")
    flags = [op.flags() for op in (net.score, net.sampler, net.balance, policy, pref)] + [net.stack.flags()]
    if net.orthogonal:
        flags.append(net.orthogonal.flags())
    assert not any(flags), flags
    return rewards, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=12)
    ap.add_argument("--pref-steps", type=int, default=12)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--step", choices=("kfac", "orthogonal"), default="kfac")
    args = ap.parse_args()
    train(args.rounds, args.pref_steps, args.seed, step=args.step)
