"""The policy update program (conv, scan, attention, log probabilities, forward
and backward together) against torch autograd over every root-to-leaf path in
fp64, and its training steps."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from prefix_tree_packed_plan_amd import policy_step as ps

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def plain_loss(model, tokens, advantage, parents, lens, temperature, bonus):
    """The same loss, every token's value taken from a path through it run
    alone, token by token for the recurrence, in fp64 on the CPU."""
    W = [w.detach().double().cpu().requires_grad_() for w in model.weights]
    embed, conv, mix, gate, wqkv = W
    tok, adv = tokens.cpu(), advantage.double().cpu()
    h, kv, d = model.heads, model.kv, model.d
    c = h * d
    off = np.concatenate([[0], np.cumsum(lens)])
    paths = []
    for s, p in enumerate(parents):
        mine = list(range(off[s], off[s + 1]))
        paths.append(mine if p < 0 else paths[p] + mine)
    total = 0.0
    for s in range(len(parents)):
        rows = paths[s]
        n, new = len(rows), int(lens[s])
        x = embed[tok[rows]]
        xin = torch.cat([torch.zeros(3, c, dtype=torch.float64), x])
        y = torch.nn.functional.silu(sum(xin[i:i + n] * conv[:, i] for i in range(4)))
        q, k, v = (y @ mix).view(n, 3, h, d).unbind(1)
        q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
        g, beta = (y @ gate).view(n, 2, h).unbind(1)
        a, beta = torch.exp(-torch.nn.functional.softplus(g)), torch.sigmoid(beta)
        S = torch.zeros(h, d, d, dtype=torch.float64)  # [h, d_k, d_v]
        outs = []
        for t in range(n):
            kt, b = k[t], beta[t][:, None, None]
            S = a[t][:, None, None] * (S - b * kt[:, :, None] * (kt[:, None, :] @ S)) + b * kt[:, :, None] * v[t][:, None, :]
            outs.append((q[t][:, None, :] @ S)[:, 0])
        x = x + torch.stack(outs).reshape(n, c)
        qkv = (x @ wqkv).view(n, h + 2 * kv, d)
        kk, vv = (qkv[:, i:i + kv].repeat_interleave(h // kv, 1) for i in (h, h + kv))
        sc = torch.einsum("ihd,jhd->hij", qkv[:, :h], kk) * d ** -0.5
        sc = sc.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool), 1), float("-inf"))
        x = x + torch.einsum("hij,jhd->ihd", sc.softmax(-1), vv).reshape(n, c)
        ls = ((x @ embed.t()) * c ** -0.5 / temperature).log_softmax(-1)
        for i in range(n - new, n):  # this segment's own tokens and rows
            if i > 0:
                total = total + adv[rows[i]] * ls[i - 1, tok[rows[i]]]
            total = total - bonus * (ls[i].exp() * ls[i]).sum()
    loss = -total / len(tok)
    loss.backward()
    return loss.item(), [w.grad for w in W]


def test_gradients_are_those_of_every_path_alone():
    parents, lens = [-1, 0, 0, 1, 1, -1], [9, 5, 7, 3, 4, 6]
    model = ps.Model(vocab=37, heads=2, d=32, dtype=torch.float32, device=DEV, seed=3)
    gen = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, 37, (sum(lens),), generator=gen).to(DEV)
    adv = torch.randn(sum(lens), generator=gen).to(DEV)
    plan = ptp.tree_plan(parents, lens, 4)
    loss = ps.policy_loss(model, tokens, adv, plan, temperature=0.8, entropy_bonus=0.1)
    loss.backward()
    torch.cuda.synchronize()
    want, grads = plain_loss(model, tokens, adv, parents, lens, 0.8, 0.1)
    print(f"loss {loss.item():.7f} {want:.7f}", file=sys.stderr, flush=True)
    # fp32 throughout; the scan splits its operands into two bf16 parts (2^-16
    # of a product's size), the loosest step on the way.
    assert abs(loss.item() - want) <= 1e-4 * abs(want)
    for w, g in zip(model.weights, grads):
        err = (w.grad.double().cpu() - g).norm() / g.norm()
        print(f"  gradient {tuple(w.shape)}: relative error {err:.2e}", file=sys.stderr, flush=True)
        assert err <= 1e-3


def test_steps_lower_the_loss():
    def run():
        model = ps.Model(vocab=1003, heads=4, d=64, dtype=torch.bfloat16, device=DEV)
        tokens, adv, plan = ps.rollouts(1003, DEV)
        losses = [ps.policy_step(model, tokens, adv, plan, lr=0.5).item() for _ in range(6)]
        return losses, model.conv.detach().clone(), model.qkv.detach().clone()

    losses, conv, qkv = run()
    print(losses, file=sys.stderr, flush=True)
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]
    again, conv2, qkv2 = run()  # the embedding gradient (a scatter of torch) is not bitwise repeatable
    assert abs(again[0] - losses[0]) == 0 and torch.isfinite(conv2.float()).all() and torch.isfinite(qkv2.float()).all()
