"""The policy update without logits: embedding and linear log probabilities with
their gradients, run together with the mixer and the attention, against torch
autograd over the logits in fp64 and against the path that keeps them; and the
two autograd functions' refusals."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from prefix_tree_packed_plan_amd import policy_step as ps

DEV = "cuda:0"
PARENTS, LENS = [-1, 0, 0, 1, 1, -1], [9, 5, 7, 3, 4, 6]


def stand_ins(monkeypatch):
    """The library's calls replaced by elementwise products, on the CPU."""
    monkeypatch.setattr(ptp, "tree_embedding", lambda tokens, table: table * table)
    monkeypatch.setattr(ptp, "tree_embedding_backward", lambda tokens, d, vocab: 2 * d)
    monkeypatch.setattr(ptp, "tree_linear_logprobs", lambda x, w, t, plan, temperature: ptp.TokenLogprobs(
        x * w, x * 2, x.detach(), None, None))
    monkeypatch.setattr(ptp, "tree_linear_logprobs_backward", lambda x, w, t, lse, h, dlogp, plan, dentropy, temperature: (
        w * dlogp + 2 * dentropy, x * dlogp))


CALLS = {
    "embedding": lambda x: ps.Embedding.apply(torch.zeros(3), x),
    "linear": lambda x: sum(ps.LinearLogprobs.apply(x, x + 1, torch.zeros(3), None, 1.0)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_second_derivatives_are_refused(name, monkeypatch):
    stand_ins(monkeypatch)
    x = torch.randn(3, 4, requires_grad=True)
    y = CALLS[name](x)
    (g,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g * g).sum().backward()


def plain(hidden, weight, tokens, parents, lens, temperature):
    """(logp, entropy) in fp64 with autograd: a token's from the row in front of it."""
    ls = (hidden @ weight.t() / temperature).log_softmax(-1)
    first = [sum(lens[:s]) for s in range(len(lens))]
    front = []
    for s, p in enumerate(parents):
        front += [first[p] + lens[p] - 1 if p >= 0 else -1] + list(range(first[s], first[s] + lens[s] - 1))
    front = torch.tensor(front)
    logp = torch.where(front >= 0, ls[front.clamp(min=0), tokens], 0.0)
    return logp, -(ls.exp() * ls).sum(-1)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [False, True])
def test_functions_together(spread):
    """One table looked up and multiplied with: both gradients meet in it, and the
    gradient of a sum (one number repeated) is taken."""
    gen = torch.Generator().manual_seed(7)
    n = sum(LENS)
    plan = ptp.tree_plan(PARENTS, LENS, 4)
    tokens = torch.randint(0, 53, (n,), generator=gen)
    start = torch.randn((53, 24), generator=gen)
    da, db = (torch.ones(n), torch.ones(n)) if spread else torch.randn((2, n), generator=gen)

    def loss(logp, entropy, da, db):
        return (logp.sum() + entropy.sum()) if spread else (logp * da).sum() + (entropy * db).sum()

    table = start.to(DEV).requires_grad_()
    x = ps.Embedding.apply(tokens.to(DEV), table)
    got = ps.LinearLogprobs.apply(x, table, tokens.to(DEV), plan, 1.7)
    loss(*got, da.to(DEV), db.to(DEV)).backward()
    torch.cuda.synchronize()
    ref = start.double().requires_grad_()
    want = plain(ref[tokens], ref, tokens, PARENTS, LENS, 1.7)
    loss(*want, da.double(), db.double()).backward()
    # 24 products of a logit and 53 of a gradient, sums of up to 53 terms in fp32
    # (2^-24 each), a handful of roundings around them: 2^-24 * 128 of the norms.
    for a, b in zip((*got, table.grad), (*want, ref.grad)):
        assert (a.detach().double().cpu() - b.detach()).norm() <= 128 * 2.0 ** -24 * b.detach().norm()


@pytest.mark.gpu
def test_update_is_that_with_logits():
    model = ps.Model(vocab=37, heads=2, d=32, dtype=torch.float32, device=DEV, seed=3)
    gen = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, 37, (sum(LENS),), generator=gen).to(DEV)
    adv = torch.randn(sum(LENS), generator=gen).to(DEV)
    plan = ptp.tree_plan(PARENTS, LENS, 4)

    def run(keep):
        for w in model.weights:
            w.grad = None
        loss = ps.policy_loss(model, tokens, adv, plan, temperature=0.8, entropy_bonus=0.1, keep_logits=keep)
        loss.backward()
        torch.cuda.synchronize()
        return loss.item(), [w.grad.clone() for w in model.weights]

    (a, ga), (b, gb), (c, gc) = run(True), run(False), run(False)
    # The operators that differ err by some 2^-24 of their results; the scan's two
    # bf16 parts (2^-16) carry that on, in the loosest step on the way.
    assert abs(a - b) <= 1e-4 * abs(a)
    for x, y in zip(ga, gb):
        assert (x - y).norm() <= 1e-3 * x.norm()
    assert b == c and all(torch.equal(x, y) for x, y in zip(gb, gc))


@pytest.mark.gpu
def test_steps_are_repeatable_bit_by_bit():
    def run():
        model = ps.Model(vocab=1003, heads=4, d=64, dtype=torch.bfloat16, device=DEV)
        tokens, adv, plan = ps.rollouts(1003, DEV)
        for _ in range(3):
            ps.policy_step(model, tokens, adv, plan, keep_logits=False)
        return [w.detach().clone() for w in model.weights]

    first, second = run(), run()
    assert all(torch.isfinite(w.float()).all() for w in first)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.gpu
def test_command_runs():
    out = subprocess.run([sys.executable, "-m", "prefix_tree_packed_plan_amd.policy_step", "--no-logits"],
                         cwd=Path(__file__).parents[1], capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr
    assert out.stdout.count("loss") == 8
