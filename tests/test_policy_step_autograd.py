"""The policy update's autograd functions: second derivatives are refused, not
left out, and expanded gradients are taken."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from prefix_tree_packed_plan_amd import policy_step as ps


def stand_ins(monkeypatch):
    """The library's calls replaced by elementwise products, on the CPU."""
    monkeypatch.setattr(ptp, "tree_conv", lambda x, w, plan, act: x * w)
    monkeypatch.setattr(ptp, "tree_conv_backward", lambda x, w, dy, plan, act: (dy * w, dy * x, None, None))
    monkeypatch.setattr(ptp, "tree_gdn_scan", lambda q, k, v, g, b, plan, return_states: (q * k * v * g * b, q))
    monkeypatch.setattr(ptp, "tree_gdn_scan_backward", lambda q, k, v, g, b, do, plan, st: (
        do * k * v * g * b, do * q * v * g * b, do * q * k * g * b, do * q * k * v * b, do * q * k * v * g, None))
    monkeypatch.setattr(ptp, "tree_attention", lambda q, k, v, plan, return_lse: (q * k * v, q.detach()))
    monkeypatch.setattr(ptp, "tree_attention_backward", lambda q, k, v, o, lse, do, plan: (
        do * k * v, do * q * v, do * q * k))
    monkeypatch.setattr(ptp, "tree_logprobs", lambda x, t, plan, temperature: ptp.TokenLogprobs(
        x * x, x * 2, x.detach(), None, None))
    monkeypatch.setattr(ptp, "tree_logprobs_backward", lambda x, t, lse, h, dlogp, plan, dentropy, temperature: (
        2 * x * dlogp + 2 * dentropy))


CALLS = {
    "conv": lambda x: ps.Conv.apply(x, x + 1, None),
    "scan": lambda x: ps.Scan.apply(x, x + 1, x + 2, x + 3, x + 4, None),
    "attention": lambda x: ps.Attention.apply(x, x + 1, x + 2, None),
    "logprobs": lambda x: sum(ps.Logprobs.apply(x, None, None, 1.0)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_second_derivatives_are_refused(name, monkeypatch):
    stand_ins(monkeypatch)
    x = torch.randn(3, 4, requires_grad=True)
    y = CALLS[name](x)
    (g,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g * g).sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("part", ["sum", "row"])
def test_attention_takes_expanded_gradients(part):
    """The gradient of o.sum() is one number repeated, of a sum over heads a
    row repeated."""
    plan = ptp.tree_plan([-1, 0, 0], [40, 30, 20], 4)
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((90, h, 32), generator=gen).to("cuda:0") for h in (4, 2, 2))
    w = torch.randn((90, 1, 32), generator=gen).to("cuda:0")

    def grads(spread):
        t = [x.clone().requires_grad_() for x in (q, k, v)]
        o = ps.Attention.apply(*t, plan)
        if spread:
            loss = o.sum() if part == "sum" else (o.sum(1, keepdim=True) * w).sum()
            loss.backward()
        else:
            o.backward((torch.ones_like(o) if part == "sum" else w.expand_as(o)).contiguous())
        torch.cuda.synchronize()
        return [x.grad for x in t]

    print(f"expanded gradients, {part}", file=sys.stderr, flush=True)
    assert all(torch.equal(a, b) for a, b in zip(grads(True), grads(False)))
