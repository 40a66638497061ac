"""Pins of oracle/linear.py: against torch autograd over every path alone, against
differences, and its bounds against arithmetic with the roundings they are for."""
import numpy as np
import pytest
import torch

from oracle.linear import tree_linear_logprobs_backward_reference, tree_linear_logprobs_reference

TRIE = ([-1, 0, 0, 2, 2, -1], [4, 3, 1, 2, 1, 3])
N, V, C, T = 14, 23, 8, 0.7


def case(seed=0):
    r = np.random.default_rng(seed)
    h, w = r.normal(size=(N, C)), r.normal(size=(V, C)) * 0.7
    tok = r.integers(0, V, size=N)
    tok[6], tok[8] = -1, V
    return h, w, tok, r.normal(size=N), r.normal(size=N) * 0.3


def paths():
    off = np.concatenate([[0], np.cumsum(TRIE[1])])
    rows = []
    for s, p in enumerate(TRIE[0]):
        mine = list(range(off[s], off[s + 1]))
        rows.append(mine if p < 0 else rows[p] + mine)
    return rows


def loss_of(h, w, tok, dlogp, dent):
    """sum dlogp logp + sum dentropy entropy, each token on its own path."""
    total, logps = 0.0, {}
    for s, rows in enumerate(paths()):
        ls = (h[rows] @ w.T / T).log_softmax(-1)
        new = TRIE[1][s]
        for i in range(len(rows) - new, len(rows)):
            if i > 0 and 0 <= tok[rows[i]] < V:
                logps[rows[i]] = ls[i - 1, tok[rows[i]]]
                total = total + dlogp[rows[i]] * logps[rows[i]]
            total = total - dent[rows[i]] * (ls[i].exp() * ls[i]).sum()
    return total, logps


def test_values_and_gradients_are_those_of_every_path_alone():
    h, w, tok, dlogp, dent = case()
    th, tw = (torch.tensor(x, requires_grad=True) for x in (h, w))
    total, logps = loss_of(th, tw, tok, dlogp, dent)
    total.backward()
    r = tree_linear_logprobs_reference(*TRIE, h, w, tok, T)
    for t in range(N):
        assert r["logp"][0][t] == pytest.approx(logps[t].item() if t in logps else 0.0, abs=1e-12)
    g = tree_linear_logprobs_backward_reference(*TRIE, h, w, tok, dlogp, dent, T)
    assert np.allclose(g["dhidden"][0], th.grad.numpy(), atol=1e-12)
    assert np.allclose(g["dweight"][0], tw.grad.numpy(), atol=1e-12)


def test_gradients_against_differences():
    h, w, tok, dlogp, dent = case(1)
    g = tree_linear_logprobs_backward_reference(*TRIE, h, w, tok, dlogp, dent, T)

    def loss(h, w):
        r = tree_linear_logprobs_reference(*TRIE, h, w, tok, T)
        return (dlogp * r["logp"][0]).sum() + (dent * r["entropy"][0]).sum()

    eps = 1e-5
    for x, name in ((h, "dhidden"), (w, "dweight")):
        for i in range(0, x.size, 7):
            at = np.unravel_index(i, x.shape)
            keep = x[at]
            x[at] = keep + eps
            up = loss(h, w)
            x[at] = keep - eps
            down = loss(h, w)
            x[at] = keep
            assert (up - down) / (2 * eps) == pytest.approx(g[name][0][at], abs=1e-7)


def test_bounds_hold_for_fp32_arithmetic_with_bf16_operands():
    """The formulas in fp32 with the logits' gradient rounded to bf16 stay inside the
    bounds, and near the root mean square of the roundings; a lost vocabulary entry
    does not."""
    h, w, tok, dlogp, dent = case(2)
    th, tw = (torch.tensor(x).to(torch.bfloat16) for x in (h, w))
    h, w = th.double().numpy(), tw.double().numpy()
    g = tree_linear_logprobs_backward_reference(*TRIE, h, w, tok, dlogp, dent, T)
    z = (th.float() @ tw.float().T / T).requires_grad_()
    ls = z.log_softmax(-1)
    off = np.concatenate([[0], np.cumsum(TRIE[1])])
    total = 0.0
    for s, p in enumerate(TRIE[0]):
        for t in range(off[s], off[s + 1]):
            front = t - 1 if t > off[s] else (off[p + 1] - 1 if p >= 0 else -1)
            if front >= 0 and 0 <= tok[t] < V:
                total = total + float(dlogp[t]) * ls[front, int(tok[t])]
    total = total - (torch.tensor(dent).float()[:, None] * ls.exp() * ls).sum()
    total.backward()
    d = (z.grad / T).to(torch.bfloat16).float()

    def ratios(d):
        out = []
        for name, x in (("dhidden", d @ tw.float()), ("dweight", d.T @ th.float())):
            err = np.abs(x.to(torch.bfloat16).double().numpy() - g[name][0])
            out.append((bool(np.all(err <= g[name][1])), np.sqrt(((err / g[name][2]) ** 2).mean())))
        return out

    for ok, rms in ratios(d):
        assert ok and 0.2 < rms < 1.0
    d[:, 5] = 0
    assert any(not ok or rms > 2.0 for ok, rms in ratios(d))
