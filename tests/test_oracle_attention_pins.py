"""The attention and log probability oracles pinned on the CPU: paths run
alone, torch autograd in fp64, finite differences, closed forms."""
import numpy as np
import pytest
import torch

from oracle.attention import tree_attention_reference
from oracle.logprobs import front_rows, tree_logprobs_backward_reference, tree_logprobs_reference

TRIES = [([-1], [7]), ([-1, 0, 0, 2, 2, -1], [4, 3, 1, 2, 5, 3]), ([-1, -1, 0, 1, 0], [2, 3, 1, 2, 2])]


def _visible(parents, lens):
    seg = np.repeat(np.arange(len(lens)), lens)
    n = len(seg)
    m = np.zeros((n, n), bool)
    for i in range(n):
        s = seg[i]
        while s >= 0:
            m[i] |= (seg == s) & (np.arange(n) <= i)
            s = parents[s]
    return m


@pytest.mark.parametrize("trie", TRIES)
@pytest.mark.parametrize("heads", [(1, 1), (4, 2)])
def test_attention_oracle_is_masked_autograd(trie, heads):
    parents, lens = trie
    n, d = sum(lens), 5
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((n, h, d)) for h in (heads[0], heads[1], heads[1]))
    do = rng.standard_normal((n, heads[0], d))
    ref = tree_attention_reference(parents, lens, q, k, v, 0.7, do=do)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    g = heads[0] // heads[1]
    s = torch.einsum("ihd,jhd->hij", tq, tk.repeat_interleave(g, 1)) * 0.7
    s = s.masked_fill(~torch.tensor(_visible(parents, lens)), float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), tv.repeat_interleave(g, 1))
    o.backward(torch.tensor(do))
    for name, t in (("o", o), ("lse", s.logsumexp(-1).t()), ("dq", tq.grad), ("dk", tk.grad), ("dv", tv.grad)):
        np.testing.assert_allclose(ref[name][0], t.detach().numpy(), rtol=1e-12, atol=1e-12)
        assert np.all(ref[name][1] > 0)


def test_front_rows():
    assert front_rows([-1, 0, 0, 2], [2, 1, 2, 1]).tolist() == [-1, 0, 1, 1, 3, 4]
    assert front_rows([-1, -1], [1, 2]).tolist() == [-1, -1, 1]


@pytest.mark.parametrize("trie", TRIES)
def test_logprob_oracle_is_autograd(trie):
    parents, lens = trie
    n, v = sum(lens), 9
    rng = np.random.default_rng(2)
    x, tok = rng.standard_normal((n, v)) * 2, rng.integers(0, v, n)
    tok[-1] = -100
    g, h = rng.standard_normal(n), rng.standard_normal(n)
    f = tree_logprobs_reference(parents, lens, x, tok, 0.6, 3)
    tx = torch.tensor(x, requires_grad=True)
    ls = (tx / 0.6).log_softmax(-1)
    front = front_rows(parents, lens)
    logp = torch.stack([ls[front[t], tok[t]] if front[t] >= 0 and tok[t] >= 0 else ls.sum() * 0 for t in range(n)])
    ent = -(ls.exp() * ls).sum(-1)
    ((logp * torch.tensor(g)).sum() + (ent * torch.tensor(h)).sum()).backward()
    np.testing.assert_allclose(f["logp"][0], logp.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(f["entropy"][0], ent.detach().numpy(), atol=1e-12)
    np.testing.assert_array_equal(f["top_ids"][0], np.argsort(-x, axis=1, kind="stable")[:, :3])
    d, bound = tree_logprobs_backward_reference(parents, lens, x, tok, g, h, 0.6)
    np.testing.assert_allclose(d, tx.grad.numpy(), atol=1e-12)
    assert np.all(bound > 0)


def test_logprob_oracle_closed_forms():
    x = np.zeros((2, 8))
    x[1] = -np.inf
    f = tree_logprobs_reference([-1], [2], x, np.array([0, 3]))
    assert np.allclose(f["logp"][0], [0, -np.log(8)]) and np.allclose(f["entropy"][0], [np.log(8), 0])
    assert f["lse"][0][1] == -np.inf
    d, _ = tree_logprobs_backward_reference([-1], [2], x, np.array([0, 3]), np.ones(2), None)
    assert np.allclose(d[0], np.eye(8)[3] - 1 / 8) and not d[1].any()
