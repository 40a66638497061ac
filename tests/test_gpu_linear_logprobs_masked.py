"""Log probabilities from hidden states and the output weight where logits reach
the ends of fp32: entries masked by the lowest number of a type, which fill tiles or
parts of them, and rows whose logits are all that large."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.linear import tree_linear_logprobs_backward_reference, tree_linear_logprobs_reference

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TERMS = {torch.bfloat16: 1, torch.float32: 6}
TRIE = ([-1, 0, 0, 2, 2, 2, -1], [5, 3, 1, 2, 1, 4, 6])
LOW = torch.finfo(torch.bfloat16).min


def np64(t):
    return t.detach().double().cpu().numpy()


def near(name, got, want, bound):
    got = np64(got)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    err = np.where(got == want, 0, np.abs(got - np.where(np.isfinite(want), want, 0)))
    assert np.all(err <= bound), (name, float((err / bound).max()))


@pytest.mark.parametrize("dtype,low", [("bf16", LOW), ("f32", LOW), ("f32", torch.finfo(torch.float32).min)])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("n,first,keep,vocab", [(22, 0, 100, 300), (22, 200, 300, 300), (22, 70, 71, 140),
                                                (300, 0, 1000, 9000), (300, 8000, 9000, 9000),
                                                (1100, 10000, 10300, 10300)])
def test_masked_entries_count_for_nothing(n, first, keep, vocab, temperature, dtype, low):
    """A first column of 1 in hidden adds the lowest number to the logits of all entries but
    first .. keep - 1: the results are those of these entries alone, and the gradients
    of the others are zero."""
    print(f"masked n={n} {first}..{keep} of {vocab} T={temperature} {dtype}", file=sys.stderr, flush=True)
    parents, lens = TRIE if n == 22 else ([-1, 0, 0, 2, 2], [n // 3, n // 4, n // 8, 1, n - n // 3 - n // 4 - n // 8 - 1])
    g = torch.Generator().manual_seed(n + vocab)
    dtype = DT[dtype]
    h = torch.randn((n, 40), generator=g).to(dtype)
    h[:, 0] = 1
    w = (torch.randn((vocab, 40), generator=g) * 0.3).to(dtype)
    w[:, 0] = 0
    masked = torch.ones(vocab, dtype=torch.bool)
    masked[first:keep] = False
    w[masked] = 0
    w[masked, 0] = low
    tok = torch.randint(first, keep, (n,), generator=g)
    dlogp, dent = torch.randn(n, generator=g), torch.randn(n, generator=g) * 0.1
    if masked[0]:
        tok[3] = 0  # a masked token is asked for; without a gradient
        dlogp[3] = 0
    plan = ptp.tree_plan(parents, lens, 4)
    h_, w_, tok_, dl_, de_ = (x.to(DEV) for x in (h, w, tok, dlogp, dent))
    r = ptp.tree_linear_logprobs(h_, w_, tok_, plan, temperature=temperature)
    dh, dw = ptp.tree_linear_logprobs_backward(h_, w_, tok_, r.lse, r.entropy, dl_, plan, dentropy=de_,
                                               temperature=temperature)
    torch.cuda.synchronize()
    few = np64(w)[first:keep]
    t = tok.numpy() - first
    if masked[0]:
        t[3] = -1
    ref = tree_linear_logprobs_reference(parents, lens, np64(h), few, t, temperature, TERMS[dtype])
    if masked[0]:
        # z / T - lse, where lse is far below a rounding of z; past fp32 -inf.
        z = low / temperature
        assert r.logp[3].item() == float("-inf") if z < -3.41e38 else abs(r.logp[3].item() / z - 1) <= 2.0 ** -22
        r.logp[3] = 0
    for name in ("logp", "entropy", "lse"):
        near(name, getattr(r, name), *ref[name])
    ref = tree_linear_logprobs_backward_reference(parents, lens, np64(h), few, t, np64(dlogp), np64(dent), temperature,
                                                  U[dtype], TERMS[dtype])
    near("dhidden", dh, *ref["dhidden"][:2])
    near("dweight", dw[first:keep], *ref["dweight"][:2])
    assert not dw[masked.to(DEV)].any()


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab", [(22, 64), (22, 1000), (300, 9000)])
@pytest.mark.parametrize("x", [1.0e38, 2.0e38, 2.5e38, 3.2e38, -1.0e38, -2.0e38, -2.5e38, -3.2e38])
def test_logits_at_the_ends_of_the_range(x, n, vocab, dtype):
    """All logits of a row equal and large: the entropy is log V and every log probability
    its negative, also where a temperature of 1/4 takes the logits out of fp32's range."""
    print(f"large {x} n={n} vocab={vocab} {dtype}", file=sys.stderr, flush=True)
    h = torch.zeros((n, 8), dtype=DT[dtype], device=DEV)
    h[:, 0] = 1
    w = torch.zeros((vocab, 8), dtype=DT[dtype], device=DEV)
    w[:, 0] = x
    tok = torch.arange(n, device=DEV) % vocab
    plan = ptp.tree_plan([-1], [n], 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    torch.cuda.synchronize()
    # exp(0) = 1 is exact and so are sums of ones; the logarithm, its product with log(2) and
    # the largest logit's are off by a rounding or two each.
    log_v = np.log(vocab)
    assert (r.entropy.double() - log_v).abs().max() <= 4 * 2.0 ** -24 * log_v
    assert (r.logp[1:].double() + log_v).abs().max() <= 4 * 2.0 ** -24 * log_v + 1e-12
    value = w[0, 0].double().item()
    assert (r.lse.double() / value - 1).abs().max() <= 2.0 ** -23
    r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=0.25)
    torch.cuda.synchronize()
    assert (r.entropy.double() - log_v).abs().max() <= 4 * 2.0 ** -24 * log_v
    assert (r.logp[1:].double() + log_v).abs().max() <= 4 * 2.0 ** -24 * log_v + 1e-12
    assert (r.lse == torch.finfo(torch.float32).max * (1 if x > 0 else -1)).all()


@pytest.mark.parametrize("dtype", sorted(DT))
def test_far_from_the_largest(dtype):
    """One entry at the top of the range, the others at its bottom, further apart than fp32
    reaches: a log probability in range is finite where the temperature brings it there."""
    h = torch.zeros((4, 8), dtype=DT[dtype], device=DEV)
    h[:, 0] = 1
    w = torch.zeros((700, 8), dtype=DT[dtype], device=DEV)
    w[:, 0] = -3.2e38
    w[300, 0] = 3.2e38
    big = w[300, 0].double().item()
    tok = torch.tensor([0, 300, 5, 699], device=DEV)
    plan = ptp.tree_plan([-1], [4], 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=4.0)
    torch.cuda.synchronize()
    assert r.logp[1] == 0 and not r.entropy.any()
    assert ((r.lse.double() * 4 / big - 1).abs() <= 2.0 ** -22).all()
    assert ((r.logp[2:].double() * -2 / big - 1).abs() <= 2.0 ** -22).all()
