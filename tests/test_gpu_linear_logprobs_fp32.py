"""fp32 gradients of log probabilities from hidden states and the output weight,
held to fp32's accuracy: the exponentials of far entries, and each of the six
partial products that stand for a product of two fp32 numbers."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.split import SPLIT_CASES, SPLIT_REL, SPLIT_RMS, split_exact, split_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("n", [64, 200])
@pytest.mark.parametrize("vocab", [40, 700])
def test_exponentials_of_far_entries(n, vocab):
    """Logits of 0, a log-sum-exp of 40 to 70 as given and hidden states of the unit
    matrix: dweight holds -exp(-lse) itself."""
    print(f"far entries n={n} vocab={vocab}", file=sys.stderr, flush=True)
    h = torch.eye(n, device=DEV)
    w = torch.zeros((vocab, n), device=DEV)
    tok = torch.full((n,), vocab - 1, device=DEV)
    lse = torch.linspace(40, 70, n, device=DEV)
    _, dw = ptp.tree_linear_logprobs_backward(h, w, tok, lse, None, torch.ones(n, device=DEV),
                                              ptp.tree_plan([-1], [n], 4))
    torch.cuda.synchronize()
    want = -torch.exp(-lse.double())
    # Roundings of 2^-24: two of the exponential, one of its correction, one of the
    # coefficient, three of the sum of its parts.  (The constant's alone would be 2^-26 x 70.)
    worst = (dw[:-1, :-1].double() / want[:-1] - 1).abs().max().item()
    assert worst <= 7 * 2.0 ** -24, worst


@pytest.mark.parametrize("n,vocab,width", SPLIT_CASES)
def test_six_partial_products(n, vocab, width):
    """The errors' size over the whole result, which no worst case's bound holds to a
    partial product: leaving one out of the products makes it three times the limit or more
    (the oracle's test plants that)."""
    print(f"six products n={n} vocab={vocab} width={width}", file=sys.stderr, flush=True)
    parents, lens, h, w, tok, dlogp = (x.to(DEV) if isinstance(x, torch.Tensor) else x
                                       for x in split_inputs(n, vocab, width))
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    dh, dw = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, None, dlogp, plan)
    torch.cuda.synchronize()
    logp, want_dh, want_dw = split_exact(parents, lens, h, w, tok, dlogp)
    for name, got, want, most in (("logp", r.logp, logp, SPLIT_RMS), ("dhidden", dh, want_dh, SPLIT_REL),
                                  ("dweight", dw, want_dw, SPLIT_REL)):
        err = (got.double() - want).norm().item() / (len(want) ** 0.5 if name == "logp" else want.norm().item())
        print(f"  {name}: {err:.2e}, limit {most:.2e}", file=sys.stderr, flush=True)
        assert err <= most, name
