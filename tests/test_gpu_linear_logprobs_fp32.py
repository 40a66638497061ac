"""fp32 gradients of log probabilities from hidden states and the output weight,
held to fp32's accuracy: the exponentials of far entries."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp

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
