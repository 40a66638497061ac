"""Log probabilities from hidden states and the output weight on tries of very many
segments: a wave looks at each for the tokens behind a call's rows."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.linear import tree_linear_logprobs_reference

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# A root of two tokens, a child of one with two of its own, two more children.
PARENTS, LENS = [-1, 0, 1, 1, 0, 0], [2, 1, 2, 1, 1, 3]


@pytest.mark.parametrize("between", [0, 1000, 300_001, (1 << 26) + 5])
def test_segments_past_a_launch(between):
    """That trie, `between` roots of one token and that trie again: more segments than a
    launch has waves for (2^18 to 2^19), and than 2^32 work items."""
    print(f"segments between={between}", file=sys.stderr, flush=True)
    k, n = len(PARENTS), sum(LENS)
    parents = np.full(between + 2 * k, -1, np.int32)
    parents[:k] = PARENTS
    parents[k + between:] = [p + k + between if p >= 0 else -1 for p in PARENTS]
    lens = np.ones(len(parents), np.int32)
    lens[:k] = lens[k + between:] = LENS
    plan = ptp.tree_plan(parents, lens, 1)
    print("  plan made", file=sys.stderr, flush=True)
    total = between + 2 * n
    assert plan.n_tokens == total
    g = torch.Generator().manual_seed(3)
    h = torch.randn((n, 16), generator=g).to(torch.bfloat16)
    w = torch.randn((300, 16), generator=g).to(torch.bfloat16)
    tok = torch.randint(0, 300, (n,), generator=g, dtype=torch.int32)
    tokens = torch.zeros(total, dtype=torch.int32, device=DEV)
    tokens[:n] = tokens[total - n:] = tok.to(DEV)
    ref = tree_linear_logprobs_reference(PARENTS, LENS, h.double().numpy(), w.double().numpy(), tok.numpy())
    logp = torch.full((total,), 5.0, device=DEV)
    for first in (0, total - n):
        r = ptp.tree_linear_logprobs(h.to(DEV), w.to(DEV), tokens, plan, first_row=first, logp=logp)
        torch.cuda.synchronize()
        for name, got in (("logp", logp[first:first + n]), ("entropy", r.entropy), ("lse", r.lse)):
            want, bound = ref[name]
            assert (np.abs(got.double().cpu().numpy() - want) <= bound).all(), (first, name)
        if first == 0:
            assert (logp[n:] == 5).all()  # tokens behind other rows are left
        else:
            assert (logp[n:first] == 5).all()
