"""Tree attention where the scaled scores are far beyond 2^24: a softmax that
has become a choice of the largest, ties sharing it."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.attention import tree_attention_reference
from tests.test_gpu_attention import DEV, DT, U, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [8, 14, 20, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("trie", [([-1], [40]), ([-1, 0, 0, 2], [100, 60, 90, 33]), ([-1], [1500])])
def test_attention_of_large_scores(trie, dtype, power):
    """q and k of small whole numbers times powers of 2: every score is exact in
    fp32, and so are the ties.  With whole scores apart by 2^(2 power - 3), a
    probability is 0 or 1 / the number of ties, but for the roundings of a bf16
    or fp32 probability and the sum."""
    n, d, hq, hkv = sum(trie[1]), 32, 2, 1
    print(f"attention large scores 2^{2 * power} {dtype} N={n}", file=sys.stderr, flush=True)
    g = torch.Generator().manual_seed(power)
    q, k = (torch.randint(-2, 3, (n, h, d), generator=g) * 2.0 ** power for h in (hq, hkv))
    v = torch.randn((n, hkv, d), generator=g)
    q, k, v = (t.to(DT[dtype]).to(DEV) for t in (q, k, v))
    o, lse = ptp.tree_attention(q, k, v, ptp.tree_plan(*trie, 4), scale=0.125, return_lse=True)
    torch.cuda.synchronize()
    ref = tree_attention_reference(*trie, np64(q), np64(k), np64(v), 0.125, u=U[DT[dtype]])
    # A row of n equal probabilities sums at most n |v| 2^-24 and rounds each to u; o itself rounds to u.
    bound = (2 * U[DT[dtype]] + (n + 8) * 2.0 ** -24) * np.abs(np64(v)).max()
    err = np.abs(np64(o) - ref["o"][0])
    print(f"  worst error {float(err.max()):.3e} of {bound:.3e}", file=sys.stderr, flush=True)
    assert np.all(err <= bound)
    # log2 e rounded, its product, a logarithm, ln 2 rounded and its product.
    want = ref["lse"][0]
    assert np.all(np.abs(np64(lse) - want) <= 6 * 2.0 ** -24 * (1 + np.abs(want)) + n * 2.0 ** -24)
