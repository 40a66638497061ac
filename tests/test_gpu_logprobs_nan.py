"""Rows of logits that hold NaN: the most likely tokens among the other columns."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from tests.test_gpu_logprobs import DEV, DT, TRIE, inputs, np64

pytestmark = pytest.mark.gpu

LONG = ([-1, 0, 0], [200, 250, 150])


def best(x, k):
    """Ids of each row's k largest values, NaN left out (-1: none left)."""
    out = np.full((x.shape[0], k), -1)
    for i, row in enumerate(x):
        ids = np.argsort(-row, kind="stable")
        ids = ids[~np.isnan(row[ids])][:k]
        out[i, :len(ids)] = ids
    return out


@pytest.mark.parametrize("k", [1, 2, 5, 16, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alternatives_beside_nan(dtype, k):
    """Whole 16-byte pieces of NaN, most of a row, all but a few columns."""
    for trie in (TRIE, LONG):
        n = sum(trie[1])
        print(f"alternatives beside NaN k={k} {dtype} rows={n}", file=sys.stderr, flush=True)
        x, tok, _, _ = inputs(n, 3000, DT[dtype], seed=13)
        rng = np.random.default_rng(k)
        nan = float("nan")
        x[1, :1500] = nan
        x[2, 1500:] = nan
        for i in range(3, 15):
            pieces = torch.as_tensor(rng.random(375) < i / 15).repeat_interleave(8).to(DEV)
            x[i, pieces] = nan
        only = x[15, [5, 100, 2000]].clone()
        x[15] = nan
        x[15, [5, 100, 2000]] = only
        x[16, 1::2] = nan
        got = ptp.tree_logprobs(x, tok, ptp.tree_plan(*trie, 4), top_k=k).top_ids.cpu().numpy()
        assert np.array_equal(got, best(np64(x), k))
