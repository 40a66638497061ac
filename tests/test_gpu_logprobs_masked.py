"""Token log probabilities where most logits, or all of a row, are large finite
numbers (masks of -1e9, -1e30, the type's lowest value, at several
temperatures), against the fp64 oracle: a mask must cost the other columns
nothing, wherever the masked columns are met first.  And +inf, which makes its
row NaN."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.logprobs import U32, tree_logprobs_reference
from tests.test_gpu_logprobs import DEV, DT, TRIE, check, inputs, np64, run_case

pytestmark = pytest.mark.gpu

LONG = ([-1, 0, 0], [200, 250, 150])  # 600 rows: one work-group each; TRIE's 22 are spread over several
FMAX = float(np.finfo(np.float32).max)


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def value(filler, dtype):
    return torch.finfo(dtype).min if filler == "lowest" else filler


@pytest.mark.parametrize("trie", [TRIE, LONG], ids=["spread rows", "whole rows"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.3, 1.0, 2.0])
@pytest.mark.parametrize("filler", [-1e9, -1e10, -1e30, "lowest"])
def test_logprobs_of_a_vocabulary_masked_by_large_numbers(filler, temperature, dtype, trie):
    """Allowed columns in the middle: whole slices, and every lane's first
    columns, are masked."""
    say(f"logprobs mask {filler} T={temperature} {dtype} rows={sum(trie[1])}")
    x, tok, dlogp, dent = inputs(sum(trie[1]), 6007, DT[dtype], seed=5)
    fill = value(filler, x.dtype)
    x[:, :3500] = fill
    x[:, 4300:] = fill
    run_case(*trie, x, 3500 + tok % 800, dlogp, dent, temperature, top_k=5)


@pytest.mark.parametrize("allowed", ["first", "last", "one", "few"])
def test_logprobs_mask_patterns(allowed):
    for dtype in DT.values():
        say(f"logprobs mask pattern {allowed} {dtype}")
        x, tok, dlogp, dent = inputs(22, 6007, dtype, seed=8)
        keep = torch.zeros(6007, dtype=torch.bool)
        ids = {"first": torch.arange(900), "last": torch.arange(6004, 6007), "one": torch.tensor([4001]),
               "few": torch.randperm(6007, generator=torch.Generator().manual_seed(1))[:60]}[allowed].to(DEV)
        keep[ids.cpu()] = True
        x[:, ~keep.to(DEV)] = -1e10
        run_case(*TRIE, x, ids[tok % len(ids)], dlogp, dent, top_k=min(3, len(ids)))


def forward_case(parents, lens, x, tok, temperature):
    """The forward against the oracle.  Values of any size: a product with 1 / T
    (rounded), log2 e (rounded), a difference, and ln 2 (rounded) are 8 half
    units; lse is held at the type's largest value."""
    r = ptp.tree_logprobs(x, tok, ptp.tree_plan(parents, lens, 4), temperature=temperature, top_k=3)
    torch.cuda.synchronize()
    ref = tree_logprobs_reference(parents, lens, np64(x), tok.cpu().numpy(), temperature, 3)
    for name in ("logp", "entropy", "lse", "top_logp"):
        want, bound = ref[name]
        with np.errstate(over="ignore"):
            check(name, getattr(r, name), np.clip(want, -FMAX, FMAX), bound + 4 * U32 * np.abs(want))
    assert np.array_equal(r.top_ids.cpu().numpy(), ref["top_ids"][0])
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.3, 1.0, 2.0])
def test_logprobs_of_rows_without_an_ordinary_value(temperature, dtype):
    """Rows of one large value (their columns share the probability), of two,
    of random large values, with one value far above the rest."""
    for trie in (TRIE, LONG):
        say(f"logprobs rows of large values T={temperature} {dtype} rows={sum(trie[1])}")
        x, tok, _, _ = inputs(sum(trie[1]), 6007, DT[dtype], seed=6)
        for i, fill in enumerate((-1e9, -1e10, -1e30, "lowest", 1e9, 1e30, -5e6, 5e6)):
            x[i] = value(fill, x.dtype)
        x[8, ::2], x[8, 1::2] = -1e9, -1.5e9
        x[9] *= 1e9
        x[10, 77] = 1e10
        x[11, 77:90] = 1e30
        x[12] -= 3e6
        x[13] -= 1e8
        x[14] += 2e7
        forward_case(*trie, x, tok, temperature)


def test_logprobs_of_masked_tokens():
    """Log probabilities of the masked tokens themselves."""
    x, tok, _, _ = inputs(22, 6007, torch.float32, seed=7)
    for fill in (-1e4, -1e9, -1e30):
        for temperature in (0.3, 1.0, 2.0):
            say(f"logprobs masked tokens {fill} T={temperature}")
            x[:, 1000:] = fill
            forward_case(*TRIE, x, 1000 + tok % 5000, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_positive_infinity_makes_its_row_nan(dtype):
    """lse, entropy, the log probabilities behind the row and its gradient; no
    other row."""
    for trie in (TRIE, LONG):
        n = sum(trie[1])
        say(f"logprobs +inf {dtype} rows={n}")
        x, tok, dlogp, dent = inputs(n, 3000, DT[dtype], seed=15)
        plan = ptp.tree_plan(*trie, 4)
        a = ptp.tree_logprobs(x, tok, plan, top_k=3)
        da = ptp.tree_logprobs_backward(x, tok, a.lse, a.entropy, dlogp, plan, dentropy=dent)
        y = x.clone()
        y[9, 1234] = float("inf")  # rows 10 and 15 are the next of their segments
        y[14, :3] = float("inf")
        rows = torch.zeros(n, dtype=torch.bool, device=DEV)
        rows[[9, 14]] = True
        behind = torch.zeros_like(rows)
        behind[[10, 15]] = True
        b = ptp.tree_logprobs(y, tok, plan, top_k=3)
        assert torch.isnan(b.lse[rows]).all() and torch.isnan(b.entropy[rows]).all()
        assert torch.isnan(b.logp[behind]).all() and torch.isnan(b.top_logp[rows]).all()
        assert b.top_ids[9, 0] == 1234 and b.top_ids[14].tolist() == [0, 1, 2]
        assert torch.equal(a.lse[~rows], b.lse[~rows]) and torch.equal(a.logp[~behind], b.logp[~behind])
        for h in (dent, None):
            db = ptp.tree_logprobs_backward(y, tok, b.lse, b.entropy, dlogp, plan, dentropy=h)
            assert torch.isnan(db[rows]).all() and torch.isfinite(db[~rows]).all()
            if h is not None:
                assert torch.equal(da[~rows], db[~rows])
