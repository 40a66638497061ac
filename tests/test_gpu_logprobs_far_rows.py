"""The logits' gradient of rows whose log-sum-exp is so large that fp32 cannot
hold its last digits (rows masked throughout by finite numbers, logits of
1e5 and more): forward and backward have to agree on the probabilities."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.logprobs import U32, front_rows, tree_logprobs_backward_reference
from tests.test_gpu_logprobs import DT, TRIE, U, inputs, np64

pytestmark = pytest.mark.gpu

LONG = ([-1, 0, 0], [200, 250, 150])


def far_logits(x):
    """Large values in most of the first rows."""
    low = torch.finfo(x.dtype).min
    for i, fill in enumerate((-1e9, -1e10, -1e30, low, 1e9, 1e30, -5e6, 5e6)):
        x[i] = fill
    x[8, ::2], x[8, 1::2] = -1e9, -1.5e9
    x[9] *= 1e9
    x[10, 77] = 1e10
    x[11, 77:90] = 1e30
    x[12] -= 4e4
    x[13] -= 1e5
    x[14] = x[14] * 40 - 1e8
    x[15] += 3e6
    x[16] = float("-inf")
    x[17] = low
    x[17, 5:9] = low / 2
    return x


def bound(parents, lens, x, tok, dlogp, dent, temperature, u):
    """The oracle's gradient, and what fp32 may be off if the probabilities are
    taken relative to the row's largest logit: a difference, 1 / T, log2 e, ln 2
    (8 half units of log p), the sum, and the products.  p below the smallest
    normal number, 2^-126 (where |log p| is 87.4), is 0 by the exponential."""
    want, _ = tree_logprobs_backward_reference(parents, lens, x, tok, dlogp, dent, temperature, u)
    n, v = x.shape
    front, sums = front_rows(parents, lens), U32 * (v / 64 + 160 + 8 * (np.log(v) + 2))
    tol = np.zeros((n, v))
    for i in range(n):
        z = x[i] / temperature
        if z.max() == -np.inf:
            continue
        lp = z - z.max()
        lp = lp - np.log(np.exp(lp).sum())
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0)
        h = -(p * lp).sum()
        g = [(int(tok[t]), abs(float(dlogp[t]))) for t in np.nonzero(front == i)[0] if 0 <= tok[t] < v]
        size, dh = sum(y for _, y in g), 0.0 if dent is None else abs(float(dent[i]))
        e = 8 * U32 * (np.abs(lp) + np.log(v) + 4) + sums
        tol[i] = p * (size + dh * (np.abs(lp) + h)) * (e + (8 + len(g)) * U32) + p * dh * (e + sums * (2 + np.log(v)))
        tol[i] += 2.0 ** -126 * (size + dh * (88 + h))
        for t, y in g:
            tol[i, t] += 4 * U32 * size
    return want, tol / temperature + u * np.abs(want) + 2.0 ** -130


def compare(parents, lens, x, tok, dlogp, dent, temperature):
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_logprobs(x, tok, plan, temperature=temperature)
    d = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy if dent is not None else None, dlogp, plan, dentropy=dent,
                                   temperature=temperature)
    torch.cuda.synchronize()
    want, tol = bound(parents, lens, np64(x), tok.cpu().numpy(), np64(dlogp), None if dent is None else np64(dent),
                      temperature, U[x.dtype])
    err = np.abs(np64(d) - want)
    worst = float((err / tol).max())
    print(f"  worst error {float(err.max()):.3e}, {worst:.3f} of its bound, row {int((err / tol).max(1).argmax())}",
          file=sys.stderr, flush=True)
    assert np.all(err <= tol), f"row {int((err / tol).max(1).argmax())}: {worst} times its bound"
    return plan, r, d


@pytest.mark.parametrize("vocab", [6007, 20008])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.3, 1.0, 2.0])
def test_gradient_of_far_rows(temperature, dtype, vocab):
    """With and without gradients of the entropy, rows whole and in slices, and
    written over the logits."""
    for trie in (TRIE, LONG):
        print(f"gradient of far rows T={temperature} {dtype} {sum(trie[1])} x {vocab}", file=sys.stderr, flush=True)
        x, tok, dlogp, dent = inputs(sum(trie[1]), vocab, DT[dtype], seed=16)
        x = far_logits(x)
        compare(*trie, x, tok, dlogp, None, temperature)
        plan, r, d = compare(*trie, x, tok, dlogp, dent, temperature)
        over = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent,
                                          temperature=temperature, out=x)
        assert over is x and torch.equal(x, d)


def test_gradient_of_a_far_row_with_many_children():
    """More children behind it than a work-group keeps in LDS, some alike."""
    parents, lens = [-1] + [0] * 700, [2] + [1] * 700
    x, tok, dlogp, dent = inputs(702, 9001, torch.float32, seed=17)
    x[1] = -1e9
    tok[2:] = tok[2:] % 200 * 45
    compare(parents, lens, x, tok, dlogp, dent, 1.0)


def test_rows_apart_and_unaligned():
    """Odd distances of the rows of the logits and of the gradient."""
    x, tok, dlogp, dent = inputs(22, 5001, torch.bfloat16, seed=18, pad=3)
    x = far_logits(x)
    compare(*TRIE, x, tok, dlogp, dent, 0.7)
