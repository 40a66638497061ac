"""fp32 products as sums of bf16 partial products, and inputs on which the size of
their error tells whether one is left out."""
from __future__ import annotations

import torch

from .logprobs import front_rows

# The six partial products (parts of the first factor, of the second) that are kept.
PRODUCTS = ((0, 0), (0, 1), (1, 0), (0, 2), (2, 0), (1, 1))

# (rows, vocabulary, width): a few rows, sums in splits, several tiles.
SPLIT_CASES = ((64, 700, 136), (40, 9000, 72), (300, 900, 256), (600, 6500, 520))
# An error relative to a gradient's norm.  Sums round by 2^-24 / sqrt(3) of a running sum in
# the mean, in 6 steps or more for 32 terms; over a few hundred steps that is a few
# 1e-7, while a partial product of parts whose exponents differ by 16 is 4e-6 of its terms.
SPLIT_REL = 1e-6
# A log probability's, in the mean: the same of logits of spread 2, and the log-sum-exp's
# rounding, 2^-22 / sqrt(3).
SPLIT_RMS = 1e-6


def split_inputs(n, vocab, width):
    """(parents, lens, hidden, weight, tokens, dlogp), fp32."""
    g = torch.Generator().manual_seed(vocab)
    h = torch.randn((n, width), generator=g)
    w = torch.randn((vocab, width), generator=g) * (2.0 / width ** 0.5)
    a = n // 3
    return ([-1, 0, 0, 1], [a, a, 5, n - 2 * a - 5], h, w, torch.randint(0, vocab, (n,), generator=g),
            torch.randn(n, generator=g))


def split_exact(parents, lens, hidden, weight, tokens, dlogp, products=None):
    """(logp, dhidden, dweight) in fp64; with `products`, matrix products of fp32
    factors by those partial products alone."""
    def product(a, b):
        if products is None:
            return a.double() @ b.double()
        pa, pb = parts(a), parts(b)
        return sum(pa[i].double() @ pb[j].double() for i, j in products)

    front = torch.as_tensor(front_rows(parents, lens), device=hidden.device)
    z = product(hidden, weight.t())
    ls = z.log_softmax(-1)
    t = torch.nonzero(front >= 0)[:, 0]
    logp = torch.zeros(len(front), dtype=torch.float64, device=hidden.device)
    logp[t] = ls[front[t], tokens[t]]
    g = dlogp[t].double()
    d = -ls.exp() * torch.zeros(len(z), dtype=torch.float64, device=z.device).index_add_(0, front[t], g)[:, None]
    d.index_put_((front[t], tokens[t]), g, accumulate=True)
    d = d if products is None else d.float()
    return logp, product(d, weight), product(d.t(), hidden)


def parts(x):
    """Three bf16 (as fp32) whose sum is x: its first 8 bits, the rest rounded, and so on."""
    out = [(x.contiguous().view(torch.int32) & -65536).view(torch.float32)]
    for _ in range(2):
        x = x - out[-1]
        out.append(x.to(torch.bfloat16).float())
    return out
