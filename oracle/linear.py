"""Log probabilities of a trie's tokens from hidden states and an output weight,
and the gradients of both, in fp64; with bounds for products and sums in fp32 and
a stored rounding u (2^-8 in bf16, 2^-24 in fp32), of the results and of the
logits' gradient as the operand of two products."""
from __future__ import annotations

import numpy as np

from .logprobs import U32, _row, front_rows, tree_logprobs_backward_reference, tree_logprobs_reference


def _logits(hidden, weight, terms):
    """The logits, and what fp32 arithmetic may be off: each of C terms is a sum of
    `terms` partial products."""
    hidden, weight = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    z = hidden @ weight.T
    return z, (terms * hidden.shape[1] + 4) * U32 * (np.abs(hidden) @ np.abs(weight).T)


def tree_linear_logprobs_reference(parents, lens, hidden, weight, tokens, temperature=1.0, terms=1):
    """{name: (value, bound)}: logp [N], entropy, lse [N]."""
    z, ez = _logits(hidden, weight, terms)
    ez = ez / temperature
    r = tree_logprobs_reference(parents, lens, z, tokens, temperature)
    front, v = front_rows(parents, lens), z.shape[1]
    n = len(z)
    worst = ez.max(1)
    wide = np.zeros(n)  # of the entropy: sum p |log p + H| dz
    for i in range(n):
        lp, _, h = _row(z[i], temperature)
        p = np.exp(lp)
        wide[i] = (p * np.abs(np.where(p > 0, lp, 0) + h) * ez[i]).sum() * 1.1
    tol = {"lse": r["lse"][1] + worst, "entropy": r["entropy"][1] + wide, "logp": r["logp"][1].copy()}
    for t in range(n):
        if front[t] >= 0 and 0 <= tokens[t] < v:
            tol["logp"][t] += worst[front[t]] + ez[front[t], tokens[t]]
    return {x: (r[x][0], tol[x]) for x in tol}


def tree_linear_logprobs_backward_reference(parents, lens, hidden, weight, tokens, dlogp, dentropy, temperature=1.0,
                                            u=2.0 ** -8, terms=1):
    """{name: (value, bound, rms)} of dhidden and dweight; rms: the root mean square
    error of roundings to u that are independent of each other (one of relative
    size u at most is u / sqrt(3) at most in the mean)."""
    hidden, weight = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    z, ez = _logits(hidden, weight, terms)
    ez = ez / temperature
    d, tol = tree_logprobs_backward_reference(parents, lens, z, tokens, dlogp, dentropy, temperature, u)
    front, v = front_rows(parents, lens), z.shape[1]
    # An error of z, and with it of the row's lse and entropy, moves p and log p.
    for i in range(len(z)):
        lp, lse, h = _row(z[i], temperature)
        if lse == -np.inf:
            continue
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0)
        g = sum(abs(float(dlogp[t])) for t in np.nonzero(front == i)[0] if 0 <= tokens[t] < v)
        dh = 0.0 if dentropy is None else abs(float(dentropy[i]))
        e = ez[i] + ez[i].max()
        tol[i] += 1.1 * p * (g * e + dh * ((np.abs(lp) + h + 1) * e + (p * np.abs(lp + h) * ez[i]).sum())) / temperature
    out = {}
    r2 = u * u / 3
    for name, a, b in (("dhidden", d, weight), ("dweight", d.T, hidden)):
        x = a @ b
        ta = tol if name == "dhidden" else tol.T
        sums = (terms * a.shape[1] + 16) * U32 * (np.abs(a) @ np.abs(b))
        out[name] = (x, ta @ np.abs(b) + sums + u * np.abs(x) + 2.0 ** -126,
                     np.sqrt(r2 * ((a * a) @ (b * b) + x * x)) + 2.0 ** -126)
    return out
