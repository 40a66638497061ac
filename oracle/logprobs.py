"""Log probabilities of a trie's tokens under the logits of the row in front of
each on its path, entropies, the largest entries, and the gradient of the
logits, in fp64; with bounds for arithmetic in fp32 on rows of V columns."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def front_rows(parents, lens):
    """The packed row in front of every token on its path (-1: none)."""
    off = np.concatenate([[0], np.cumsum(np.asarray(lens, np.int64))])
    front = np.arange(off[-1]) - 1
    for s, p in enumerate(parents):
        front[off[s]] = off[p + 1] - 1 if p >= 0 else -1
    return front


def _row(x, temperature):
    """log p, lse, entropy of one row; a row of -inf has log p = lse = -inf and
    entropy 0."""
    z = np.asarray(x, np.float64) / temperature
    m = z.max()
    if m == -np.inf:
        return np.full_like(z, -np.inf), -np.inf, 0.0
    log_s = np.log(np.exp(z - m).sum())
    lp = z - m - log_s
    p = np.exp(lp)
    return lp, m + log_s, -(p * np.where(p > 0, lp, 0)).sum()


def tree_logprobs_reference(parents, lens, logits, tokens, temperature=1.0, top_k=0):
    """{name: (value, bound)}: logp [N], entropy, lse [N], top_logp, top_ids
    (its bound 0) [N, top_k]."""
    logits = np.asarray(logits, np.float64)
    n, v = logits.shape
    front = front_rows(parents, lens)
    r = {"logp": np.zeros(n), "entropy": np.zeros(n), "lse": np.zeros(n), "top_logp": np.zeros((n, top_k)),
         "top_ids": np.zeros((n, top_k), np.int64)}
    # The sums: a lane adds v / 256 values or more, then 8 + 64 partial sums
    # are joined; each term's exponential is off by a few roundings of its
    # argument, whose weighted size is below log v + 2.
    sums = U32 * (v / 256 + 160 + 8 * (np.log(v) + 2))
    lps = []
    for i in range(n):
        lp, r["lse"][i], r["entropy"][i] = _row(logits[i], temperature)
        lps.append(lp)
        order = np.argsort(-logits[i], kind="stable")[:top_k]
        r["top_ids"][i] = order
        r["top_logp"][i] = lp[order]
    for t in range(n):
        if front[t] >= 0 and 0 <= tokens[t] < v:
            r["logp"][t] = lps[front[t]][tokens[t]]
    fin = lambda x: np.where(np.isfinite(x), np.abs(x), 0)  # noqa: E731
    tol = {"lse": sums + 4 * U32 * fin(r["lse"]), "entropy": sums * (2 + np.log(v)) + 4 * U32 * np.abs(r["entropy"]),
           "logp": sums + 4 * U32 * (fin(r["logp"]) + np.log(v)), "top_ids": 0,
           "top_logp": sums + 4 * U32 * (fin(r["top_logp"]) + np.log(v))}
    return {x: (r[x], tol[x]) for x in r}


def tree_logprobs_backward_reference(parents, lens, logits, tokens, dlogp, dentropy, temperature=1.0, u=2.0 ** -8):
    """(dlogits, bound), u the relative rounding of a stored gradient."""
    logits = np.asarray(logits, np.float64)
    n, v = logits.shape
    front = front_rows(parents, lens)
    d, tol = np.zeros((n, v)), np.zeros((n, v))
    sums = U32 * (v / 256 + 160 + 8 * (np.log(v) + 2))
    for i in range(n):
        lp, lse, h = _row(logits[i], temperature)
        if lse == -np.inf:
            continue
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0)
        g = [(int(tokens[t]), float(dlogp[t])) for t in np.nonzero(front == i)[0] if 0 <= tokens[t] < v]
        total, size = sum(x for _, x in g), sum(abs(x) for _, x in g)
        dh = 0.0 if dentropy is None else float(dentropy[i])
        d[i] = -p * total - dh * p * (lp + h)
        # p from the stored lse: the error of log p is its relative error.
        e_lp = 4 * U32 * (np.where(p > 0, np.abs(logits[i]), 0) / temperature + abs(lse) + np.abs(lp) + 4) + sums
        tol[i] = p * (size + abs(dh) * (np.abs(lp) + h)) * (e_lp + (8 + len(g)) * U32) \
            + p * abs(dh) * (e_lp + sums * (2 + np.log(v)))
        for tok, x in g:
            d[i, tok] += x
            tol[i, tok] += 4 * U32 * size
    return d / temperature, tol / temperature + u * np.abs(d) / temperature + 2.0 ** -130
