"""Tree attention and its gradients in fp64, one segment at a time against the
keys of its own root path ("Tree Training" section 3.1 Eq. 6), and for every
value a bound on what arithmetic with given roundings may be off.

tree_attention_reference(parents, lens, q, k, v, scale, do=None, u=..) with
q [N, H_q, d], k, v [N, H_kv, d]; u is the relative rounding of a stored value
(2^-8 in bf16, 2^-24 in fp32): outputs, and the probabilities and their
gradients as operands of a product.  Sums and scores are taken to be in fp32.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def _paths(parents, lens):
    off = np.concatenate([[0], np.cumsum(np.asarray(lens, np.int64))])
    rows = []
    for s, p in enumerate(parents):
        mine = np.arange(off[s], off[s + 1])
        rows.append(mine if p < 0 else np.concatenate([rows[p], mine]))
    return off, rows


def tree_attention_reference(parents, lens, q, k, v, scale, do=None, u=2.0 ** -8):
    """Returns {name: (value, bound)} for o, lse and, given do, dq, dk, dv."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    hkv = k.shape[1]
    off, paths = _paths(parents, lens)
    out = {"o": np.zeros((n, hq, d)), "lse": np.zeros((n, hq))}
    tol = {"o": np.zeros((n, hq, d)), "lse": np.zeros((n, hq))}
    if do is not None:
        do = np.asarray(do, np.float64)
        for x, shape in (("dq", q.shape), ("dk", k.shape), ("dv", v.shape)):
            out[x], tol[x] = np.zeros(shape), np.zeros(shape)
    for s in range(len(parents)):
        rows, a, b = paths[s], int(off[s]), int(off[s + 1])
        see = np.arange(len(rows))[None, :] <= len(rows) - (b - a) + np.arange(b - a)[:, None]
        for h in range(hq):
            g = h // (hq // hkv)
            kk, vv, qq = k[rows, g], v[rows, g], q[a:b, h]
            with np.errstate(over="ignore", invalid="ignore"):
                w = np.where(see, qq @ kk.T * scale, -np.inf)
            m = w.max(1, keepdims=True)
            e = np.exp(w - m)
            z = e.sum(1, keepdims=True)
            p = e / z
            # A score's error: d products summed in fp32, the scale, and the
            # base-2 argument of exp; it is the relative error of exp.
            size = (np.abs(qq) @ np.abs(kk).T) * scale
            es = U32 * ((d + 4) * size + 4 * np.abs(w - m, where=see, out=np.zeros_like(w)) + 4)
            ep = np.where(see, es, 0)  # relative, of exp(w - m)
            cnt = len(rows)
            ez = (p * ep).sum(1, keepdims=True) + cnt * U32
            out["lse"][a:b, h] = (m + np.log(z))[:, 0]
            tol["lse"][a:b, h] = (ez + 4 * U32 * (1 + np.abs(m) + np.abs(np.log(z))) + (d + 4) * U32 * size.max(1, keepdims=True))[:, 0]
            av = np.abs(vv)
            o = p @ vv
            po = p @ av
            out["o"][a:b, h] = o
            tol["o"][a:b, h] = (p * (ep + u)) @ av + (ez + cnt * U32) * po + u * np.abs(o) + 1e-30
            if do is None:
                continue
            dd = do[a:b, h]
            dp = dd @ vv.T
            delta = (dd * o).sum(1, keepdims=True)
            ds = p * (dp - delta)
            # The backward recomputes p from the stored lse, and takes the
            # stored (rounded) o for delta.
            e_rel = ep + tol["lse"][a:b, h][:, None] + 4 * U32 * (1 + np.abs(out["lse"][a:b, h])[:, None])
            e_delta = (np.abs(dd) * tol["o"][a:b, h]).sum(1, keepdims=True) + (d + 4) * U32 * (np.abs(dd) * np.abs(o)).sum(1, keepdims=True)
            e_dp = (d + 4) * U32 * (np.abs(dd) @ av.T)
            e_ds = np.where(see, p * (e_delta + e_dp) + np.abs(ds) * (e_rel + u + 4 * U32), 0)
            out["dq"][a:b, h] = scale * ds @ kk
            tol["dq"][a:b, h] = scale * ((e_ds + cnt * U32 * np.abs(ds)) @ np.abs(kk))
            np.add.at(out["dk"], (rows, g), scale * ds.T @ qq)
            np.add.at(tol["dk"], (rows, g), scale * (e_ds + n * U32 * np.abs(ds)).T @ np.abs(qq))
            np.add.at(out["dv"], (rows, g), p.T @ dd)
            np.add.at(tol["dv"], (rows, g), (p * (e_rel + u + n * U32)).T @ np.abs(dd))
    for x in ("dq", "dk", "dv"):
        if x in out:
            tol[x] += u * np.abs(out[x]) + 1e-30
    return {x: (out[x], tol[x]) for x in out}


def tree_attention_rms(parents, lens, q, k, v, scale, do, u=2.0 ** -8):
    """Returns {name: root mean square error} for o, dq, dk, dv, element by
    element, of arithmetic whose roundings to u are independent of each other:
    one of relative size u at most is u / sqrt(3) at most in the mean.  Far
    tighter than the bounds above, which add every rounding at its worst, and
    so what a lost part of a list or a wrong delta shows against (rms_ratio).

    o: the probabilities as operands, and its own rounding.  delta takes o's
    error, the same for all keys of a row.  dq, dk: delta, ds as operands, their
    own rounding; dv: p as operands, and its own."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    n, hq, d = q.shape
    hkv = k.shape[1]
    off, paths = _paths(parents, lens)
    r2 = u * u / 3
    var = {"o": np.zeros(q.shape), "dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    sums = {"dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for s in range(len(parents)):
        rows, a, b = paths[s], int(off[s]), int(off[s + 1])
        see = np.arange(len(rows))[None, :] <= len(rows) - (b - a) + np.arange(b - a)[:, None]
        for h in range(hq):
            g = h // (hq // hkv)
            kk, vv, qq, dd = k[rows, g], v[rows, g], q[a:b, h], do[a:b, h]
            w = np.where(see, qq @ kk.T * scale, -np.inf)
            p = np.exp(w - w.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ vv
            vo = r2 * ((p * p) @ (vv * vv) + o * o)
            vdelta = (dd * dd * vo).sum(1, keepdims=True)
            ds = p * (dd @ vv.T - (dd * o).sum(1, keepdims=True))
            dq = scale * ds @ kk
            var["o"][a:b, h] = vo
            var["dq"][a:b, h] = scale ** 2 * (r2 * (ds * ds) @ (kk * kk) + vdelta * (p @ kk) ** 2) + r2 * dq * dq
            np.add.at(var["dk"], (rows, g), scale ** 2 * (r2 * ds * ds + vdelta * p * p).T @ (qq * qq))
            np.add.at(var["dv"], (rows, g), r2 * (p * p).T @ (dd * dd))
            np.add.at(sums["dk"], (rows, g), scale * ds.T @ qq)
            np.add.at(sums["dv"], (rows, g), p.T @ dd)
    for x in sums:
        var[x] += r2 * sums[x] ** 2
    return {x: np.sqrt(var[x]) + 1e-30 for x in var}


def rms_ratio(err, rms, rows=64):
    """The largest root mean square of err / rms over `rows` consecutive rows
    (a rest of less than half as many belongs to the ones before) of one head."""
    n, h, d = err.shape
    z = ((err / rms) ** 2).mean(-1)
    cuts = list(range(0, n, rows))
    if len(cuts) > 1 and n - cuts[-1] < rows // 2:
        cuts.pop()
    return float(np.sqrt(max(z[a:b].mean(0).max() for a, b in zip(cuts, cuts[1:] + [n]))))
