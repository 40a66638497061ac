"""Workloads of the policy-training operators over a packed prefix trie.

Four operators, two for each end of a policy update on a trie of rollouts:

  attention            o and log-sum-exp of softmax attention in which a token
                       sees its own root-to-token path, and nothing else
  attention_backward   dq, dk, dv of it
  logprobs             for every token, its log probability under the logits
                       of the token in front of it on its path; for every row
                       of logits the entropy, the log-sum-exp and the top
                       alternatives
  logprobs_backward    the gradient of the logits for given gradients of the
                       log probabilities and the entropies

Plain forms are elementary torch operations in fp32.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NEG = float("-inf")


# ------------------------------------------------------------------- tries

def trie(case):
    """(parents, seg_lens) of a case, segments in depth-first pre-order."""
    kind, r = case["trie"], random.Random(case.get("trie_seed", 0))
    parents, lens = [], []

    def add(parent, n):
        parents.append(parent)
        lens.append(n)
        return len(parents) - 1

    if kind == "tiny":  # root 64 -> 2 x 32 -> 2 x 16 each
        return [-1, 0, 1, 1, 0, 4, 4], [64, 32, 16, 16, 32, 16, 16]
    if kind == "chains":  # independent samples of about `seg` tokens
        for _ in range(case["roots"]):
            add(-1, max(1, int(case["seg"] * r.uniform(0.75, 1.25))) if case["roots"] > 1 else case["seg"])
    elif kind == "group":  # prompts of `seg` tokens with `fan` completions of `leaf`, some of which fork once more
        for _ in range(case["roots"]):
            root = add(-1, case["seg"])
            for _ in range(case["fan"]):
                n = case["leaf"] if case["even"] else max(1, int(case["leaf"] * r.uniform(0.2, 1.0)))
                c = add(root, n)
                if not case["even"] and r.random() < 0.25:
                    add(c, max(1, n // 4))
                    add(c, max(1, n // 3))
    elif kind == "turns":  # agent sessions: short turns, branching at random, `segs` segments
        def grow(parent, left):
            me = add(parent, max(1, int(case["seg"] * r.uniform(0.05, 1.0))))
            left -= 1
            k = r.choice((1, 1, 2, 3))
            for i in range(k):
                if left <= 0:
                    break
                part = left if i == k - 1 else max(1, int(left * r.uniform(0.2, 0.8)))
                left -= part
                grow(me, part)

        for i in range(case["roots"]):
            grow(-1, max(1, case["segs"] // case["roots"]))
    return parents, lens


def offsets(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, np.int64))])


def before(parents, lens):
    """Tokens in front of each segment on its path."""
    b = []
    for p, _ in zip(parents, lens):
        b.append(0 if p < 0 else b[p] + lens[p])
    return b


def pairs(parents, lens):
    """Visible (query, key) pairs."""
    return sum(n * b + n * (n + 1) // 2 for n, b in zip(lens, before(parents, lens)))


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One short trie of the unit-test size: the call's own latency.
        {"name": "attention tiny", "op": "attention", "trie": "tiny", "hq": 1, "hkv": 1, "d": 32, "dtype": "f32",
         "fused": False},
        # One prompt with 8 sampled completions, q, k, v cut from one projection: a group-sampled update.
        {"name": "attention group", "op": "attention", "trie": "group", "roots": 1, "seg": 2048, "fan": 8, "leaf": 1024,
         "even": True, "hq": 16, "hkv": 4, "d": 128, "dtype": "bf16", "fused": True},
        # One long sample without any branch: the most work a token can have.
        {"name": "attention long chain", "op": "attention", "trie": "chains", "roots": 1, "seg": 16383, "hq": 8,
         "hkv": 2, "d": 128, "dtype": "bf16", "fused": False},
        # Agent sessions of many short turns: ragged segments, deep paths, smaller heads.
        {"name": "attention turns", "op": "attention", "trie": "turns", "roots": 2, "segs": 220, "seg": 120,
         "trie_seed": 7, "hq": 12, "hkv": 4, "d": 64, "dtype": "bf16", "fused": False},
        # The gradients on the same kinds of trie: the unit-test size, the sampled group, the long sample.
        {"name": "attention backward tiny", "op": "attention_backward", "trie": "tiny", "hq": 2, "hkv": 1, "d": 64,
         "dtype": "f32", "fused": False},
        {"name": "attention backward group", "op": "attention_backward", "trie": "group", "roots": 1, "seg": 2048,
         "fan": 8, "leaf": 1024, "even": True, "hq": 16, "hkv": 4, "d": 128, "dtype": "bf16", "fused": True},
        {"name": "attention backward chain", "op": "attention_backward", "trie": "chains", "roots": 1, "seg": 16383,
         "hq": 8, "hkv": 2, "d": 128, "dtype": "bf16", "fused": False},
        # A handful of tokens scored at once, with the alternatives a sampler shows.
        {"name": "logprobs few", "op": "logprobs", "trie": "group", "roots": 1, "seg": 9, "fan": 4, "leaf": 6,
         "even": True, "vocab": 32000, "dtype": "f32", "temperature": 1.0, "top_k": 8},
        # An odd vocabulary (rows of logits are not aligned), top alternatives, a sampling temperature.
        {"name": "logprobs odd vocabulary", "op": "logprobs", "trie": "group", "roots": 2, "seg": 300, "fan": 8,
         "leaf": 301, "even": False, "trie_seed": 3, "vocab": 50001, "dtype": "bf16", "temperature": 0.7, "top_k": 5},
        # A chunk of an update's logits over a large vocabulary: bound by reading the logits once.
        {"name": "logprobs large", "op": "logprobs", "trie": "group", "roots": 1, "seg": 2048, "fan": 6, "leaf": 1024,
         "even": True, "vocab": 131072, "dtype": "bf16", "temperature": 1.0, "top_k": 0},
        # The gradients: an odd vocabulary in fp32, and the chunk above.
        {"name": "logprobs backward odd", "op": "logprobs_backward", "trie": "group", "roots": 1, "seg": 200, "fan": 6,
         "leaf": 300, "even": False, "trie_seed": 5, "vocab": 50001, "dtype": "f32", "temperature": 1.3},
        {"name": "logprobs backward large", "op": "logprobs_backward", "trie": "group", "roots": 1, "seg": 2048,
         "fan": 6, "leaf": 1024, "even": True, "vocab": 131072, "dtype": "bf16", "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_trie(rng, tokens):
    kind = rng.choice(("chains", "group", "turns"))
    c = {"trie": kind, "trie_seed": rng.randrange(1 << 20)}
    if kind == "chains":
        c["roots"] = rng.choice((1, 1, 2, 3, 5))
        c["seg"] = max(1, int(tokens / c["roots"] / 1.25))
    elif kind == "group":
        c["roots"], c["fan"], c["even"] = rng.choice((1, 1, 2, 4)), rng.randint(2, 12), False
        share = rng.uniform(0.1, 0.6)
        c["seg"] = max(1, int(share * tokens / c["roots"]))
        c["leaf"] = max(1, int((1 - share) * tokens / c["roots"] / c["fan"]))
    else:
        c["roots"] = rng.choice((1, 2, 3))
        c["seg"] = min(max(2, tokens // 8), _log(rng, 8, 512))
        c["segs"] = max(c["roots"], min(400, int(tokens / (0.55 * c["seg"]))))
    return c


def draw(rng):
    op = rng.choice(("attention", "attention_backward", "logprobs", "logprobs_backward"))
    if op.startswith("attention"):
        hkv, group, d = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 8)), rng.choice((32, 64, 128))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        # At most the long chain's score matrices (8 heads of 16383 tokens), a quarter of that in fp32.
        room = 8 * 16383 ** 2 / (1 if dtype == "bf16" else 4)
        most = int(math.sqrt(room / (hkv * group)) / 1.3)
        tokens = _log(rng, 40, min(16383, most))
        return {"op": op, **_draw_trie(rng, tokens), "hq": hkv * group, "hkv": hkv, "d": d, "dtype": dtype,
                "fused": rng.random() < 0.4}
    vocab = _log(rng, 1000, 131072)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    tokens = _log(rng, 4, min(8192, int(8192 * 131072 / vocab / (1 if dtype == "bf16" else 2) / 1.3)))
    c = {"op": op, **_draw_trie(rng, max(tokens, 4)), "vocab": vocab, "dtype": dtype,
         "temperature": rng.choice((1.0, 1.0, 0.7, 1.5))}
    if op == "logprobs":
        c["top_k"] = rng.choice((0, 0, 1, 5, 8, 20, 32))
    return c


# ------------------------------------------------------------------- state

def _seg_tables(parents, lens):
    """Host tables: the segment of each token, each segment's ancestors or
    itself [n_seg, n_seg], and the token in front of each token on its path
    (-1: none)."""
    n = len(parents)
    seg = np.repeat(np.arange(n), lens)
    anc = np.zeros((n, n), bool)
    for s, p in enumerate(parents):
        if p >= 0:
            anc[s] = anc[p]
        anc[s, s] = True
    off = offsets(lens)
    prev = np.arange(off[-1]) - 1
    for s, p in enumerate(parents):
        prev[off[s]] = off[p + 1] - 1 if p >= 0 else -1
    return seg, anc, prev


def prepare(case, seed):
    dev = "cuda:0" if torch.cuda.is_available() else "cpu"
    parents, lens = trie(case)
    n = int(sum(lens))
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    st = {"op": case["op"], "n": n}
    seg, anc, prev = _seg_tables(parents, lens)
    if case["op"].startswith("attention"):
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        st["scale"] = d ** -0.5
        if case["fused"]:
            # One projection's output; q, k, v are views of it.
            qkv = randn(n, hq + 2 * hkv, d).to(dtype)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            st["q"], st["k"], st["v"] = (randn(n, h, d).to(dtype) for h in (hq, hkv, hkv))
        st["seg"] = torch.as_tensor(seg, device=dev)
        st["anc"] = torch.as_tensor(anc, device=dev)
        if case["op"] == "attention_backward":
            st["do"] = randn(n, hq, d).to(dtype)
            st["o"], st["lse"] = plain_attention(st)  # what the forward left
    else:
        v = case["vocab"]
        # Logits of a language model: a wide spread with a few likely tokens.
        x = torch.empty((n, v), dtype=dtype, device=dev)
        hot = torch.randint(0, v, (n, 4), generator=g, device=dev)
        step = max(1, (1 << 28) // v)
        for i in range(0, n, step):
            y = randn(min(step, n - i), v) * 2.0
            y.scatter_add_(1, hot[i:i + step], 6.0 + 2.0 * torch.rand((y.shape[0], 4), generator=g, device=dev))
            x[i:i + step] = y.to(dtype)
        st["logits"] = x
        # Sampled tokens: mostly likely ones of the row in front.
        front = torch.as_tensor(np.maximum(prev, 0), device=dev)
        pick = hot[front, torch.randint(0, 4, (n,), generator=g, device=dev)]
        rare = torch.randint(0, v, (n,), generator=g, device=dev)
        st["tokens"] = torch.where(torch.rand(n, generator=g, device=dev) < 0.7, pick, rare)
        st["prev"] = torch.as_tensor(prev, device=dev)
        st["inv_t"] = 1.0 / case["temperature"]
        st["temperature"] = case["temperature"]
        st["top_k"] = case.get("top_k", 0)
        if case["op"] == "logprobs_backward":
            st["dlogp"] = randn(n)
            st["dentropy"] = randn(n) * 0.01
            r = plain_logprobs(dict(st, top_k=0))
            st["lse"], st["entropy"] = r["lse"], r["entropy"]
    if own:
        import prefix_tree_packed_plan_amd as ptp
        st["ptp"] = ptp
        st["plan"] = ptp.tree_plan(parents, lens, 4)
    return st


# ------------------------------------------------------------- plain forms

def _by_group(x, hkv):
    """[N, hq, d] -> [hkv, group, N, d] fp32, contiguous."""
    n, hq, d = x.shape
    return x.float().reshape(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).contiguous()


def _visible(st):
    """[N, N]: key j (column) on the path of query i (row), up to i itself."""
    seg, n = st["seg"], st["n"]
    at = torch.arange(n, device=seg.device)
    return st["anc"][seg[:, None], seg[None, :]] & (at[None, :] <= at[:, None])


def _scores(st, q, k):
    """Scaled scores [hkv, group, N, N], -inf where not visible."""
    hkv, group, n, d = q.shape
    s = torch.matmul(q.reshape(hkv, group * n, d), k.transpose(1, 2).contiguous()).reshape(hkv, group, n, n)
    return s.mul_(st["scale"]).masked_fill_(~_visible(st), NEG)


def plain_attention(st):
    hkv = st["k"].shape[1]
    q, k, v = _by_group(st["q"], hkv), _by_group(st["k"], hkv)[:, 0], _by_group(st["v"], hkv)[:, 0]
    group, n, d = q.shape[1:]
    s = _scores(st, q, k)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(hkv, group * n, n), v).reshape(hkv, group, n, d) / z
    lse = (m + z.log())[..., 0]
    o = o.permute(2, 0, 1, 3).reshape(n, hkv * group, d).to(st["q"].dtype)
    return o, lse.permute(2, 0, 1).reshape(n, hkv * group).contiguous()


def plain_attention_backward(st):
    dtype, hkv = st["q"].dtype, st["k"].shape[1]
    q, k, v = _by_group(st["q"], hkv), _by_group(st["k"], hkv)[:, 0], _by_group(st["v"], hkv)[:, 0]
    do, o = _by_group(st["do"], hkv), _by_group(st["o"], hkv)
    group, n, d = q.shape[1:]
    lse = st["lse"].reshape(n, hkv, group).permute(1, 2, 0)[..., None]
    p = _scores(st, q, k).sub_(lse).exp_().reshape(hkv, group * n, n)
    do2, q2 = do.reshape(hkv, group * n, d), q.reshape(hkv, group * n, d)
    dv = torch.matmul(p.transpose(1, 2), do2)
    ds = torch.matmul(do2, v.transpose(1, 2).contiguous())
    ds.sub_((do * o).sum(-1).reshape(hkv, group * n, 1)).mul_(p).mul_(st["scale"])
    dk = torch.matmul(ds.transpose(1, 2), q2)
    dq = torch.matmul(ds, k).reshape(hkv, group, n, d)
    dq = dq.permute(2, 0, 1, 3).reshape(n, hkv * group, d).to(dtype)
    return dq, dk.permute(1, 0, 2).contiguous().to(dtype), dv.permute(1, 0, 2).contiguous().to(dtype)


def plain_logprobs(st):
    x = st["logits"].float() * st["inv_t"]
    m = x.amax(-1, keepdim=True)
    y = x - m
    e = y.exp()
    z = e.sum(-1, keepdim=True)
    log_z = z.log()
    entropy = (log_z - (e * y).sum(-1, keepdim=True) / z)[:, 0]
    lse = (m + log_z)[:, 0]
    prev, tok = st["prev"], st["tokens"]
    front = prev.clamp_min(0)
    logp = y[front, tok] - log_z[front, 0]
    r = {"logp": torch.where(prev >= 0, logp, torch.zeros_like(logp)), "entropy": entropy, "lse": lse}
    if st["top_k"]:
        # Largest first, the lowest index first among equals: one whole
        # number for each value, ordered as the value and then by the index.
        bits = st["logits"].float().view(torch.int32).to(torch.int64)
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 20)
        order -= torch.arange(x.shape[1], device=x.device)
        ids = torch.topk(order, st["top_k"], dim=-1).indices
        r["top_logp"] = y.gather(1, ids) - log_z
        r["top_ids"] = ids.to(torch.int32)
    return r


def plain_logprobs_backward(st):
    x = st["logits"].float() * st["inv_t"]
    logp = x - st["lse"][:, None]
    p = logp.exp()
    prev, g = st["prev"], torch.where(st["prev"] >= 0, st["dlogp"], torch.zeros_like(st["dlogp"]))
    front = prev.clamp_min(0)
    total = torch.zeros_like(g).index_add_(0, front, g)
    d = p * (logp + st["entropy"][:, None])
    d.mul_(-st["dentropy"][:, None])
    d.sub_(p * total[:, None])
    d.index_put_((front, st["tokens"]), g, accumulate=True)
    return d.mul_(st["inv_t"]).to(st["logits"].dtype)


# --------------------------------------------------------------------- run

def run(st):
    op = st["op"]
    if own:
        ptp, plan = st["ptp"], st["plan"]
        if op == "attention":
            o, lse = ptp.tree_attention(st["q"], st["k"], st["v"], plan, return_lse=True)
            return {"o": o, "lse": lse}
        if op == "attention_backward":
            dq, dk, dv = ptp.tree_attention_backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], plan)
            return {"dq": dq, "dk": dk, "dv": dv}
        if op == "logprobs":
            r = ptp.tree_logprobs(st["logits"], st["tokens"], plan, temperature=st["temperature"], top_k=st["top_k"])
            out = {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
            if st["top_k"]:
                out.update(top_logp=r.top_logp, top_ids=r.top_ids)
            return out
        return {"dlogits": ptp.tree_logprobs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"],
                                                      st["dlogp"], plan, dentropy=st["dentropy"],
                                                      temperature=st["temperature"])}
    if op == "attention":
        o, lse = plain_attention(st)
        return {"o": o, "lse": lse}
    if op == "attention_backward":
        dq, dk, dv = plain_attention_backward(st)
        return {"dq": dq, "dk": dk, "dv": dv}
    if op == "logprobs":
        return plain_logprobs(st)
    return {"dlogits": plain_logprobs_backward(st)}


def work(case):
    parents, lens = trie(case)
    n, size = int(sum(lens)), 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("attention"):
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        seen = pairs(parents, lens)
        if case["op"] == "attention":  # q, k, v read; o, lse written; two products
            return {"bytes": n * (2 * hq + 2 * hkv) * d * size + 4 * n * hq, "flops": 4 * d * hq * seen}
        # q, k, v, o, do, lse read; dq, dk, dv written; five products
        return {"bytes": n * (4 * hq + 4 * hkv) * d * size + 4 * n * hq, "flops": 10 * d * hq * seen}
    v, k = case["vocab"], case.get("top_k", 0)
    if case["op"] == "logprobs":
        return {"bytes": n * v * size + n * (8 + 12) + 8 * n * k, "flops": 6 * n * v}
    return {"bytes": 2 * n * v * size + n * (8 + 16), "flops": 8 * n * v}


# ------------------------------------------------------------------- exact

def _paths(parents, lens):
    """Per segment: its rows and the rows of its whole path, root first."""
    off = offsets(lens)
    rows = []
    for s, p in enumerate(parents):
        mine = np.arange(off[s], off[s + 1])
        rows.append(mine if p < 0 else np.concatenate([rows[p], mine]))
    return off, rows


def exact(case, seed):
    """From the definition, in 64 bits: every segment alone against its path's
    keys; every row of logits alone."""
    if case["op"].startswith("attention"):
        parents, lens = trie(case)
        if pairs(parents, lens) * case["hq"] * case["d"] > 2.5e11:
            return None
    st = prepare(case, seed)
    dd = torch.float64
    if case["op"].startswith("attention"):
        off, paths = _paths(parents, lens)
        hq, hkv, d, n = case["hq"], case["hkv"], case["d"], st["n"]
        grp, dev = hq // hkv, st["q"].device
        q, k, v = (st[x].to(dd).transpose(0, 1).contiguous() for x in "qkv")
        o = torch.zeros(hq, n, d, dtype=dd, device=dev)
        lse = torch.zeros(hq, n, dtype=dd, device=dev)
        back = case["op"] == "attention_backward"
        if back:
            do = st["do"].to(dd).transpose(0, 1).contiguous()
            dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for s in range(len(parents)):
            rows = torch.as_tensor(paths[s], device=dev)
            depth = len(rows) - lens[s]
            for lo in range(0, lens[s], 1024):
                hi = min(lens[s], lo + 1024)
                a, b = int(off[s]) + lo, int(off[s]) + hi
                keys = rows[:depth + hi]
                later = torch.arange(len(keys), device=dev)[None, :] > depth + torch.arange(lo, hi, device=dev)[:, None]
                for h in range(hq):
                    kk, vv = k[h // grp, keys], v[h // grp, keys]
                    w = (q[h, a:b] @ kk.t()) / math.sqrt(d)
                    w[later] = NEG
                    lse[h, a:b] = torch.logsumexp(w, -1)
                    w = torch.softmax(w, -1)
                    o[h, a:b] = w @ vv
                    if back:
                        dv[h // grp].index_add_(0, keys, w.t() @ do[h, a:b])
                        dw = do[h, a:b] @ vv.t()
                        dw = w * (dw - (w * dw).sum(-1, keepdim=True)) / math.sqrt(d)
                        dq[h, a:b] = dw @ kk
                        dk[h // grp].index_add_(0, keys, dw.t() @ q[h, a:b])
        if back:
            return {"dq": dq.transpose(0, 1), "dk": dk.transpose(0, 1), "dv": dv.transpose(0, 1)}
        return {"o": o.transpose(0, 1), "lse": lse.t()}
    x, tok, prev = st["logits"], st["tokens"], st["prev"]
    n, vocab = x.shape
    temp = case["temperature"]
    dev = x.device
    succ = torch.nonzero(prev >= 0)[:, 0]
    step = max(1, (1 << 27) // vocab)
    logp = torch.zeros(n, dtype=dd, device=dev)
    if case["op"] == "logprobs":
        entropy, lse = torch.zeros(n, dtype=dd, device=dev), torch.zeros(n, dtype=dd, device=dev)
        top, ids = [], []
        for i in range(0, n, step):
            raw = x[i:i + step].to(dd)
            ls = torch.log_softmax(raw / temp, -1)
            lse[i:i + step] = torch.logsumexp(raw / temp, -1)
            entropy[i:i + step] = -(ls.exp() * ls).sum(-1)
            mine = succ[(prev[succ] >= i) & (prev[succ] < i + step)]
            logp[mine] = ls[prev[mine] - i, tok[mine]]
            if case["top_k"]:
                best = torch.sort(raw, dim=-1, descending=True, stable=True).indices[:, :case["top_k"]]
                ids.append(best.to(torch.int32))
                top.append(ls.gather(1, best))
        r = {"logp": logp, "entropy": entropy, "lse": lse}
        if case["top_k"]:
            r.update(top_logp=torch.cat(top), top_ids=torch.cat(ids))
        return r
    d = torch.zeros((n, vocab), dtype=dd, device=dev)
    for i in range(0, n, step):
        ls = torch.log_softmax(x[i:i + step].to(dd) / temp, -1)
        p = ls.exp()
        h = -(p * ls).sum(-1, keepdim=True)
        part = -st["dentropy"][i:i + step, None].to(dd) * p * (ls + h)
        mine = succ[(prev[succ] >= i) & (prev[succ] < i + step)]
        gr = st["dlogp"][mine].to(dd)
        part -= p * torch.zeros(len(p), dtype=dd, device=dev).index_add_(0, prev[mine] - i, gr)[:, None]
        part.index_put_((prev[mine] - i, tok[mine]), gr, accumulate=True)
        d[i:i + step] = part / temp
    return {"dlogits": d}
