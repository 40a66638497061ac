"""Workloads of the two ends of a language model over a packed prefix trie: the
token table where it begins, and the output weight with its loss where it ends.

  embedding                   scale x a row of the table for every token
  embedding_backward          the table's gradient, equal tokens added up
  linear_logprobs             for every token, its log probability under the
                              logits hidden @ weight.T of the row in front of
                              it on its path; every row's entropy and
                              log-sum-exp; the logits themselves are not kept
  linear_logprobs_backward    the gradients of hidden and weight for given
                              gradients of the log probabilities and entropies

Plain forms are elementary torch operations in fp32.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- tries

def trie(case):
    """(parents, seg_lens): prompts of `seg` tokens with `fan` completions of
    `leaf` tokens; uneven ones differ in length and some fork once more."""
    r = random.Random(case.get("trie_seed", 0))
    parents, lens = [], []
    for _ in range(case["roots"]):
        root = len(parents)
        parents.append(-1)
        lens.append(case["seg"])
        for _ in range(case["fan"]):
            me = len(parents)
            n = case["leaf"] if case["even"] else max(1, int(case["leaf"] * r.uniform(0.2, 1.0)))
            parents.append(root)
            lens.append(n)
            if not case["even"] and r.random() < 0.25:
                parents += [me, me]
                lens += [max(1, n // 4), max(1, n // 3)]
    return parents, lens


def fronts(parents, lens):
    """The packed row in front of every token on its path (-1: none)."""
    off = np.concatenate([[0], np.cumsum(np.asarray(lens, np.int64))])
    front = np.arange(off[-1]) - 1
    for s, p in enumerate(parents):
        front[off[s]] = off[p + 1] - 1 if p >= 0 else -1
    return front


# ------------------------------------------------------------------- cases

def listed():
    return [
        # A handful of tokens looked up at once: the call's own latency.
        {"name": "embedding few", "op": "embedding", "n": 33, "vocab": 32000, "width": 2048, "dtype": "bf16",
         "scale": 1.0, "often": 0.0, "outside": 0.0},
        # An odd width (rows are not aligned), padding among the tokens (no row of the table), a scale of sqrt(width).
        {"name": "embedding odd width", "op": "embedding", "n": 4283, "vocab": 50001, "width": 1001, "dtype": "f32",
         "scale": math.sqrt(1001), "often": 0.0, "outside": 0.1},
        # One prompt with 8 completions, packed: bound by reading and writing the rows.
        {"name": "embedding group", "op": "embedding", "n": 10240, "vocab": 131072, "width": 4096, "dtype": "bf16",
         "scale": 64.0, "often": 0.0, "outside": 0.0},
        # A small update's gradient, of the width and vocabulary of a test model.
        {"name": "embedding backward few", "op": "embedding_backward", "n": 700, "vocab": 1003, "width": 256,
         "dtype": "f32", "scale": 1.0, "often": 0.0, "outside": 0.0},
        # The packed group's gradient: most of a large table has none.
        {"name": "embedding backward group", "op": "embedding_backward", "n": 10240, "vocab": 131072, "width": 4096,
         "dtype": "bf16", "scale": 64.0, "often": 0.0, "outside": 0.0},
        # A batch of prompts in which one token (a turn's separator) is every fifth: a long sum in one row.
        {"name": "embedding backward repeats", "op": "embedding_backward", "n": 65536, "vocab": 32000, "width": 2048,
         "dtype": "bf16", "scale": 1.0, "often": 0.2, "outside": 0.05},
        # A handful of rows scored at once: bound by reading the weight.
        {"name": "linear logprobs few", "op": "linear_logprobs", "roots": 1, "seg": 9, "fan": 4, "leaf": 6,
         "even": True, "vocab": 32000, "width": 2048, "dtype": "bf16", "temperature": 1.0},
        # fp32, an odd vocabulary, a width that is no multiple of a tile, a sampling temperature.
        {"name": "linear logprobs odd", "op": "linear_logprobs", "roots": 1, "seg": 200, "fan": 6, "leaf": 300,
         "even": False, "trie_seed": 5, "vocab": 50001, "width": 1000, "dtype": "f32", "temperature": 1.3},
        # An update's rows over a large vocabulary: one large matrix product with its softmax.
        {"name": "linear logprobs large", "op": "linear_logprobs", "roots": 1, "seg": 2048, "fan": 6, "leaf": 1024,
         "even": True, "vocab": 131072, "width": 4096, "dtype": "bf16", "temperature": 1.0},
        # The gradients of the same kinds: few rows, odd sizes in fp32, an update's rows.
        {"name": "linear logprobs backward few", "op": "linear_logprobs_backward", "roots": 1, "seg": 9, "fan": 4,
         "leaf": 6, "even": True, "vocab": 32000, "width": 2048, "dtype": "bf16", "temperature": 1.0},
        {"name": "linear logprobs backward odd", "op": "linear_logprobs_backward", "roots": 2, "seg": 150, "fan": 8,
         "leaf": 101, "even": False, "trie_seed": 3, "vocab": 20001, "width": 1000, "dtype": "f32",
         "temperature": 0.7},
        {"name": "linear logprobs backward large", "op": "linear_logprobs_backward", "roots": 1, "seg": 2048,
         "fan": 6, "leaf": 1024, "even": True, "vocab": 131072, "width": 2048, "dtype": "bf16", "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("embedding", "embedding_backward", "linear_logprobs", "linear_logprobs_backward"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    vocab = _log(rng, 1000, 131072)
    if op.startswith("embedding"):
        width = _log(rng, 32, 4096)
        if rng.random() < 0.7:
            width = max(8, width // 8 * 8)
        n = _log(rng, 1, min(65536, 65536 * 2048 // width))
        return {"op": op, "n": n, "vocab": vocab, "width": width, "dtype": dtype,
                "scale": rng.choice((1.0, math.sqrt(width))), "often": rng.choice((0.0, 0.0, 0.2, 0.6)),
                "outside": rng.choice((0.0, 0.0, 0.1))}
    width = 8 * _log(rng, 16, 512)
    # At most the large case's products, an eighth of them in fp32.
    room = 8192 * 131072 * 2048 // (1 if dtype == "bf16" else 8)
    n = _log(rng, 4, max(5, min(8192, int(room / vocab / width / 1.3))))
    c = {"op": op, "roots": rng.choice((1, 1, 2, 4)), "fan": rng.randint(2, 12), "even": False,
         "trie_seed": rng.randrange(1 << 20), "vocab": vocab, "width": width, "dtype": dtype,
         "temperature": rng.choice((1.0, 1.0, 0.7, 1.5))}
    share = rng.uniform(0.1, 0.6)
    c["seg"] = max(1, int(share * n / c["roots"]))
    c["leaf"] = max(1, int((1 - share) * n / c["roots"] / c["fan"]))
    return c


# ------------------------------------------------------------------- state

def prepare(case, seed):
    dev = "cuda:0" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dtype, vocab, width = DTYPES[case["dtype"]], case["vocab"], case["width"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    st = {"op": case["op"], "vocab": vocab}
    if case["op"].startswith("embedding"):
        n = case["n"]
        # Token frequencies fall as 1 / rank; one token more often than that, and some outside the table.
        tok = (torch.exp(rand(n).double() * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)
        tok[rand(n) < case["often"]] = vocab // 3
        tok[rand(n) < case["outside"]] = -1
        st["tokens"], st["scale"] = tok, case["scale"]
        if case["op"] == "embedding":
            st["table"] = randn(vocab, width).to(dtype)
        else:
            st["dout"] = randn(n, width).to(dtype)
    else:
        parents, lens = trie(case)
        n = int(sum(lens))
        # Logits of a spread of 2, with one token of each row raised by 4 to 8.
        w = torch.empty((vocab, width), dtype=dtype, device=dev)
        for i in range(0, vocab, 16384):
            m = min(16384, vocab - i)
            w[i:i + m] = (randn(m, width) * (2.0 / math.sqrt(width))).to(dtype)
        hot = torch.randint(0, vocab, (n,), generator=g, device=dev)
        st["hidden"] = (randn(n, width) + w[hot].float() * (1.0 + rand(n, 1))).to(dtype)
        st["weight"] = w
        front = fronts(parents, lens)
        st["front"] = torch.as_tensor(front, device=dev)
        rare = torch.randint(0, vocab, (n,), generator=g, device=dev)
        st["tokens"] = torch.where(rand(n) < 0.7, hot[st["front"].clamp_min(0)], rare)
        st["temperature"] = case["temperature"]
        if case["op"] == "linear_logprobs_backward":
            st["dlogp"], st["dentropy"] = randn(n), randn(n) * 0.01
            r = plain_linear_logprobs(st)  # what the forward left
            st["lse"], st["entropy"] = r["lse"], r["entropy"]
    if own:
        import prefix_tree_packed_plan_amd as ptp
        st["ptp"] = ptp
        if not case["op"].startswith("embedding"):
            st["plan"] = ptp.tree_plan(parents, lens, 4)
    return st


# ------------------------------------------------------------- plain forms

def plain_embedding(st):
    tok = st["tokens"]
    x = st["table"][tok.clamp_min(0)].float() * st["scale"]
    return torch.where(tok[:, None] >= 0, x, torch.zeros_like(x)).to(st["table"].dtype)


def plain_embedding_backward(st):
    tok, dout = st["tokens"], st["dout"]
    x = dout.float() * st["scale"]
    x = torch.where(tok[:, None] >= 0, x, torch.zeros_like(x))
    d = torch.zeros((st["vocab"], dout.shape[1]), dtype=torch.float32, device=dout.device)
    return d.index_add_(0, tok.clamp_min(0), x).to(dout.dtype)


def _logits(st):
    return torch.matmul(st["hidden"].float(), st["weight"].float().t()).mul_(1.0 / st["temperature"])


def plain_linear_logprobs(st):
    z = _logits(st)
    m = z.amax(-1, keepdim=True)
    y = z.sub_(m)
    e = y.exp()
    s = e.sum(-1, keepdim=True)
    log_s = s.log()
    entropy = (log_s - e.mul_(y).sum(-1, keepdim=True) / s)[:, 0]
    front, tok = st["front"], st["tokens"]
    at = front.clamp_min(0)
    logp = y[at, tok] - log_s[at, 0]
    return {"logp": torch.where(front >= 0, logp, torch.zeros_like(logp)), "entropy": entropy,
            "lse": (m + log_s)[:, 0]}


def plain_linear_logprobs_backward(st):
    logp = _logits(st).sub_(st["lse"][:, None])
    p = logp.exp()
    front, tok = st["front"], st["tokens"]
    g = torch.where(front >= 0, st["dlogp"], torch.zeros_like(st["dlogp"]))
    at = front.clamp_min(0)
    total = torch.zeros_like(g).index_add_(0, at, g)
    d = logp.add_(st["entropy"][:, None]).mul_(st["dentropy"][:, None]).add_(total[:, None]).mul_(p).neg_()
    d.index_put_((at, tok), g, accumulate=True)
    d.mul_(1.0 / st["temperature"])
    dh = torch.matmul(d, st["weight"].float())
    dw = torch.matmul(d.t(), st["hidden"].float())
    return {"dhidden": dh.to(st["hidden"].dtype), "dweight": dw.to(st["weight"].dtype)}


# --------------------------------------------------------------------- run

def run(st):
    op = st["op"]
    if own:
        ptp = st["ptp"]
        if op == "embedding":
            return ptp.tree_embedding(st["tokens"], st["table"], scale=st["scale"])
        if op == "embedding_backward":
            return ptp.tree_embedding_backward(st["tokens"], st["dout"], st["vocab"], scale=st["scale"])
        if op == "linear_logprobs":
            r = ptp.tree_linear_logprobs(st["hidden"], st["weight"], st["tokens"], st["plan"],
                                         temperature=st["temperature"])
            return {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
        dh, dw = ptp.tree_linear_logprobs_backward(st["hidden"], st["weight"], st["tokens"], st["lse"], st["entropy"],
                                                   st["dlogp"], st["plan"], dentropy=st["dentropy"],
                                                   temperature=st["temperature"])
        return {"dhidden": dh, "dweight": dw}
    if op == "embedding":
        return plain_embedding(st)
    if op == "embedding_backward":
        return plain_embedding_backward(st)
    if op == "linear_logprobs":
        return plain_linear_logprobs(st)
    return plain_linear_logprobs_backward(st)


def work(case):
    size, vocab, width = 4 if case["dtype"] == "f32" else 2, case["vocab"], case["width"]
    if case["op"] == "embedding":
        # Distinct rows read: at most one a token; of tokens falling as 1 / rank about this many.
        n = case["n"]
        each = n * (1 - case["often"]) * (1 - case["outside"]) / math.log(vocab)
        distinct = each * math.log(1 + vocab / each) + each * (1 - math.exp(-vocab / each)) if each > 0 else 1
        return {"bytes": int((min(n, distinct) + n) * width * size + 8 * n), "flops": n * width}
    if case["op"] == "embedding_backward":  # dout read, the whole table's gradient written
        n = case["n"]
        return {"bytes": int(n * (1 - case["outside"]) + vocab) * width * size + 8 * n, "flops": n * width}
    n = int(sum(trie(case)[1]))
    if case["op"] == "linear_logprobs":
        return {"bytes": (n + vocab) * width * size + n * (8 + 12), "flops": 2 * n * vocab * width + 6 * n * vocab}
    # hidden and weight read, their gradients written; the logits again, and two products
    return {"bytes": 2 * (n + vocab) * width * size + n * (8 + 16), "flops": 6 * n * vocab * width + 8 * n * vocab}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """From the definition, in 64 bits: every table row's tokens; every block of
    rows of logits."""
    st = prepare(case, seed)
    dd = torch.float64
    tok = st["tokens"]
    if case["op"] == "embedding":
        rows = st["table"].to(dd)[tok.clamp_min(0)]
        return rows * (case["scale"] * (tok >= 0).to(dd))[:, None]
    if case["op"] == "embedding_backward":
        dout = st["dout"]
        d = torch.zeros((case["vocab"], case["width"]), dtype=dd, device=dout.device)
        order = torch.argsort(tok, stable=True)
        order = order[tok[order] >= 0]
        for i in range(0, len(order), 8192):
            at = order[i:i + 8192]
            d.index_add_(0, tok[at], dout[at].to(dd))
        return d * case["scale"]
    h, w = st["hidden"], st["weight"]
    n, vocab = h.shape[0], w.shape[0]
    front, temp, dev = st["front"], case["temperature"], h.device
    w64, h64 = w.to(dd), h.to(dd)
    succ = torch.nonzero(front >= 0)[:, 0]
    step = max(1, (1 << 27) // vocab)
    back = case["op"] == "linear_logprobs_backward"
    out = {x: torch.zeros(n, dtype=dd, device=dev) for x in ("logp", "entropy", "lse")}
    if back:
        dh, dw = torch.zeros_like(h64), torch.zeros_like(w64)
    for i in range(0, n, step):
        z = (h64[i:i + step] @ w64.t()) / temp
        ls = torch.log_softmax(z, -1)
        p = ls.exp()
        ent = -(p * ls).sum(-1)
        mine = succ[(front[succ] >= i) & (front[succ] < i + step)]
        if not back:
            out["lse"][i:i + step] = torch.logsumexp(z, -1)
            out["entropy"][i:i + step] = ent
            out["logp"][mine] = ls[front[mine] - i, tok[mine]]
            continue
        gr = st["dlogp"][mine].to(dd)
        d = -st["dentropy"][i:i + step, None].to(dd) * p * (ls + ent[:, None])
        d -= p * torch.zeros(len(p), dtype=dd, device=dev).index_add_(0, front[mine] - i, gr)[:, None]
        d.index_put_((front[mine] - i, tok[mine]), gr, accumulate=True)
        d /= temp
        dh[i:i + step] = d @ w64
        dw += d.t() @ h64[i:i + step]
    return {"dhidden": dh, "dweight": dw} if back else out
