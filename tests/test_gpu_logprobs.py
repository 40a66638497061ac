"""Token log probabilities on the GPU, forward and backward, against the fp64
oracle (oracle/logprobs.py) with its own error bounds: odd vocabularies and
row distances, temperatures, top alternatives with ties, masked vocabularies,
tokens outside of it, many children behind one row, parts of a trie, in-place
gradients, graphs."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.logprobs import tree_logprobs_backward_reference, tree_logprobs_reference
from prefix_tree_packed_plan_amd import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TRIE = ([-1, 0, 0, 2, 2, 2, -1], [5, 3, 1, 2, 1, 4, 6])


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(n, vocab, dtype, seed=1, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, vocab + pad), generator=g) * spread).to(dtype).to(DEV)[:, :vocab]
    tok = torch.randint(0, vocab, (n,), generator=g).to(DEV)
    dlogp = torch.randn(n, generator=g).to(DEV)
    dent = (torch.randn(n, generator=g) * 0.1).to(DEV)
    return x, tok, dlogp, dent


def check(name, got, want, bound):
    got = np64(got)
    with np.errstate(invalid="ignore"):
        err = np.where(got == want, 0, np.abs(got - want))
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    worst = float((err / bound).max()) if np.ndim(bound) else float(err.max())
    say(f"  {name}: worst error {float(err.max()):.3e}, {worst:.3f} of its bound")
    assert np.all(err <= bound), f"{name}: {worst} times its bound"


def run_case(parents, lens, x, tok, dlogp, dent, temperature=1.0, top_k=0):
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_logprobs(x, tok, plan, temperature=temperature, top_k=top_k)
    torch.cuda.synchronize()
    say("  forward done")
    d = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, temperature=temperature)
    torch.cuda.synchronize()
    ref = tree_logprobs_reference(parents, lens, np64(x), tok.cpu().numpy(), temperature, top_k)
    for name in ("logp", "entropy", "lse"):
        check(name, getattr(r, name), *ref[name])
    if top_k:
        assert np.array_equal(r.top_ids.cpu().numpy(), ref["top_ids"][0])
        check("top_logp", r.top_logp, *ref["top_logp"])
    want, bound = tree_logprobs_backward_reference(parents, lens, np64(x), tok.cpu().numpy(), np64(dlogp),
                                                   None if dent is None else np64(dent), temperature, U[x.dtype])
    check("dlogits", d, want, bound)
    return plan, r, d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 1000, 2047, 2049, 8192, 20001])
def test_logprobs_vocabularies(vocab, dtype):
    say(f"logprobs vocab={vocab} {dtype}")
    x, tok, dlogp, dent = inputs(22, vocab, DT[dtype])
    run_case(*TRIE, x, tok, dlogp, dent, top_k=min(vocab, 5))


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_logprobs_rows_further_apart(pad):
    for dtype in DT.values():
        say(f"logprobs pad={pad} {dtype}")
        x, tok, dlogp, dent = inputs(22, 5001, dtype, pad=pad)
        run_case(*TRIE, x, tok, dlogp, dent, top_k=3)


@pytest.mark.parametrize("temperature", [0.3, 1.7])
@pytest.mark.parametrize("top_k", [1, 16, 64])
def test_logprobs_temperature_and_top(temperature, top_k):
    say(f"logprobs T={temperature} k={top_k}")
    x, tok, dlogp, dent = inputs(22, 3001, torch.bfloat16, seed=4)
    run_case(*TRIE, x, tok, dlogp, dent, temperature, top_k)
    run_case(*TRIE, x.float(), tok.int(), dlogp, None, temperature, top_k)


def test_logprobs_many_rows():
    """From 512 rows on a row is one work-group's; below, several share it."""
    rng = np.random.default_rng(2)
    parents = [-1] + [int(rng.integers(0, i)) for i in range(1, 40)]
    lens = rng.integers(1, 40, size=40).tolist()
    n = sum(lens)
    assert n > 512
    say(f"logprobs N={n}")
    x, tok, dlogp, dent = inputs(n, 2311, torch.bfloat16, seed=6)
    run_case(parents, lens, x, tok, dlogp, dent, top_k=8)


def test_logprobs_ties_go_to_the_lowest_index():
    x, tok, dlogp, dent = inputs(22, 4100, torch.bfloat16, seed=7, spread=0.01)
    x = (x * 100).round() / 4  # a handful of values only
    say("logprobs ties")
    run_case(*TRIE, x, tok, dlogp, dent, top_k=32)
    run_case(*TRIE, torch.zeros_like(x), tok, dlogp, dent, top_k=64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_masked_vocabulary(dtype):
    """-inf and the type's lowest value over most of the vocabulary, a row of
    nothing but -inf, a row of nothing but the lowest value."""
    x, tok, dlogp, dent = inputs(22, 3000, DT[dtype], seed=9)
    x[:, 40:2500] = float("-inf")
    x[3:9, 2500:] = torch.finfo(x.dtype).min
    x[4] = float("-inf")
    x[11] = torch.finfo(x.dtype).min
    tok[1:] = torch.where(tok[1:] % 2 == 0, tok[1:] % 40, tok[1:])
    say(f"logprobs masked {dtype}")
    plan, r, d = run_case(*TRIE, x, tok, dlogp, dent, top_k=4)
    assert r.lse[4] == float("-inf") and r.entropy[4] == 0 and not d[4].any()
    assert r.top_ids[4].tolist() == [0, 1, 2, 3]
    assert (d[:, 40:2500][:4] == 0).sum() >= 4 * 2460 - 8


def test_logprobs_nan_and_inf_stay_in_their_rows():
    x, tok, dlogp, dent = inputs(22, 1000, torch.bfloat16, seed=3)
    plan = ptp.tree_plan(*TRIE, 4)
    a = ptp.tree_logprobs(x, tok, plan, top_k=4)
    y = x.clone()
    y[2, 17] = float("nan")
    y[9, 5] = float("inf")
    b = ptp.tree_logprobs(y, tok, plan, top_k=4)
    keep = torch.ones(22, dtype=torch.bool, device=DEV)
    keep[[2, 9]] = False
    assert torch.equal(a.lse[keep], b.lse[keep]) and torch.equal(a.entropy[keep], b.entropy[keep])
    assert torch.equal(a.top_ids[keep], b.top_ids[keep])
    assert torch.isnan(b.lse[2]) and torch.isnan(b.entropy[2]) and torch.isnan(b.logp[3])
    assert not torch.isfinite(b.lse[9]) and not torch.isfinite(b.entropy[9])
    assert 17 not in b.top_ids[2].tolist() and b.top_ids[9, 0] == 5
    y[2] = float("nan")
    assert ptp.tree_logprobs(y, tok, plan, top_k=4).top_ids[2].tolist() == [-1] * 4


def test_logprobs_tokens_outside_the_vocabulary():
    x, tok, dlogp, dent = inputs(22, 999, torch.float32, seed=12)
    tok[2], tok[7], tok[15] = -100, 999, 1 << 40
    say("logprobs ignored tokens")
    plan, r, d = run_case(*TRIE, x, tok, dlogp, dent)
    assert r.logp[2] == 0 and r.logp[7] == 0 and r.logp[15] == 0
    dlogp[2] = float("nan")  # not read
    assert torch.equal(d, ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent))


@pytest.mark.parametrize("fan", [3, 300, 700])
def test_logprobs_many_children_of_one_row(fan):
    """More children than a work-group keeps in LDS, several with the same
    first token: their gradients add up in the common row."""
    parents, lens = [-1] + [0] * fan, [2] + [1] * fan
    x, tok, dlogp, dent = inputs(fan + 2, 600, torch.float32, seed=fan)
    tok[2:] = tok[2:] % 200
    say(f"logprobs fan={fan}")
    run_case(parents, lens, x, tok, dlogp, dent)


@pytest.mark.parametrize("pad", [0, 3])
def test_logprobs_parts_of_a_trie_and_in_place(pad):
    """Rows a part at a time give the bits of the whole; the gradient written
    over the logits gives the bits of the one written apart."""
    x, tok, dlogp, dent = inputs(22, 2600, torch.bfloat16, seed=14, pad=pad)
    plan = ptp.tree_plan(*TRIE, 4)
    say(f"logprobs parts pad={pad}")
    r = ptp.tree_logprobs(x, tok, plan, top_k=3)
    d = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
    logp = torch.full((22,), 7.0, device=DEV)
    for a, b in ((0, 5), (5, 6), (6, 22)):
        p = ptp.tree_logprobs(x[a:b], tok, plan, top_k=3, first_row=a, logp=logp)
        for whole, part in ((r.lse, p.lse), (r.entropy, p.entropy), (r.top_logp, p.top_logp)):
            torch.testing.assert_close(part, whole[a:b], rtol=2e-6, atol=2e-5)
        assert torch.equal(p.top_ids, r.top_ids[a:b])
        dp = ptp.tree_logprobs_backward(x[a:b], tok, r.lse[a:b].contiguous(), r.entropy[a:b].contiguous(), dlogp, plan,
                                        dentropy=dent[a:b].contiguous(), first_row=a)
        assert torch.equal(dp, d[a:b])
    torch.testing.assert_close(logp, r.logp, rtol=2e-6, atol=2e-5)
    y = x.clone() if pad == 0 else x
    out = ptp.tree_logprobs_backward(y, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, out=y)
    assert out is y and torch.equal(y, d)


def test_logprobs_vocabulary_of_several_slices():
    """More columns than one work-group of the backward takes."""
    parents, lens = [-1, 0, 0], [2, 1, 1]
    x, tok, dlogp, dent = inputs(4, 300_001, torch.bfloat16, seed=21)
    say("logprobs 300001 columns")
    run_case(parents, lens, x, tok, dlogp, dent, top_k=8)


def test_logprobs_against_differences():
    """The gradient of sum_t g_t logp_t + sum_r h_r entropy_r by central
    differences of the forward in fp64 (the oracle's)."""
    x, tok, dlogp, dent = inputs(22, 12, torch.float32, seed=31)
    plan = ptp.tree_plan(*TRIE, 4)
    r = ptp.tree_logprobs(x, tok, plan, temperature=0.8)
    d = np64(ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, temperature=0.8))
    xs, toks = np64(x), tok.cpu().numpy()

    def loss(y):
        f = tree_logprobs_reference(*TRIE, y, toks, 0.8)
        return (f["logp"][0] * np64(dlogp)).sum() + (f["entropy"][0] * np64(dent)).sum()

    rng, h = np.random.default_rng(0), 1e-4
    for _ in range(40):
        i, j = rng.integers(0, 22), rng.integers(0, 12)
        y = xs.copy()
        y[i, j] += h
        up = loss(y)
        y[i, j] -= 2 * h
        # fp32 sums (2e-6) and the third derivative's h^2 term
        assert abs((up - loss(y)) / (2 * h) - d[i, j]) <= 2e-5


def test_logprobs_in_a_graph():
    plan = ptp.tree_plan(*TRIE, 4)
    x, tok, dlogp, dent = inputs(22, 5003, torch.bfloat16)
    r = ptp.tree_logprobs(x, tok, plan, top_k=4)
    ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gr = ptp.tree_logprobs(x, tok, plan, top_k=4)
        gd = ptp.tree_logprobs_backward(x, tok, gr.lse, gr.entropy, dlogp, plan, dentropy=dent)
    for i in range(4):
        say(f"logprobs replay {i}")
        for t, s in zip((x, tok, dlogp, dent), inputs(22, 5003, torch.bfloat16, seed=70 + i)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        r = ptp.tree_logprobs(x, tok, plan, top_k=4)
        d = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(r, gr)) and torch.equal(d, gd)


def test_logprobs_beyond_32_bit_offsets():
    """36,000 rows of 131,072 columns (9.4 GB): the last rows against the oracle,
    the gradient written over the logits."""
    n, vocab, last = 36_000, 131_072, 6
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    x = torch.empty((n, vocab), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    tok = torch.randint(0, vocab, (n,), generator=gen, device=DEV)
    dlogp = torch.randn(n, generator=gen, device=DEV)
    dent = torch.randn(n, generator=gen, device=DEV) * 0.1
    plan = ptp.tree_plan([-1, 0], [n - last, last], 4)
    say("logprobs 36000 x 131072")
    r = ptp.tree_logprobs(x, tok, plan, top_k=3)
    tail = np64(x[-last:])
    d = ptp.tree_logprobs_backward(x, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, out=x)
    torch.cuda.synchronize()
    ref = tree_logprobs_reference([-1], [last], tail, tok[-last:].cpu().numpy(), 1.0, 3)
    check("logp", r.logp[-last + 1:], ref["logp"][0][1:], ref["logp"][1][1:])
    check("entropy", r.entropy[-last:], *ref["entropy"])
    assert np.array_equal(r.top_ids[-last:].cpu().numpy(), ref["top_ids"][0])
    want, bound = tree_logprobs_backward_reference([-1], [last], tail, tok[-last:].cpu().numpy(), np64(dlogp[-last:]),
                                                   np64(dent[-last:]), 1.0, U[torch.bfloat16])
    check("dlogits", d[-last:], want, bound)
    assert torch.isfinite(r.logp).all() and d is x


def test_logprobs_more_rows_than_one_launch_takes():
    """17 million rows of 4 columns, forward and backward, against torch in
    fp64 on the same device."""
    n, vocab = 17_000_000, 4
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    x = torch.empty((n, vocab), device=DEV).normal_(generator=gen)
    tok = torch.randint(0, vocab, (n,), generator=gen, device=DEV, dtype=torch.int32)
    g = torch.empty(n, device=DEV).normal_(generator=gen)
    plan = ptp.tree_plan([-1], [n], 4)
    say("logprobs 17000000 x 4")
    r = ptp.tree_logprobs(x, tok, plan, top_k=1)
    d = ptp.tree_logprobs_backward(x, tok, r.lse, None, g, plan)
    torch.cuda.synchronize()
    ls = x.double().log_softmax(-1)
    bound = 200 * 2.0 ** -24  # a few roundings of values below 12
    want = torch.cat([ls.new_zeros(1), ls[:-1].gather(1, tok[1:, None].long())[:, 0]])
    assert (r.logp - want).abs().max() <= bound
    assert (r.entropy + (ls.exp() * ls).sum(-1)).abs().max() <= bound
    assert torch.equal(r.top_ids[:, 0].long(), x.argmax(-1))
    gd = torch.cat([g[1:].double(), g.new_zeros(1).double()])[:, None]
    one = torch.zeros_like(ls)
    one[:-1].scatter_(1, tok[1:, None].long(), 1.0)
    assert ((d - gd * (one - ls.exp())).abs() <= bound * (1 + gd.abs())).all()


def test_logprobs_refusals():
    x, tok, dlogp, dent = inputs(22, 100, torch.bfloat16)
    plan = ptp.tree_plan(*TRIE, 4)
    r = ptp.tree_logprobs(x, tok, plan)
    with pytest.raises(TypeError):
        ptp.tree_logprobs(x, tok.float(), plan)
    with pytest.raises(ValueError):
        ptp.tree_logprobs(x, tok[:21], plan)
    with pytest.raises(ValueError):
        ptp.tree_logprobs(x, tok, plan, first_row=1)
    with pytest.raises(ValueError):
        ptp.tree_logprobs(x.t().contiguous().t(), tok, plan)
    for k in (-1, 65):
        with pytest.raises(_lib.TreeError, match="top_k"):
            ptp.tree_logprobs(x, tok, plan, top_k=k)
    with pytest.raises(_lib.TreeError, match="top_k"):
        ptp.tree_logprobs(x[:, :3], tok, plan, top_k=4)
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        with pytest.raises(_lib.TreeError, match="temperature"):
            ptp.tree_logprobs(x, tok, plan, temperature=t)
    with pytest.raises(TypeError):
        ptp.tree_logprobs_backward(x, tok, r.lse.double(), r.entropy, dlogp, plan)
    with pytest.raises(TypeError):
        ptp.tree_logprobs_backward(x, tok, r.lse, None, dlogp, plan, dentropy=dent)
    with pytest.raises(ValueError, match="workspace"):
        ptp.tree_logprobs(inputs(22, 5000, torch.bfloat16)[0], tok, plan, top_k=1,
                          workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
