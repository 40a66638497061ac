"""Log probabilities from hidden states and the output weight on the GPU, forward
and backward, against the fp64 oracle (oracle/linear.py) with its bounds: widths
and vocabularies that end inside a tile, every tile size, split contractions,
several pieces of the vocabulary and parts of the rows, rows far apart, tokens
outside the vocabulary, many children, values that are not finite, graphs."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.linear import tree_linear_logprobs_backward_reference, tree_linear_logprobs_reference
from prefix_tree_packed_plan_amd import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# Partial products of a term, each added in fp32.
TERMS = {torch.bfloat16: 1, torch.float32: 6}
TRIE = ([-1, 0, 0, 2, 2, 2, -1], [5, 3, 1, 2, 1, 4, 6])


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def np64(t):
    return t.detach().double().cpu().numpy()


def chain(n):
    """A trie of n tokens: a root with two children, one of which forks."""
    if n < 8:
        return [-1], [n]
    a, b, c = n // 3, n // 4, n // 8
    return [-1, 0, 0, 2, 2], [a, b, c, 1, n - a - b - c - 1]


def inputs(n, vocab, width, dtype, seed=1, pad=0, ids=torch.int64):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((n, width + pad), generator=g).to(dtype).to(DEV)[:, :width]
    w = (torch.randn((vocab, width), generator=g) * (2.0 / width ** 0.5)).to(dtype).to(DEV)
    tok = torch.randint(0, vocab, (n,), generator=g).to(ids).to(DEV)
    dlogp = torch.randn(n, generator=g).to(DEV)
    dent = (torch.randn(n, generator=g) * 0.1).to(DEV)
    return h, w, tok, dlogp, dent


def check(name, got, want, bound):
    got = np64(got)
    assert got.shape == want.shape
    with np.errstate(invalid="ignore"):
        err = np.where(got == want, 0, np.abs(got - want))
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), name
    say(f"  {name}: worst error {float(err.max()):.3e}, {float((err / bound).max()):.3f} of its bound")
    assert np.all(err <= bound), name
    return err


def run_case(parents, lens, h, w, tok, dlogp, dent, temperature=1.0, rms_too=True):
    plan = ptp.tree_plan(parents, lens, 4)
    terms = TERMS[h.dtype]
    r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=temperature)
    torch.cuda.synchronize()
    say("  forward done")
    d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy if dent is not None else None, dlogp, plan,
                                          dentropy=dent, temperature=temperature)
    torch.cuda.synchronize()
    t = tok.cpu().numpy()
    ref = tree_linear_logprobs_reference(parents, lens, np64(h), np64(w), t, temperature, terms)
    for name in ("logp", "entropy", "lse"):
        check(name, getattr(r, name), *ref[name])
    assert r.top_logp is None and r.top_ids is None
    ref = tree_linear_logprobs_backward_reference(parents, lens, np64(h), np64(w), t, np64(dlogp),
                                                  None if dent is None else np64(dent), temperature, U[h.dtype], terms)
    for name, x in zip(("dhidden", "dweight"), d):
        assert x.dtype == h.dtype
        want, bound, rms = ref[name]
        err = check(name, x, want, bound)
        if rms_too and h.dtype == torch.bfloat16 and err.size > 5000:
            ratio = np.sqrt(((err / rms) ** 2).mean())
            say(f"  {name}: {ratio:.3f} of the roundings' size")
            # Relative roundings are u / sqrt(3) in the mean at most, 0.74 of that for
            # mantissas spread evenly; fp32 sums add little.
            assert ratio < 1.0
    return plan, r, d


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("width", [8, 16, 40, 64, 72, 120, 128, 136, 520])
def test_widths(width, dtype):
    say(f"linear logprobs width={width} {dtype}")
    run_case(*TRIE, *inputs(22, 700, width, DT[dtype], seed=width))


@pytest.mark.parametrize("width", [4, 12, 36, 100])
def test_widths_of_fp32(width):
    say(f"linear logprobs width={width} f32")
    run_case(*TRIE, *inputs(22, 333, width, torch.float32, seed=width))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 32, 33, 127, 128, 129, 255, 257, 1003, 2049])
def test_vocabularies(vocab, dtype):
    say(f"linear logprobs vocab={vocab} {dtype}")
    run_case(*TRIE, *inputs(22, vocab, 72, DT[dtype], seed=vocab))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n", [1, 2, 31, 33, 63, 64, 65, 127, 129, 200, 257])
def test_rows(n, dtype):
    """Up to 64 rows the tiles are 64 rows wide, then 128."""
    say(f"linear logprobs n={n} {dtype}")
    run_case(*chain(n), *inputs(n, 500, 96, DT[dtype], seed=n))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab,width", [(300, 25000, 64), (1100, 10300, 72), (600, 6500, 1032), (129, 24700, 264)])
def test_large_tiles_and_splits(n, vocab, width, dtype):
    """256 x 256 tiles where they fill the chip; few tiles over a long contraction are split."""
    say(f"linear logprobs n={n} vocab={vocab} width={width} {dtype}")
    run_case(*chain(n), *inputs(n, vocab, width, DT[dtype], seed=n))


def exact(parents, lens, h, w, tok, dlogp, dent, temperature):
    """The formulas in 64 bits on the GPU, by blocks of rows."""
    from oracle.logprobs import front_rows
    front = torch.as_tensor(front_rows(parents, lens), device=DEV)
    h, w = h.double(), w.double()
    n = len(h)
    logp = torch.zeros(n, dtype=torch.float64, device=DEV)
    lse, ent = torch.zeros_like(logp), torch.zeros_like(logp)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for i in range(0, n, 2048):
        ls = (h[i:i + 2048] @ w.t() / temperature)
        lse[i:i + 2048] = ls.logsumexp(-1)
        ls = ls.log_softmax(-1)
        p = ls.exp()
        e = -(p * ls).sum(-1)
        ent[i:i + 2048] = e
        t = torch.nonzero((front >= i) & (front < i + 2048))[:, 0]
        logp[t] = ls[front[t] - i, tok[t].long()]
        g = dlogp[t].double()
        d = -dent[i:i + 2048, None].double() * p * (ls + e[:, None])
        d -= p * torch.zeros(len(p), dtype=torch.float64, device=DEV).index_add_(0, front[t] - i, g)[:, None]
        d.index_put_((front[t] - i, tok[t].long()), g, accumulate=True)
        d /= temperature
        dh[i:i + 2048] = d @ w
        dw += d.t() @ h[i:i + 2048]
    return logp, ent, lse, dh, dw


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab", [(16385, 16500), (33000, 700), (200, 40000)])
def test_parts_of_rows_and_pieces_of_the_vocabulary(n, vocab, dtype):
    """More rows than the backward takes at once (16384) and the forward (32768), more
    entries than a piece holds for so many rows."""
    width = 64
    say(f"linear logprobs n={n} vocab={vocab} {dtype}")
    parents, lens = chain(n)
    h, w, tok, dlogp, dent = inputs(n, vocab, width, DT[dtype], seed=2)
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=0.9)
    torch.cuda.synchronize()
    d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, temperature=0.9)
    torch.cuda.synchronize()
    want = exact(parents, lens, h, w, tok, dlogp, dent, 0.9)
    # Sums of 64 products and of exponentials in fp32, of values up to about 20.
    for name, x, y in zip(("logp", "entropy", "lse"), (r.logp, r.entropy, r.lse), want):
        err = (x.double() - y).abs().max().item()
        say(f"  {name}: {err:.2e}")
        assert err <= 2e-5
    # A rounding of D and one of the result, u / sqrt(3) each at most in the mean;
    # fp32 sums of a few thousand terms, by the square root of their number.
    most = 2.0 ** -8 * (2 / 3) ** 0.5 if dtype == "bf16" else 3e-6
    for name, x, y in zip(("dhidden", "dweight"), d, want[3:]):
        rel = ((x.double() - y).norm() / y.norm()).item()
        worst = ((x.double() - y).norm(dim=1) / (y.norm(dim=1) + 1e-3 * y.norm(dim=1).mean())).max().item()
        say(f"  {name}: {rel:.2e} of the norm, worst row {worst:.2e}")
        assert rel <= most and worst <= 4 * most


@pytest.mark.parametrize("n,vocab,width", [(1100, 30001, 2056), (4100, 1100, 2056)])
def test_large_tiles_of_the_hidden_states_gradient(n, vocab, width):
    """dhidden by 256 x 256 tiles, in several splits and in one; bf16."""
    say(f"linear logprobs n={n} vocab={vocab} width={width} bf16")
    parents, lens = chain(n)
    h, w, tok, dlogp, dent = inputs(n, vocab, width, torch.bfloat16, seed=3)
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
    torch.cuda.synchronize()
    want = exact(parents, lens, h, w, tok, dlogp, dent, 1.0)
    # 65 sums of 32 products, each rounded at a size of 16 at most (2^-21), and as many
    # of the exponentials' sums, to whose logarithm each gives 2^-24.
    for name, x, y in zip(("logp", "entropy", "lse"), (r.logp, r.entropy, r.lse), want):
        err = (x.double() - y).abs().max().item()
        say(f"  {name}: {err:.2e}")
        assert err <= 65 * 2.0 ** -21 + 1e-5
    # As above: two roundings.
    most = 2.0 ** -8 * (2 / 3) ** 0.5
    for name, x, y in zip(("dhidden", "dweight"), d, want[3:]):
        rel = ((x.double() - y).norm() / y.norm()).item()
        worst = ((x.double() - y).norm(dim=1) / (y.norm(dim=1) + 1e-3 * y.norm(dim=1).mean())).max().item()
        say(f"  {name}: {rel:.2e} of the norm, worst row {worst:.2e}")
        assert rel <= most and worst <= 4 * most


@pytest.mark.parametrize("n,vocab,width", [(1, 300, 264), (5, 9001, 72), (32, 2000, 136), (33, 32000, 64),
                                           (64, 5000, 264), (40, (1 << 20) + 300, 8), (65, 5000, 264)])
def test_few_rows_round_once(n, vocab, width):
    """Up to 64 rows of bf16 the logits' gradient is two bf16 numbers, so that the gradients
    are off by their own rounding alone; 65 and more by both."""
    say(f"linear logprobs n={n} vocab={vocab} width={width} bf16")
    parents, lens = chain(n)
    h, w, tok, dlogp, dent = inputs(n, vocab, width, torch.bfloat16, seed=n, pad=8)
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
    torch.cuda.synchronize()
    want = exact(parents, lens, h, w, tok, dlogp, dent, 1.0)
    for name, x, y in zip(("dhidden", "dweight"), d, want[3:]):
        rel = ((x.double() - y).norm() / y.norm()).item()
        say(f"  {name}: {rel:.2e} of the norm")
        # A rounding is 2^-8 / sqrt(3) at most in the mean, 0.74 of that over mantissas
        # spread evenly, which leaves room for chance over 264 values and more.
        assert rel <= 2.0 ** -8 * ((1 if n <= 64 else 2) / 3) ** 0.5


@pytest.mark.parametrize("temperature", [0.3, 1.7])
def test_temperature_and_strides(temperature):
    for dtype in DT.values():
        for pad in (0, 8, 64):
            say(f"linear logprobs T={temperature} pad={pad} {dtype}")
            h, w, tok, dlogp, dent = inputs(22, 900, 48, dtype, seed=4, pad=pad, ids=torch.int32)
            run_case(*TRIE, h, w, tok, dlogp, dent, temperature)
            run_case(*TRIE, h, w, tok, dlogp, None, temperature)


def test_parts_of_a_trie():
    """Rows a part at a time give the same logp, and gradients that add up."""
    for dtype in DT.values():
        say(f"linear logprobs parts {dtype}")
        parents, lens = chain(200)
        h, w, tok, dlogp, dent = inputs(200, 800, 64, dtype, seed=5)
        plan, r, (dh, dw) = run_case(parents, lens, h, w, tok, dlogp, dent)
        logp = torch.full((200,), float("nan"), device=DEV)
        total = torch.zeros_like(dw, dtype=torch.float32)
        for a, b in ((0, 67), (67, 68), (68, 200)):
            q = ptp.tree_linear_logprobs(h[a:b], w, tok, plan, first_row=a, logp=logp)
            assert q.logp is logp
            assert torch.allclose(q.lse, r.lse[a:b], rtol=0, atol=1e-5)
            x, y = ptp.tree_linear_logprobs_backward(h[a:b], w, tok, q.lse, q.entropy, dlogp, plan,
                                                     dentropy=dent[a:b], first_row=a)
            torch.cuda.synchronize()
            assert (x.float() - dh[a:b].float()).norm() <= 2 * U[dtype] * dh[a:b].float().norm() + 1e-5
            total += y.float()
        assert torch.allclose(logp, r.logp, rtol=0, atol=1e-5)
        assert (total - dw.float()).norm() <= 4 * U[dtype] * dw.float().norm() + 1e-5


def test_tokens_outside_and_many_children():
    """A row with hundreds of tokens behind it, several of them equal; tokens that are
    not asked for, whose dlogp is not read."""
    parents = [-1] + [0] * 700
    lens = [3] + [1] * 700
    for dtype in DT.values():
        say(f"linear logprobs children {dtype}")
        h, w, tok, dlogp, dent = inputs(703, 400, 40, dtype, seed=6)
        tok[5::3] = 17
        tok[7], tok[8], tok[9] = -1, 400, 2 ** 40
        tok[0] = -5
        dlogp[7:10] = float("nan")
        dlogp[0] = float("nan")  # a root's first token has no row in front
        clean = torch.nan_to_num(dlogp)
        plan = ptp.tree_plan(parents, lens, 4)
        r = ptp.tree_linear_logprobs(h, w, tok, plan)
        d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
        torch.cuda.synchronize()
        assert r.logp[0] == 0 and not r.logp[7:10].any()
        _, r2, d2 = run_case(parents, lens, h, w, tok, clean, dent)
        assert torch.equal(r.logp, r2.logp) and all(torch.equal(a, b) for a, b in zip(d, d2))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("vocab", [41, 700])
def test_hundreds_of_children(vocab, dtype):
    """More children than lanes, at two branch points of one tile of rows and one of
    another, many with the same token and some outside the vocabulary; and the rows in
    two calls, which must write the tokens behind their own rows alone."""
    parents = [-1] + [0] * 150 + [3] * 70 + [150] * 130 + [-1]
    lens = [4] + [1 + i % 2 for i in range(350)] + [3]
    n = sum(lens)
    say(f"linear logprobs n={n} children={350} vocab={vocab} {dtype}")
    h, w, tok, dlogp, dent = inputs(n, vocab, 40, DT[dtype], seed=vocab)
    tok[10:300:17] = -1
    tok[40:90] = 7
    plan, r, (_, dw) = run_case(parents, lens, h, w, tok, dlogp, dent)
    logp = torch.full((n,), 5.0, device=DEV)
    for a, b in ((130, n), (0, 130)):
        before = logp.clone()
        ptp.tree_linear_logprobs(h[a:b], w, tok, plan, first_row=a, logp=logp)
        front = _front(parents, lens)
        mine = torch.tensor([a <= f < b for f in front], device=DEV)
        start = torch.tensor([f < 0 and a <= t < b for t, f in enumerate(front)], device=DEV)
        assert torch.equal(logp[~mine & ~start], before[~mine & ~start])
    # The two calls' tiles are cut elsewhere: sums differ in their order.
    assert (logp - r.logp).abs().max() <= 2.0 ** -17


def _front(parents, lens):
    first = np.concatenate([[0], np.cumsum(lens)])
    out = []
    for s, p in enumerate(parents):
        out += [int(first[p + 1]) - 1 if p >= 0 else -1] + list(range(int(first[s]), int(first[s + 1]) - 1))
    return out


def test_values_that_are_not_finite():
    for dtype in DT.values():
        say(f"linear logprobs not finite {dtype}")
        h, w, tok, dlogp, dent = inputs(22, 300, 40, dtype, seed=7)
        plan = ptp.tree_plan(*TRIE, 4)
        a = ptp.tree_linear_logprobs(h, w, tok, plan)
        g = h.clone()
        g[4, 3], g[12, 0] = float("nan"), float("inf")
        b = ptp.tree_linear_logprobs(g, w, tok, plan)
        torch.cuda.synchronize()
        rows = torch.ones(22, dtype=torch.bool, device=DEV)
        rows[[4, 12]] = False
        assert torch.equal(a.lse[rows], b.lse[rows]) and torch.equal(a.entropy[rows], b.entropy[rows])
        assert torch.isnan(b.lse[~rows]).all() and torch.isnan(b.entropy[~rows]).all()
        # dhidden of the others is as before; the last row of a tile is not repeated into others.
        g = h.clone()
        g[21] = float("nan")
        b = ptp.tree_linear_logprobs(g, w, tok, plan)
        da, _ = ptp.tree_linear_logprobs_backward(h, w, tok, a.lse, a.entropy, dlogp, plan)
        db, _ = ptp.tree_linear_logprobs_backward(g, w, tok, b.lse, b.entropy, dlogp, plan)
        torch.cuda.synchronize()
        assert torch.equal(da[:21], db[:21]) and torch.isnan(db[21]).all()


def test_rows_whose_logits_are_all_minus_infinity():
    """Hidden states of -inf against a positive weight (bf16; in fp32 the parts of an
    infinity are not numbers): lse -inf, entropy 0, log probabilities -inf."""
    h, w, tok, dlogp, dent = inputs(22, 300, 8, torch.bfloat16, seed=8)
    w = w.abs() + 0.1
    h[6] = float("-inf")
    plan = ptp.tree_plan(*TRIE, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    torch.cuda.synchronize()
    assert r.lse[6] == float("-inf") and r.entropy[6] == 0 and r.logp[7] == float("-inf")
    assert torch.isfinite(torch.cat([r.lse[:6], r.lse[7:], r.entropy])).all()


def test_large_logits():
    """Logits of thousands: probabilities of 1 and 0 without overflow."""
    for dtype in DT.values():
        say(f"linear logprobs large {dtype}")
        h, w, tok, dlogp, dent = inputs(22, 300, 40, dtype, seed=9)
        # Without the mean size of the roundings: where p is 1 to fp32, D = g - G p is a
        # difference of equal numbers, which is off by 2^-24 |lse| g and whose value, 0,
        # has no rounding to be held against.
        run_case(*TRIE, h * 64, w * 16, tok, dlogp, dent, rms_too=False)


def test_repeats_streams_workspaces_and_graphs():
    for dtype in DT.values():
        h, w, tok, dlogp, dent = inputs(300, 9000, 136, dtype, seed=10)
        parents, lens = chain(300)
        plan = ptp.tree_plan(parents, lens, 4)

        def both(ws=(None, None)):
            r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=0.8, workspace=ws[0])
            d = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent,
                                                  temperature=0.8, workspace=ws[1])
            return r.logp, r.entropy, r.lse, *d

        lib, code = _lib.load(), _lib._dtype_code(h)
        sizes = (lib.tree_linear_logprobs_workspace_bytes(300, 9000, 136, code),
                 lib.tree_linear_logprobs_backward_workspace_bytes(300, 9000, 136, code))
        say(f"linear logprobs workspaces {sizes} {dtype}")
        want = both()
        ws = [torch.full((s,), 0xFF, dtype=torch.uint8, device=DEV) for s in sizes]  # NaN throughout
        assert all(torch.equal(a, b) for a, b in zip(want, both(ws)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = both()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        for i in range(4):
            for x, y in zip((h, w, tok, dlogp, dent), inputs(300, 9000, 136, dtype, seed=30 + i)):
                x.copy_(y)
            for x in out:
                x.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, both()))


def test_python_refusals():
    h, w, tok, dlogp, dent = inputs(22, 300, 40, torch.bfloat16, seed=7)
    plan = ptp.tree_plan(*TRIE, 4)
    f, b = ptp.tree_linear_logprobs, ptp.tree_linear_logprobs_backward
    lse = torch.zeros(22, device=DEV)
    for bad in (lambda: f(h[:, :32], w, tok, plan), lambda: f(h, w[:, :32], tok, plan), lambda: f(h, w, tok[1:], plan),
                lambda: f(h, w, tok, plan, first_row=1), lambda: f(h[:0], w, tok, plan), lambda: f(h, w[0], tok, plan),
                lambda: f(h.t(), w, tok, plan), lambda: f(h, w, tok, plan, logp=lse[:5]),
                lambda: f(h, w, tok, plan, workspace=torch.empty(8, device=DEV)),
                lambda: b(h, w, tok, lse[1:], None, dlogp, plan), lambda: b(h, w, tok, lse, None, dlogp[1:], plan),
                lambda: b(h, w, tok, lse, lse, dlogp, plan, dentropy=dent[2:]),
                lambda: b(h, w, tok, lse, lse, dlogp, plan, workspace=torch.empty(8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(h, w.float(), tok, plan), lambda: f(h.half(), w.half(), tok, plan),
                lambda: f(h, w, tok.float(), plan), lambda: b(h, w, tok, lse, None, dlogp, plan, dentropy=dent)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(h[:, :36].contiguous(), w[:, :36].contiguous(), tok, plan),
                lambda: f(h, w, tok, plan, temperature=0.0), lambda: b(h, w, tok, lse, None, dlogp, plan, temperature=-1.0),
                lambda: f(torch.empty(22 * 40 + 4, dtype=h.dtype, device=DEV)[4:].view(22, 40), w, tok, plan)):
        with pytest.raises(_lib.TreeError):
            bad()
