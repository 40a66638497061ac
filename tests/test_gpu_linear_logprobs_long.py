"""Log probabilities from hidden states and the output weight where element offsets
pass 2^31 and byte offsets 2^32: in the weight and its gradient, between far rows
of hidden, and in hidden and its gradient."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.logprobs import front_rows

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def fill(x, scale, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    step = max(1, (1 << 26) // x.shape[1])
    for i in range(0, len(x), step):
        m = min(step, len(x) - i)
        x[i:i + m] = torch.randn((m, x.shape[1]), generator=g, device=DEV) * scale
    return x


def run(n, vocab, width, h, w, dtype):
    """Against fp64 by pieces of the vocabulary, which hold a few GB."""
    g = torch.Generator().manual_seed(n)
    parents, lens = [-1, 0, 0], [n // 2, 1, n - n // 2 - 1]
    tok = torch.randint(0, vocab, (n,), generator=g)
    tok[-1] = vocab - 1
    tok, dlogp, dent = tok.to(DEV), torch.randn(n, generator=g).to(DEV), torch.randn(n, generator=g).to(DEV) * 0.1
    plan = ptp.tree_plan(parents, lens, 4)
    r = ptp.tree_linear_logprobs(h, w, tok, plan)
    torch.cuda.synchronize()
    say("  forward done")
    dh, dw = ptp.tree_linear_logprobs_backward(h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent)
    torch.cuda.synchronize()
    say("  backward done")
    front = torch.as_tensor(front_rows(parents, lens), device=DEV)
    t = torch.nonzero(front >= 0)[:, 0]
    rows = max(1, min(n, (1 << 27) // width))
    piece = max(1, min(vocab, (1 << 27) // max(width, rows)))
    lse, ent = torch.empty(n, dtype=torch.float64, device=DEV), torch.empty(n, dtype=torch.float64, device=DEV)
    z = torch.empty((n, vocab), dtype=torch.float64, device=DEV)
    for i in range(0, n, rows):
        hi = h[i:i + rows].double()
        for v in range(0, vocab, piece):
            z[i:i + rows, v:v + piece] = hi @ w[v:v + piece].double().t()
    ls = z.log_softmax(-1)
    lse = z.logsumexp(-1)
    del z
    p = ls.exp()
    ent = -(p * ls).sum(-1)
    logp = torch.zeros(n, dtype=torch.float64, device=DEV)
    logp[t] = ls[front[t], tok[t]]
    # Logits of up to 12 or so, of width / 32 sums or more, each rounded at 2^-21: at random, by
    # the square root of their number, and five times that.
    most = 5 * max(1.0, width / 32) ** 0.5 * 2.0 ** -21 + 1e-5
    for name, x, y in (("logp", r.logp, logp), ("entropy", r.entropy, ent), ("lse", r.lse, lse)):
        err = (x.double() - y).abs().max().item()
        say(f"  {name}: {err:.2e} of {most:.2e}")
        assert err <= most, name
    g64 = dlogp[t].double()
    d = -dent[:, None].double() * p * (ls + ent[:, None])
    del ls
    d -= p * torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, front[t], g64)[:, None]
    del p
    d.index_put_((front[t], tok[t]), g64, accumulate=True)
    # Two roundings, 2^-8 / sqrt(3) each at most in the mean; fp32: the sums, and the logits'.
    most = 2.0 ** -8 * (2 / 3) ** 0.5 if dtype == torch.bfloat16 else 3e-6 + most
    for name, got, a, b in (("dhidden", dh, d, w), ("dweight", dw, d.t(), h)):
        err = size = 0.0
        step = max(1, (1 << 27) // width)
        for i in range(0, len(got), step):
            x = torch.zeros((len(got[i:i + step]), width), dtype=torch.float64, device=DEV)
            for k in range(0, len(b), step):
                x += a[i:i + step, k:k + step] @ b[k:k + step].double()
            off = (got[i:i + step].double() - x).square().sum(1)
            whole = x.square().sum(1)
            err, size = err + off.sum().item(), size + whole.sum().item()
            # Each row by itself too: a wrong one among many would not show.
            assert (off.sqrt() <= 4 * most * (whole.sqrt() + 1e-3 * whole.mean().sqrt())).all(), (name, i)
        say(f"  {name}: {(err / size) ** 0.5:.2e} of the norm, limit {most:.2e}")
        assert (err / size) ** 0.5 <= most, name


@pytest.mark.parametrize("dtype", sorted(DT))
def test_a_large_weight(dtype):
    """2^22 entries (several pieces) of 520: 2^31 elements."""
    vocab, width = 1 << 22, 520
    say(f"large weight {vocab} x {width} {dtype}")
    w = fill(torch.empty((vocab, width), dtype=DT[dtype], device=DEV), 2 / width ** 0.5, 1)
    h = fill(torch.empty((7, width), dtype=DT[dtype], device=DEV), 1.0, 2)
    run(7, vocab, width, h, w, DT[dtype])


@pytest.mark.parametrize("dtype", sorted(DT))
def test_far_rows_of_hidden(dtype):
    """Rows 2^20 elements apart."""
    n, vocab, width = 2100, 700, 72
    say(f"far rows of hidden {n} {dtype}")
    h = torch.empty((n, 1 << 20), dtype=DT[dtype], device=DEV)[:, :width]
    fill(h, 1.0, 3)
    w = fill(torch.empty((vocab, width), dtype=DT[dtype], device=DEV), 2 / width ** 0.5, 4)
    run(n, vocab, width, h, w, DT[dtype])


@pytest.mark.parametrize("dtype", sorted(DT))
def test_large_hidden(dtype):
    """33000 rows (several parts) of 65536: 2^31 elements, and so is their gradient."""
    n, vocab, width = 33000, 100, 65536
    say(f"large hidden {n} x {width} {dtype}")
    h = fill(torch.empty((n, width), dtype=DT[dtype], device=DEV), 1.0, 5)
    w = fill(torch.empty((vocab, width), dtype=DT[dtype], device=DEV), 2 / width ** 0.5, 6)
    run(n, vocab, width, h, w, DT[dtype])
