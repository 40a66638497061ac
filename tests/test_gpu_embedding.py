"""Token embedding and its gradient on the GPU against sums in 64 bits: odd and
unaligned widths, tokens without a row, rows with one token, many or all of
them, tables larger than the sorting work-groups cover at once, other streams,
captured graphs.

Bounds: a product and a stored value are off by half a step each (bf16 2^-8,
fp32 2^-24 of the value); a sum of k terms in fp32 by k 2^-24 of the sum of
their sizes, in any order."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from prefix_tree_packed_plan_amd import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def check_forward(tok, table, scale):
    out = ptp.tree_embedding(tok, table, scale=scale)
    torch.cuda.synchronize()
    t, x = tok.cpu().numpy().astype(np.int64), np64(table)
    ok = (t >= 0) & (t < len(x))
    want = np.where(ok[:, None], np.float64(np.float32(scale)) * x[np.where(ok, t, 0)], 0)
    assert out.shape == want.shape and out.dtype == table.dtype
    err = np.abs(np64(out) - want)
    assert np.all(err <= (half_step(table.dtype) + U32) * np.abs(want) * (1 + U32)), err.max()
    if scale == 1.0:
        assert np.array_equal(np64(out), want)
    return out


def check_backward(tok, dout, vocab, scale, **kw):
    d = ptp.tree_embedding_backward(tok, dout, vocab, scale=scale, **kw)
    torch.cuda.synchronize()
    t, x = tok.cpu().numpy().astype(np.int64), np64(dout)
    ok = (t >= 0) & (t < vocab)
    want, size, count = np.zeros((vocab, x.shape[1])), np.zeros((vocab, x.shape[1])), np.zeros(vocab)
    np.add.at(want, t[ok], x[ok])
    np.add.at(size, t[ok], np.abs(x[ok]))
    np.add.at(count, t[ok], 1)
    s = np.float64(np.float32(scale))
    want, size = want * s, size * s
    bound = size * (count[:, None] + 1) * U32 * 1.01 + half_step(dout.dtype) * np.abs(want) * 1.01
    got = np64(d)
    assert d.dtype == dout.dtype
    err = np.abs(got - want)
    say(f"  worst error {err.max():.3e}, {(err / np.maximum(bound, 1e-300)).max():.3f} of its bound")
    assert np.all(err <= bound)
    assert not got[count == 0].any()
    return d


def inputs(n, vocab, width, dtype, seed=1, ids=torch.int64):
    g = torch.Generator().manual_seed(seed)
    tok = torch.randint(0, vocab, (n,), generator=g).to(ids).to(DEV)
    table = torch.randn((vocab, width), generator=g).to(dtype).to(DEV)
    dout = torch.randn((n, width), generator=g).to(dtype).to(DEV)
    return tok, table, dout


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 9, 33, 100, 255, 256, 1001, 2048, 2056, 4100])
def test_widths(width, dtype):
    say(f"embedding width={width} {dtype}")
    tok, table, dout = inputs(150, 61, width, DT[dtype], seed=width)
    check_forward(tok, table, 1.0)
    check_forward(tok, table, width ** 0.5)
    check_backward(tok, dout, 61, width ** 0.5)


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 127, 128, 129, 1023, 1025, 8193])
def test_lengths(n):
    say(f"embedding n={n}")
    for dtype, ids in ((torch.bfloat16, torch.int64), (torch.float32, torch.int32)):
        tok, table, dout = inputs(n, 37, 24, dtype, seed=n, ids=ids)
        check_forward(tok, table, 2.5)
        check_backward(tok, dout, 37, 2.5)


@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 513, 1003, 1025, 262144, 262145, 524288, 524289, 600001])
def test_vocabularies(vocab):
    """262144 rows are what 512 sorting work-groups cover; beyond that there are more."""
    say(f"embedding vocab={vocab}")
    tok, table, dout = inputs(3000, vocab, 16, torch.bfloat16, seed=vocab)
    tok[:3] = vocab - 1
    tok[5] = 0
    check_forward(tok, table, 1.0)
    check_backward(tok, dout, vocab, 1.0)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_tokens_outside_the_table(ids):
    tok, table, dout = inputs(700, 90, 40, torch.float32, seed=3, ids=ids)
    tok[::3] = -1
    tok[1::7] = 90
    tok[4] = torch.iinfo(ids).max
    tok[5] = torch.iinfo(ids).min
    say(f"embedding outside {ids}")
    check_forward(tok, table, 3.0)
    check_backward(tok, dout, 90, 3.0)
    tok.fill_(-100)
    assert not check_forward(tok, table, 1.0).any()
    assert not check_backward(tok, dout, 90, 1.0).any()
    # What a token without a row holds goes nowhere.
    tok[0], tok[1] = 7, 8
    dout[5:] = float("nan")
    d = ptp.tree_embedding_backward(tok, dout, 90)
    torch.cuda.synchronize()
    assert torch.isfinite(d).all() and torch.equal(d[7], dout[0]) and torch.equal(d[8], dout[1])


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("width", [5, 1024, 2600])
@pytest.mark.parametrize("kind", ["all one", "two halves", "runs", "one often", "just over"])
def test_long_lists(kind, width, dtype):
    """Rows with more tokens than a part, beginning and ending anywhere in one."""
    n = 2000
    g = torch.Generator().manual_seed(11)
    tok, _, dout = inputs(n, 50, width, DT[dtype], seed=5)
    if kind == "all one":
        tok.fill_(31)
    elif kind == "two halves":
        tok[:] = torch.where(torch.rand(n, generator=g) < 0.5, 3, 4).to(DEV)
    elif kind == "runs":  # lists of 1, 63, 64, 65, 66, 127, 128, 129, 200, ...
        lens = [1, 63, 64, 65, 66, 127, 128, 129, 200, 64, 65, 1, 2, 300]
        t = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        tok[:] = -1
        tok[:len(t)] = t[torch.randperm(len(t), generator=g)].to(DEV)
    elif kind == "one often":
        tok[torch.rand(n, generator=g).to(DEV) < 0.3] = 17
    else:
        tok[:] = torch.arange(n, device=DEV) // 65 % 50
    say(f"embedding {kind} width={width} {dtype}")
    check_backward(tok, dout, 50, 0.5)


def test_repeats_give_the_same_bits_in_token_order():
    """Sums run in ascending order of the tokens: up to 64 of them the exact fp32 sum
    one after another."""
    tok, _, dout = inputs(40, 3, 64, torch.float32, seed=8)
    tok.fill_(1)
    say("embedding order")
    d = check_backward(tok, dout, 3, 1.0)
    x = np.zeros(64, np.float32)
    for row in dout.cpu().numpy():
        x = x + row
    assert np.array_equal(d[1].cpu().numpy(), x)
    tok, _, dout = inputs(30000, 300, 264, torch.bfloat16, seed=9)
    tok[::2] = 5
    a = check_backward(tok, dout, 300, 1.0)
    for _ in range(3):
        assert torch.equal(a, ptp.tree_embedding_backward(tok, dout, 300))


@pytest.mark.parametrize("n", [5000, 70000])
def test_sorting_waves_with_more_tokens_than_they_keep(n):
    """A wave keeps 256 tokens of its rows at hand and looks for the others again; some
    waves do and some do not."""
    g = torch.Generator().manual_seed(n)
    tok = torch.randint(0, 40000, (n,), generator=g)
    tok[:n // 2] = torch.randint(0, 30, (n // 2,), generator=g)
    tok[n // 2 + 7] = 39999
    dout = torch.randn((n, 20), generator=g).to(DEV)
    say(f"embedding kept n={n}")
    check_backward(tok.to(DEV), dout, 40000, 1.0)
    check_backward(tok.int().to(DEV), dout.bfloat16(), 40000, 2.0)


def test_unaligned_tensors():
    for dtype in DT.values():
        say(f"embedding unaligned {dtype}")
        g = torch.Generator().manual_seed(4)
        flat = torch.randn(200 * 24 + 1, generator=g).to(dtype).to(DEV)
        x = flat[1:].view(200, 24)
        tok = torch.randint(0, 200, (333,), generator=g).to(DEV)
        out = torch.empty(333 * 24 + 1, dtype=dtype, device=DEV)[1:].view(333, 24)
        assert ptp.tree_embedding(tok, x, scale=2.0, out=out) is out
        assert torch.equal(out, check_forward(tok, x.clone(), 2.0))
        check_backward(tok[:200], x, 77, 1.0)


def test_values_that_are_not_finite_stay_in_their_rows():
    tok, table, dout = inputs(300, 40, 72, torch.bfloat16, seed=6)
    table[7, 3], table[9] = float("inf"), float("nan")
    out = ptp.tree_embedding(tok, table, scale=2.0)
    torch.cuda.synchronize()
    assert torch.equal(torch.isfinite(out), torch.isfinite(table[tok]))
    dout[11, 5] = float("inf")
    d = ptp.tree_embedding_backward(tok, dout, 40)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(d)
    assert bad.sum() == 1 and bad[tok[11], 5]


def test_workspace_and_refusals():
    tok, table, dout = inputs(300, 40, 72, torch.float32, seed=6)
    need = _lib.load().tree_embedding_backward_workspace_bytes(300, 40, 72)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    a = check_backward(tok, dout, 40, 1.0, workspace=ws)
    assert torch.equal(a, check_backward(tok, dout, 40, 1.0))
    with pytest.raises(ValueError, match="workspace"):
        ptp.tree_embedding_backward(tok, dout, 40, workspace=ws[:-1])
    for bad in (lambda: ptp.tree_embedding(tok, table[:, ::2]), lambda: ptp.tree_embedding(tok[None], table),
                lambda: ptp.tree_embedding(tok, table[0]), lambda: ptp.tree_embedding(tok, table, out=table),
                lambda: ptp.tree_embedding_backward(tok[:-1], dout, 40), lambda: ptp.tree_embedding(tok.cpu(), table),
                lambda: ptp.tree_embedding_backward(tok, dout, 40, out=table[:, :8])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ptp.tree_embedding(tok.float(), table), lambda: ptp.tree_embedding(tok, table.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ptp.tree_embedding(tok, table, scale=0.0), lambda: ptp.tree_embedding(tok, table, scale=-1.0),
                lambda: ptp.tree_embedding_backward(tok, dout, 40, scale=float("nan"))):
        with pytest.raises(_lib.TreeError):
            bad()


def test_streams_and_graphs():
    """On another stream than the current one's default, and captured: every replay
    on new inputs gives what an eager call gives."""
    tok, table, dout = inputs(1000, 200, 264, torch.bfloat16, seed=12)
    tok[::3] = 7
    want = check_forward(tok, table, 3.0), check_backward(tok, dout, 200, 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ptp.tree_embedding(tok, table, scale=3.0), ptp.tree_embedding_backward(tok, dout, 200, scale=3.0)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    say("embedding capture")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ptp.tree_embedding(tok, table, scale=3.0)
        d = ptp.tree_embedding_backward(tok, dout, 200, scale=3.0)
    for i in range(4):
        t, x, y = inputs(1000, 200, 264, torch.bfloat16, seed=20 + i)
        t[i::2] = 100 + i
        tok.copy_(t), table.copy_(x), dout.copy_(y)
        out.fill_(float("nan")), d.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ptp.tree_embedding(tok, table, scale=3.0))
        assert torch.equal(d, ptp.tree_embedding_backward(tok, dout, 200, scale=3.0))
