"""Token embedding and its gradient where element offsets pass 2^31 and byte
offsets 2^32, in the table, the output, the upstream gradient and the table's
gradient; and every bf16 number looked up."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("width", [1032, 1031])
def test_a_large_table(width, dtype):
    """2^21 + 5 rows, more than 2^31 elements, and as many tokens."""
    vocab = n = (1 << 21) + 5
    say(f"large table {vocab} x {width} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(1)
    some = torch.randn((4099, width), generator=g, device=DEV).to(DT[dtype])
    table = torch.empty((vocab, width), dtype=DT[dtype], device=DEV)
    for i in range(0, vocab, 4099):
        table[i:i + 4099] = some[:min(4099, vocab - i)].roll(i // 4099 % 64, 1)
    tok = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    tok[:3] = torch.tensor([vocab - 1, 0, vocab])
    tok[-3:] = torch.tensor([-1, vocab - 1, vocab - 2])
    out = ptp.tree_embedding(tok, table)
    torch.cuda.synchronize()
    say("  forward done")
    zero = torch.zeros(width, dtype=table.dtype, device=DEV)
    for i in range(0, n, 1 << 17):
        t = tok[i:i + (1 << 17)]
        has = (t >= 0) & (t < vocab)
        want = torch.where(has[:, None], table[t.clamp(0, vocab - 1)], zero)
        assert torch.equal(out[i:i + (1 << 17)], want), i


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("width", [1032, 1031])
def test_the_gradient_of_a_large_table(width, dtype):
    """As many tokens, in any order: most rows have one or none, the last has 5000."""
    vocab = n = (1 << 21) + 5
    say(f"large table's gradient {vocab} x {width} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(2)
    dout = torch.empty((n, width), dtype=DT[dtype], device=DEV)
    for i in range(0, n, 1 << 17):
        m = min(1 << 17, n - i)
        dout[i:i + m] = torch.randn((m, width), generator=g, device=DEV)
    tok = torch.randperm(n, generator=g, device=DEV)
    often = torch.randperm(n, generator=g, device=DEV)[:5000]
    tok[often] = vocab - 1
    tok[torch.randperm(n, generator=g, device=DEV)[:3000]] = -1
    d = ptp.tree_embedding_backward(tok, dout, vocab)
    torch.cuda.synchronize()
    say("  backward done")
    last = dout[tok == vocab - 1]
    assert len(last) > 4000
    want, size = last.double().sum(0), last.double().abs().sum(0)
    # fp32 sums of k numbers are off by k 2^-24 of their sizes at most; and a rounding.
    u = torch.finfo(d.dtype).eps / 2
    assert ((d[-1].double() - want).abs() <= len(last) * 2.0 ** -24 * size + u * want.abs()).all()
    where = torch.full((vocab,), -1, dtype=torch.int64, device=DEV)
    at = torch.nonzero((tok >= 0) & (tok < vocab - 1))[:, 0]
    where[tok[at]] = at
    for i in range(0, vocab - 1, 1 << 17):
        w = where[i:min(i + (1 << 17), vocab - 1)]
        want = torch.where((w >= 0)[:, None], dout[w.clamp_min(0)], torch.zeros((), dtype=d.dtype, device=DEV))
        assert torch.equal(d[i:i + len(w)], want), i


def test_every_number_is_copied():
    """All bf16 bit patterns (numbers too small to be normal and infinities among them) and
    fp32 ones of every exponent: a scale of 1 copies them, a token's only gradient is its
    row's."""
    say("every number")
    bits = torch.arange(1 << 16, dtype=torch.int32, device=DEV)
    for table in ((bits << 16).view(torch.float32).to(torch.bfloat16),
                  ((bits << 16) + 12345 * (bits % 5)).view(torch.float32)):
        table = table.reshape(256, 256)
        tok = torch.arange(255, -1, -1, device=DEV)
        for x in (table, table.t().contiguous()[:, :255].contiguous()):
            out = ptp.tree_embedding(tok, x)
            d = ptp.tree_embedding_backward(tok, out, 256)
            torch.cuda.synchronize()
            nan = torch.isnan(x)
            for got, want in ((out, x.flip(0)), (d, x)):
                nan = torch.isnan(want)
                assert torch.equal(torch.isnan(got), nan)
                assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want))
