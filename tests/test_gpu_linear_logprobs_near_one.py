"""Log probabilities from hidden states and the output weight where a token has
nearly all of its row's probability: its logit and the row's largest one are the
same number, whatever the tile size, so that no log probability is above 0 and a
small one is not lost in two logits' difference."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# Rows and entries that take tiles of 64 x 64, 128 x 128 and (bf16) 256 x 256.
SIZES = [(22, 1), (22, 700), (600, 10300), (2100, 9000), (300, 25000)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab", SIZES)
@pytest.mark.parametrize("width", [8, 40, 504, 520, 1000, 2048, 4104])
def test_equal_logits(width, n, vocab, dtype):
    """With all rows of the weight equal, every log probability is bitwise minus the entropy:
    exp(0) = 1 for every entry, and the token's is one of them."""
    print(f"equal logits n={n} vocab={vocab} width={width} {dtype}", file=sys.stderr, flush=True)
    g = torch.Generator().manual_seed(width)
    h = torch.randn((n, width), generator=g).to(DT[dtype]).to(DEV)
    w = torch.randn((1, width), generator=g).to(DT[dtype]).to(DEV).repeat(vocab, 1)
    tok = torch.randint(0, vocab, (n,), generator=g).to(DEV)
    a = n // 3
    # A root with two children of one token and a long one, the second of which forks.
    plan = ptp.tree_plan([-1, 0, 0, 0, 2, 2], [a, 1, 1, n - a - 6, 2, 2], 4)
    front = torch.tensor([-1] + list(range(a - 1)) + [a - 1] * 3 + list(range(a + 2, n - 5))
                         + [a + 1, n - 4, a + 1, n - 2], device=DEV)
    assert len(front) == n
    for temperature in (1.0, 0.7):
        r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=temperature)
        torch.cuda.synchronize()
        assert torch.equal(r.logp[1:], -r.entropy[front[1:]])


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab", [(64, 1000), (600, 10300), (300, 25000)])
@pytest.mark.parametrize("width", [40, 256, 2048, 4096])
def test_probabilities_near_one(width, n, vocab, dtype):
    print(f"near one n={n} vocab={vocab} width={width} {dtype}", file=sys.stderr, flush=True)
    g = torch.Generator().manual_seed(width)
    h = torch.randn((n, width), generator=g)
    w = torch.randn((vocab, width), generator=g) * (0.5 / width ** 0.5)
    h, w = h.to(DT[dtype]).to(DEV), w.to(DT[dtype]).to(DEV)
    tok = torch.arange(n, device=DEV)
    # The next token's logit is 6 to 30 where the others' are about 0.5, or its row's length apart.
    size = torch.linspace(6, 30, n, device=DEV)[:, None]
    w[1:n] = (h[:-1].float() * (size[1:] / h[:-1].float().square().sum(1, keepdim=True))).to(h.dtype)
    r = ptp.tree_linear_logprobs(h, w, tok, ptp.tree_plan([-1], [n], 4))
    torch.cuda.synchronize()
    want = (h.double() @ w.double().t()).log_softmax(-1)[:-1].gather(1, tok[1:, None])[:, 0]
    assert (r.logp <= 0).all()
    # Where the token is nearly certain: a sum of 1 and little else, rounded in 16 steps at
    # most (2^-24 each), its logarithm; the little, of 1e-3, by the logits' errors, of 1e-4.
    sure = want > -1e-3
    assert sure.any()
    assert (r.logp[1:].double() - want)[sure].abs().max() <= 2.0 ** -20
