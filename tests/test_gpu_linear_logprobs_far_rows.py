"""Log probabilities from hidden states and the output weight, and their
gradients, of rows whose logits are so large that their fp32 log-sum-exp does not
hold its last digits, or is out of range: forward and backward have to agree on
the probabilities."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.logprobs import front_rows

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LOW = torch.finfo(torch.bfloat16).min
# A logit's common part, by rows in turn.  With hidden states of -1, 0 and 1 and a weight in
# steps of 1/2 (1 in its first column), products are exact in fp32 up to 2^22; the last
# two rows have nothing but this part.
FAR = [0, 2.0 ** 13, -2.0 ** 15, 2.0 ** 17, 0, -2.0 ** 20, 2.0 ** 22, 5, -2.0 ** 22, 1e30, LOW]


def case(n, vocab, width, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    h = torch.randint(-1, 2, (n, width), generator=g).float()
    h[:, 6:] = 0
    w = torch.randint(-4, 5, (vocab, width), generator=g).float() / 2
    w[:, 0] = 1
    tok = torch.randint(0, vocab, (n,), generator=g)
    dlogp, dent = torch.randn(n, generator=g), torch.randn(n, generator=g) * 0.1
    far = torch.tensor([FAR[i % len(FAR)] for i in range(n)], dtype=torch.float64).to(dtype).float()
    h[:, 0] = far
    h[far.abs() > 1e9, 1:] = 0
    return h.to(dtype), w.to(dtype), tok, dlogp, dent, far


def formula(parents, lens, h, w, tok, dlogp, dent, temperature):
    """logp, entropy, lse, the logits' gradient and its terms' sizes in fp64."""
    n, front = len(h), front_rows(parents, lens)
    z = h @ w.T / temperature
    y = z - z.max(1, keepdims=True)
    ls = np.log(np.exp(y).sum(1))
    lp = y - ls[:, None]
    p = np.exp(lp)
    ent = -(p * lp).sum(1)
    logp, d = np.zeros(n), -dent[:, None] * p * (lp + ent[:, None])
    size = np.abs(dent)[:, None] * p * (np.abs(lp) + ent[:, None])
    for t in range(n):
        if front[t] >= 0:
            logp[t] = lp[front[t], tok[t]]
            d[front[t]] -= dlogp[t] * p[front[t]]
            d[front[t], tok[t]] += dlogp[t]
            size[front[t]] += abs(dlogp[t]) * p[front[t]]
            size[front[t], tok[t]] += abs(dlogp[t])
    return logp, ent, z.max(1) + ls, d / temperature, size / temperature


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("temperature", [0.7, 1.0, 4.0])
@pytest.mark.parametrize("n,vocab,width", [(22, 300, 8), (22, 37, 40), (60, 5000, 520), (300, 9000, 72), (300, 25000, 8),
                                           (17000, 300, 8)])
def test_gradients_of_far_rows(n, vocab, width, temperature, dtype):
    print(f"far rows n={n} vocab={vocab} width={width} T={temperature} {dtype}", file=sys.stderr, flush=True)
    dtype = DT[dtype]
    parents, lens = [-1, 0, 0, 2, 2], [n // 3, n // 4, n // 8, 1, n - n // 3 - n // 4 - n // 8 - 1]
    h, w, tok, dlogp, dent, far = case(n, vocab, width, dtype, seed=n + vocab)
    front = front_rows(parents, lens)
    for t in range(n):  # so that sums of these rows' products stay in range
        if front[t] >= 0 and abs(far[front[t]]) > 1e9:
            dlogp[t] *= 2.0 ** -12
    dent[far.abs() > 1e9] *= 2.0 ** -12
    plan = ptp.tree_plan(parents, lens, 4)
    a = [x.to(DEV) for x in (h, w, tok, dlogp, dent)]
    r = ptp.tree_linear_logprobs(*a[:3], plan, temperature=temperature)
    dh, dw = ptp.tree_linear_logprobs_backward(*a[:3], r.lse, r.entropy, a[3], plan, dentropy=a[4],
                                               temperature=temperature)
    torch.cuda.synchronize()
    h, w, dlogp, dent = (x.double().numpy() for x in (h, w, dlogp, dent))
    logp, ent, lse, d, size = formula(parents, lens, h, w, tok.numpy(), dlogp, dent, temperature)
    x64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    # Exact products; a difference, its scale (two roundings, 2^-24 each, of up to 150
    # units), the sum of exponentials and its logarithm.
    assert np.abs(x64(r.logp) - logp).max() <= 3e-5
    assert np.abs(x64(r.entropy) - ent).max() <= 3e-5
    most = np.finfo(np.float32).max
    want = np.clip(lse, -most, most)
    assert (np.abs(x64(r.lse) - want) <= 2.0 ** -22 * np.abs(want) + 3e-5).all()
    # The logits' gradient by the same, 5e-5 of its terms' sizes (rows near 2^14 have theirs
    # from the fp32 log-sum-exp: 2^-24 x 2^14 / 2 more), rounded to the type as both
    # products' operand; these sums in fp32, and a last rounding.
    u, e = U[dtype], 5e-5 + 2.0 ** -11
    for name, got, b, k in (("dhidden", dh, w, vocab), ("dweight", dw, h, n)):
        x, y = (d, size) if name == "dhidden" else (d.T, size.T)
        bound = u * np.abs(x @ b) + (u + e + 6 * k * 2.0 ** -24) * (y @ np.abs(b)) + 2.0 ** -100
        err = np.abs(x64(got) - x @ b)
        assert np.isfinite(x64(got)).all(), name
        print(f"  {name}: {(err / bound).max():.3f} of its bound", file=sys.stderr, flush=True)
        assert (err <= bound).all(), name
