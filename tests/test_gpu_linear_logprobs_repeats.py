"""Log probabilities from hidden states and the output weight, and their gradients,
are the same bits again: in every way that a call is cut, with other values in
between, on another stream, with workspaces full of NaN and from captured graphs,
with and without rows whose log-sum-exp is large."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from prefix_tree_packed_plan_amd import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n,vocab,width", [(1, 300, 72), (33, 32000, 64), (64, 5000, 264), (40, (1 << 20) + 300, 8),
                                           (65, 5000, 264), (1100, 10300, 72), (300, 25000, 2056), (16390, 700, 64)])
def test_the_same_bits(n, vocab, width, dtype):
    print(f"repeats n={n} vocab={vocab} width={width} {dtype}", file=sys.stderr, flush=True)
    dtype = DT[dtype]
    a, b = n // 3, n // 4
    plan = ptp.tree_plan([-1, 0, 0], [a, b, n - a - b], 4) if n > 8 else ptp.tree_plan([-1], [n], 4)

    def inputs(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        h = torch.randn((n, width), generator=g, device=DEV)
        w = torch.randn((vocab, width), generator=g, device=DEV) * (2.0 / width ** 0.5)
        if seed % 2:  # some far rows
            h[::5, 0], w[:, 0] = 2.0 ** 16, 1
        return [h.to(dtype), w.to(dtype), torch.randint(0, vocab, (n,), generator=g, device=DEV),
                torch.randn(n, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV) * 0.1]

    def both(x, ws=(None, None)):
        h, w, tok, dlogp, dent = x
        r = ptp.tree_linear_logprobs(h, w, tok, plan, temperature=0.8, workspace=ws[0])
        return r.logp, r.entropy, r.lse, *ptp.tree_linear_logprobs_backward(
            h, w, tok, r.lse, r.entropy, dlogp, plan, dentropy=dent, temperature=0.8, workspace=ws[1])

    def same(x, y):
        return all(torch.equal(p, q) for p, q in zip(x, y))

    sets = [inputs(i) for i in range(4)]
    want = [both(x) for x in sets]
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for x in want for t in x)
    lib, code = _lib.load(), _lib._dtype_code(sets[0][0])
    ws = [torch.full((f(n, vocab, width, code),), 0xFF, dtype=torch.uint8, device=DEV)
          for f in (lib.tree_linear_logprobs_workspace_bytes, lib.tree_linear_logprobs_backward_workspace_bytes)]
    for x, y in zip(sets, want):
        assert same(both(x, ws), y)
    for i in (3, 0, 2, 1):
        again = [both(sets[j]) for j in (i, (i + 1) % 4, i)]
        assert same(again[0], want[i]) and same(again[1], want[(i + 1) % 4]) and same(again[2], want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [both(x) for x in sets]
    side.synchronize()
    assert all(same(p, q) for p, q in zip(got, want))
    del got, again
    held = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(held)
    for i in (0, 1, 2, 3, 0):
        for p, q in zip(held, sets[i]):
            p.copy_(q)
        for p in out:
            p.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[i]), i
        assert same(both(sets[i]), want[i])
