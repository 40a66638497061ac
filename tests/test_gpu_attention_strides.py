"""Tree attention on tensors whose token rows are far apart (time-major storage:
[T, B, heads, d] with a large B), forward and backward: the bits of contiguous
copies, on both sides of a row distance of 2^24 bytes, where the kernels change
how they address a tile."""
import sys

import pytest
import torch

import prefix_tree_packed_plan_amd as ptp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def far_apart(x, row_bytes):
    """A copy of x [N, H, d] whose token rows are row_bytes apart."""
    n, h, d = x.shape
    row = row_bytes // x.element_size()
    y = torch.empty((n - 1) * row + h * d, dtype=x.dtype, device=x.device).as_strided((n, h, d), (row, d, 1))
    y.copy_(x)
    return y


def run(q, k, v, do, plan, o=None, lse=None):
    if o is None:
        o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    return o, lse, *ptp.tree_attention_backward(q, k, v, o, lse, do, plan)


# 260 rows: the third query tile's list holds two whole tiles all of it sees.
TRIES = {"chain": ([-1], [260]), "branches": ([-1, 0, 0, 2], [200, 90, 70, 33])}


@pytest.mark.parametrize("which", ["k", "v", "k and v", "all"])
@pytest.mark.parametrize("row_bytes", [(1 << 24) - 16, 1 << 24, (1 << 24) + 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_token_rows_far_apart(dtype, row_bytes, which):
    for trie, (parents, lens) in TRIES.items():
        n = sum(lens)
        print(f"attention rows {row_bytes} bytes apart: {which}, {trie}, {dtype}", file=sys.stderr, flush=True)
        g = torch.Generator().manual_seed(5)
        q, k, v, do = (torch.randn((n, h, 64), generator=g).to(DT[dtype]).to(DEV) for h in (2, 1, 1, 2))
        plan = ptp.tree_plan(parents, lens, 4)
        want = run(q, k, v, do, plan)
        o = want[0]
        if "k" in which or which == "all":
            k = far_apart(k, row_bytes)
        if "v" in which or which == "all":
            v = far_apart(v, row_bytes)
        if which == "all":
            q, do, o = (far_apart(t, row_bytes) for t in (q, do, o))
        assert torch.equal(ptp.tree_attention(q, k, v, plan), want[0])
        got = run(q, k, v, do, plan, o, want[1])
        assert ptp.tree_attention(q, k, v, plan, return_lse=True)[1].equal(want[1])
        for name, a, b in zip(("dq", "dk", "dv"), got[2:], want[2:]):
            assert torch.equal(a, b), name


@pytest.mark.parametrize("d", [32, 128])
def test_attention_token_rows_far_apart_in_parts(d):
    """Lists long enough to be cut into parts, 16 MiB and more between rows."""
    n = 1100
    print(f"attention rows far apart, parts, d={d}", file=sys.stderr, flush=True)
    g = torch.Generator().manual_seed(6)
    q, k, v, do = (torch.randn((n, h, d), generator=g).to(torch.bfloat16).to(DEV) for h in (2, 1, 1, 2))
    plan = ptp.tree_plan([-1], [n], 4)
    want = run(q, k, v, do, plan)
    k, v = (far_apart(t, (1 << 24) + 64) for t in (k, v))
    got = run(q, k, v, do, plan)
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name
