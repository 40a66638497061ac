"""Tree attention on lists long enough to be cut into parts and joined: bf16
against the mean size of its roundings (a lost tile or part shows), fp32 with
heads of 128 against the oracle's bounds, and values that are not finite in
tiles that every row of a part sees."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.attention import rms_ratio, tree_attention_reference, tree_attention_rms
from prefix_tree_packed_plan_amd import _lib
from tests.test_gpu_attention import DEV, DT, np64, run_case, tensors

pytestmark = pytest.mark.gpu

TRIES = {"fan": ([-1] + [0] * 5, [70, 900, 1000, 700, 33, 1]), "chain": ([-1], [2100]),
         "mixed": ([-1, 0, -1, 2, 2, -1], [1300, 77, 50, 400, 30, 9]),
         # Parents first, but not depth first.
         "turns": ([-1, -1, 0, 1, 0, 1, 2, 3], [300, 350, 200, 270, 90, 400, 60, 33])}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def parts(plan, hq, hkv, d, dtype):
    """Bytes of parts in the forward's workspace, and in the backward's beyond
    its statistics."""
    lib, a, code = _lib.load(), plan.attention().handle, 1 if dtype == torch.bfloat16 else 0
    stats = (2 * plan.n_tokens * hq * 4 + 255) // 256 * 256
    return (lib.tree_attention_workspace_bytes(a, hq, d, code),
            lib.tree_attention_backward_workspace_bytes(a, hq, hkv, d, code) - stats)


@pytest.mark.parametrize("heads,d", [((1, 1), 64), ((4, 1), 64), ((2, 2), 128), ((2, 1), 32)])
@pytest.mark.parametrize("trie", sorted(TRIES))
def test_bf16_errors_are_those_of_its_roundings(trie, heads, d):
    """Each 64 rows of a head, root mean square: at most twice what independent
    roundings of the operands give."""
    parents, lens = TRIES[trie]
    say(f"attention long {trie} heads={heads} d={d}")
    q, k, v, do = tensors(sum(lens), *heads, d, torch.bfloat16)
    plan = ptp.tree_plan(parents, lens, 4)
    assert min(parts(plan, *heads, d, torch.bfloat16)) > 0
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    dq, dk, dv = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    torch.cuda.synchronize()
    args = parents, lens, np64(q), np64(k), np64(v), d ** -0.5
    ref, rms = tree_attention_reference(*args, do=np64(do)), tree_attention_rms(*args, np64(do))
    for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        ratio = rms_ratio(np64(t) - ref[name][0], rms[name])
        say(f"  {name}: {ratio:.3f} of the roundings' root mean square")
        assert ratio <= 2, name


@pytest.mark.parametrize("heads", [(1, 1), (2, 1)])
@pytest.mark.parametrize("trie", ["chain", "fan"])
def test_fp32_heads_of_128(trie, heads):
    parents, lens = TRIES[trie]
    say(f"attention long fp32 d=128 {trie} heads={heads}")
    assert min(parts(ptp.tree_plan(parents, lens, 4), *heads, 128, torch.float32)) > 0
    run_case(parents, lens, *heads, 128, torch.float32)


@pytest.mark.parametrize("at", [0, 130, 500])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_key_that_is_not_finite_in_parts(dtype, at):
    """A NaN key of one branch, `at` tokens into it, in tiles that later rows
    see whole: dq of the rows that see it, dk and dv of the tokens those rows
    see are NaN, the other branch keeps its bits."""
    lens = [400, 1500, 700]
    plan = ptp.tree_plan([-1, 0, 0], lens, 4)
    n, d = sum(lens), 64
    say(f"attention NaN key in parts {dtype} at {at}")
    assert min(parts(plan, 2, 1, d, DT[dtype])) > 0
    q, k, v, do = tensors(n, 2, 1, d, DT[dtype])
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    good = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    k2 = k.clone()
    k2[400 + at, 0, 3] = float("nan")
    o2, lse2 = ptp.tree_attention(q, k2, v, plan, return_lse=True)
    bad = ptp.tree_attention_backward(q, k2, v, o2, lse2, do, plan)
    torch.cuda.synchronize()
    sees = torch.zeros(n, dtype=torch.bool, device=DEV)
    sees[400 + at:1900] = True
    seen = torch.zeros_like(sees)
    seen[:1900] = True
    assert torch.isnan(o2[sees]).all() and torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2[~sees], lse[~sees])
    assert torch.isnan(bad[0][sees]).all() and torch.equal(bad[0][~sees], good[0][~sees])
    for a, b in zip(bad[1:], good[1:]):
        assert torch.isnan(a[seen]).all() and torch.equal(a[~seen], b[~seen])
    assert np.isfinite(np64(good[0])).all()
