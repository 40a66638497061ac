"""Tree attention on the GPU, forward and backward, against the fp64 per-path
oracle (oracle/attention.py) with its own error bounds: head layouts, head
sizes, both dtypes, ragged and deep tries, numberings other than depth-first,
slices of one projection, values that are not finite where a token must not
see them, graphs, other streams, determinism."""
import sys

import numpy as np
import pytest
import torch

import prefix_tree_packed_plan_amd as ptp
from oracle.attention import tree_attention_reference
from prefix_tree_packed_plan_amd import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dfs_trie(seed, n_seg, lens):
    """Random depth-first-numbered trie: each segment's parent lies on the path
    of the segment before it."""
    rng = np.random.default_rng(seed)
    parents = [-1]
    for i in range(1, n_seg):
        p = i - 1
        while p >= 0 and rng.random() < 0.4:
            p = parents[p]
        parents.append(p)
    return np.array(parents, np.int32), rng.choice(lens, size=n_seg).astype(np.int32)


def any_trie(seed, n_seg, lens):
    """Random trie numbered with parents first, not depth first."""
    rng = np.random.default_rng(seed)
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, n_seg)]
    return np.array(parents, np.int32), rng.choice(lens, size=n_seg).astype(np.int32)


def tensors(n, hq, hkv, d, dtype, seed=1, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn((n, hq + 2 * hkv, d), generator=g).to(dtype).to(DEV)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((n, h, d), generator=g).to(dtype).to(DEV) for h in (hq, hkv, hkv))
    do = torch.randn((n, hq, d), generator=g).to(dtype).to(DEV)
    return q, k, v, do


def np64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, want):
    value, bound = want
    err = np.abs(np64(got) - value)
    worst = float(np.nanmax(err / bound))
    say(f"  {name}: worst error {float(np.nanmax(err)):.3e}, {worst:.3f} of its bound")
    assert np.all(err <= bound), f"{name}: {worst} times its bound"


def run_case(parents, lens, hq, hkv, d, dtype, seed=1, fused=False, scale=None):
    n = int(sum(lens))
    q, k, v, do = tensors(n, hq, hkv, d, dtype, seed, fused)
    plan = ptp.tree_plan(parents, lens, 4)
    o, lse = ptp.tree_attention(q, k, v, plan, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    say("  forward done")
    dq, dk, dv = ptp.tree_attention_backward(q, k, v, o, lse, do, plan, scale=scale)
    torch.cuda.synchronize()
    ref = tree_attention_reference(parents, lens, np64(q), np64(k), np64(v), d ** -0.5 if scale is None else scale,
                                   do=np64(do), u=U[dtype])
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, t, ref[name])
    return q, k, v, do, plan, o, lse, dq, dk, dv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (6, 1), (3, 3)])
def test_attention_ragged_trie(heads, d, dtype):
    parents, lens = dfs_trie(11, 14, [1, 2, 5, 31, 32, 33, 64, 100])
    say(f"attention ragged heads={heads} d={d} {dtype} N={int(lens.sum())}")
    run_case(parents, lens, *heads, d, DT[dtype])


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 257])
def test_attention_one_segment(n):
    say(f"attention chain N={n}")
    run_case([-1], [n], 2, 1, 64, torch.bfloat16)
    run_case([-1], [n], 2, 1, 64, torch.float32)


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attention_other_numbering(seed):
    """Parents first, but not depth first: branches interleaved in memory."""
    parents, lens = any_trie(20 + seed, 24, [1, 3, 17, 40, 90])
    say(f"attention numbering seed={seed} N={int(lens.sum())}")
    run_case(parents, lens, 4, 2, 64, torch.bfloat16, seed)
    run_case(parents, lens, 2, 2, 32, torch.float32, seed)


def test_attention_deep_trie_of_short_segments():
    """300 segments of 1..3 tokens, a leaf beside every step of a long path."""
    parents, lens, at = [-1], [2], 0
    for i in range(150):
        parents += [at, at]
        lens += [1 + i % 3, 1 + (i + 1) % 2]
        at = len(parents) - 1
    say(f"attention deep N={sum(lens)}")
    run_case(parents, lens, 2, 1, 128, torch.bfloat16)


@pytest.mark.parametrize("case", ["fan", "chain", "mixed"])
def test_attention_lists_cut_into_parts(case):
    """Lists long enough to be spread over work-groups, forward and backward,
    and the query heads of a group spread too; parts some rows see nothing of."""
    parents, lens = {"fan": ([-1] + [0] * 5, [70, 900, 1000, 700, 33, 1]), "chain": ([-1], [2100]),
                     "mixed": ([-1, 0, -1, 2, 2, -1], [1300, 77, 50, 400, 30, 9])}[case]
    say(f"attention parts {case} N={sum(lens)}")
    plan = ptp.tree_plan(parents, lens, 4)
    assert _lib.load().tree_attention_workspace_bytes(plan.attention().handle, 1, 32, 0) > 0
    run_case(parents, lens, 4, 1, 64, torch.bfloat16)
    run_case(parents, lens, 1, 1, 32, torch.float32)
    run_case(parents, lens, 2, 2, 128, torch.bfloat16)


def test_attention_nan_in_a_part():
    """A NaN score makes its row NaN in whichever part of the list it is, and
    no other row."""
    n = 2100
    q, k, v, do = tensors(n, 1, 1, 64, torch.bfloat16)
    plan = ptp.tree_plan([-1], [n], 4)
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    for at in (0, 300, 2099):
        k2 = k.clone()
        k2[at] = float("nan")
        o2, lse2 = ptp.tree_attention(q, k2, v, plan, return_lse=True)
        assert torch.isnan(o2[at:]).all() and torch.isnan(lse2[at:]).all()
        assert torch.equal(o2[:at], o[:at]) and torch.equal(lse2[:at], lse[:at])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_slices_of_one_projection(dtype):
    parents, lens = dfs_trie(5, 9, [3, 40, 77])
    say(f"attention fused {dtype}")
    a = run_case(parents, lens, 4, 2, 64, DT[dtype], fused=True)
    q, k, v, do, plan = a[:5]
    o, lse = ptp.tree_attention(q.contiguous(), k.contiguous(), v.contiguous(), plan, return_lse=True)
    grads = ptp.tree_attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), o, lse, do, plan)
    assert torch.equal(o, a[5]) and torch.equal(lse, a[6])
    assert all(torch.equal(x, y) for x, y in zip(grads, a[7:]))


def test_attention_head_major_and_repeated_tensors():
    """Head-major storage, and k, v repeated over tokens' storage (stride 0):
    the bits of the contiguous tensors."""
    parents, lens = dfs_trie(9, 7, [20, 61])
    n = int(lens.sum())
    say("attention strides")
    q, k, v, do = tensors(n, 4, 2, 64, torch.bfloat16)
    plan = ptp.tree_plan(parents, lens, 4)
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    grads = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    q2, k2, v2, o2, do2 = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, o, do))
    assert not q2.is_contiguous()
    o3, lse3 = ptp.tree_attention(q2, k2, v2, plan, return_lse=True)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
    assert all(torch.equal(x, y) for x, y in zip(grads, ptp.tree_attention_backward(q2, k2, v2, o2, lse, do2, plan)))
    one = k[:1].expand(n, 2, 64)
    same = ptp.tree_attention(q, one, one, plan)
    assert torch.equal(same, ptp.tree_attention(q, one.contiguous(), one.contiguous(), plan))
    assert torch.equal(same.view(n, 2, 2, 64), one[:, :, None].expand(n, 2, 2, 64))


def test_attention_scale_and_large_scores():
    """Scores of several hundred: the running maximum moves far and often."""
    parents, lens = dfs_trie(8, 8, [50, 130, 70])
    say("attention large scores")
    run_case(parents, lens, 2, 1, 64, torch.float32, scale=4.0)
    run_case(parents, lens, 2, 1, 64, torch.bfloat16, scale=0.02)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_attention_unseen_values_that_are_not_finite(bad, dtype):
    """q, k, v and dO of one branch hold `bad`: every other branch and the
    prefix are bitwise what they are with ordinary values there, forward and
    (dq) backward, and dk, dv of every other branch."""
    parents, lens = [-1, 0, 0, 0, 2], [40, 30, 21, 50, 13]
    off = np.concatenate([[0], np.cumsum(lens)])
    n, hq, hkv, d = int(off[-1]), 4, 2, 64
    q, k, v, do = tensors(n, hq, hkv, d, DT[dtype])
    plan = ptp.tree_plan(parents, lens, 4)
    say(f"attention bad values {bad} {dtype}")
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    dq, dk, dv = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    rows = torch.arange(int(off[2]) + 5, int(off[3]), device=DEV)  # the tail of segment 2
    below = torch.arange(int(off[4]), n, device=DEV)               # its child
    hit = torch.zeros(n, dtype=torch.bool, device=DEV)
    hit[rows] = True
    hit[below] = True
    q2, k2, v2, do2 = (t.clone() for t in (q, k, v, do))
    for t in (q2, k2, v2, do2):
        t[rows, :, ::3] = bad
    o2, lse2 = ptp.tree_attention(q2, k2, v2, plan, return_lse=True)
    dq2, dk2, dv2 = ptp.tree_attention_backward(q2, k2, v2, o2, lse2, do2, plan)
    torch.cuda.synchronize()
    other = torch.zeros(n, dtype=torch.bool, device=DEV)  # neither the branch nor what it sees
    for s in (1, 3):
        other[int(off[s]):int(off[s + 1])] = True
    assert torch.equal(o[~hit], o2[~hit]) and torch.equal(lse[~hit], lse2[~hit])
    assert torch.equal(dq[~hit], dq2[~hit])
    assert torch.equal(dk[other], dk2[other]) and torch.equal(dv[other], dv2[other])
    assert not torch.isfinite(o2[rows].float()).all(-1).any()
    # What those tokens see is not hidden from them.
    want = tree_attention_reference(parents, lens, np64(q), np64(k), np64(v), d ** -0.5)
    check("o of the other rows", o2[~hit], tuple(x[(~hit).cpu().numpy()] for x in want["o"]))


def test_attention_infinite_value_reaches_those_that_see_it():
    """v = +inf in one column of one token: +inf there for the tokens that see
    it, untouched values elsewhere."""
    parents, lens = [-1, 0, 0], [20, 30, 30]
    q, k, v, _ = tensors(80, 2, 1, 32, torch.bfloat16)
    plan = ptp.tree_plan(parents, lens, 4)
    o = ptp.tree_attention(q, k, v, plan)
    v2 = v.clone()
    v2[25, 0, 7] = float("inf")
    o2 = ptp.tree_attention(q, k, v2, plan)
    sees = torch.zeros(80, dtype=torch.bool, device=DEV)
    sees[25:50] = True
    assert torch.isinf(o2[sees][:, :, 7].float()).all()
    keep = torch.ones(32, dtype=torch.bool, device=DEV)
    keep[7] = False
    assert torch.equal(o2[:, :, keep], o[:, :, keep])
    assert torch.equal(o2[~sees], o[~sees])


def test_attention_is_deterministic_and_follows_the_stream():
    parents, lens = dfs_trie(4, 12, [64, 200, 333])
    a = run_case(parents, lens, 4, 2, 128, torch.bfloat16)
    q, k, v, do, plan = a[:5]
    for i in range(3):
        say(f"attention again {i}")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
            grads = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, a[5]) and torch.equal(lse, a[6])
        assert all(torch.equal(x, y) for x, y in zip(grads, a[7:]))


def test_attention_in_a_graph():
    """Forward and backward captured once, replayed on new inputs."""
    parents, lens = dfs_trie(6, 10, [30, 150])
    n = int(lens.sum())
    plan = ptp.tree_plan(parents, lens, 4)
    q, k, v, do = tensors(n, 4, 2, 64, torch.bfloat16)
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, glse = ptp.tree_attention(q, k, v, plan, return_lse=True)
        gg = ptp.tree_attention_backward(q, k, v, go, glse, do, plan)
    for i in range(4):
        say(f"attention replay {i}")
        for t, s in zip((q, k, v, do), tensors(n, 4, 2, 64, torch.bfloat16, seed=50 + i)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
        want = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
        torch.cuda.synchronize()
        assert torch.equal(o, go) and torch.equal(lse, glse)
        assert all(torch.equal(x, y) for x, y in zip(gg, want))


def test_attention_tokens_equal_their_own_path():
    """Eq. 6 directly: every leaf's path run alone gives the same outputs and,
    summed over the leaves (each with its share of dO), the same gradients to
    the rounding of the stored values."""
    parents, lens = [-1, 0, 0, 1, 1], [60, 40, 70, 33, 21]
    off = np.concatenate([[0], np.cumsum(lens)])
    n = int(off[-1])
    q, k, v, _ = tensors(n, 2, 1, 64, torch.float32)
    plan = ptp.tree_plan(parents, lens, 4)
    o = ptp.tree_attention(q, k, v, plan)
    ref = tree_attention_reference(parents, lens, np64(q), np64(k), np64(v), 64 ** -0.5, u=U[torch.float32])
    for leaf in (2, 3, 4):
        segs, s = [], leaf
        while s >= 0:
            segs.insert(0, s)
            s = parents[s]
        rows = torch.cat([torch.arange(int(off[s]), int(off[s + 1]), device=DEV) for s in segs])
        alone = ptp.tree_attention(q[rows].contiguous(), k[rows].contiguous(), v[rows].contiguous(),
                                   ptp.tree_plan([-1], [len(rows)], 4))
        bound = 2 * ref["o"][1][rows.cpu().numpy()]
        assert np.all(np.abs(np64(alone) - np64(o[rows])) <= bound)


def test_attention_rl_batch_beyond_32_bit_offsets():
    """The RL batch trie (428,843 tokens), q, k, v cut from one 5.3 GB
    projection: the last completion's outputs and gradients against the oracle
    on its path alone (a leaf's dk, dv come from its own rows only); every value
    finite."""
    from workloads import make_trie
    parents, lens, _ = make_trie(5)
    off = np.concatenate([[0], np.cumsum(lens)])
    n, hq, hkv, d = int(off[-1]), 32, 8, 128
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    qkv = torch.empty((n, hq + 2 * hkv, d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    do = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    assert qkv.numel() * 2 > 1 << 32
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    say(f"attention rl_batch N={n}")
    plan = ptp.tree_plan(parents, lens, 4)
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    torch.cuda.synchronize()
    say("  forward done")
    dq, dk, dv = ptp.tree_attention_backward(q, k, v, o, lse, do, plan)
    torch.cuda.synchronize()
    for t in (o, lse, dq, dk, dv):
        assert torch.isfinite(t).all()
    leaf = len(lens) - 1
    path, s = [], leaf
    while s >= 0:
        path.insert(0, s)
        s = int(parents[s])
    rows = torch.cat([torch.arange(int(off[s]), int(off[s + 1]), device=DEV) for s in path])
    m = int(lens[leaf])
    for hk in (0, 7):
        h = slice(4 * hk, 4 * hk + 2)  # two query heads of the group: dq, o; dk, dv need all four
        ref = tree_attention_reference([-1], [len(rows)], np64(q[rows, h]), np64(k[rows, hk:hk + 1]),
                                       np64(v[rows, hk:hk + 1]), d ** -0.5, do=np64(do[rows, h]))
        for name, t in (("o", o), ("lse", lse), ("dq", dq)):
            check(name, t[rows[-m:], h], tuple(x[-m:] for x in ref[name]))
    own = rows[-m:]
    grads = [np.zeros((m, d)) for _ in range(4)]
    for h in range(28, 32):
        ref = tree_attention_reference([-1], [len(rows)], np64(q[rows, h:h + 1]), np64(k[rows, 7:8]),
                                       np64(v[rows, 7:8]), d ** -0.5, do=np64(do[rows, h:h + 1]))
        for i, name in enumerate(("dk", "dv")):
            grads[i] += ref[name][0][-m:, 0]
            grads[2 + i] += ref[name][1][-m:, 0]
    check("dk", dk[own, 7], (grads[0], grads[2]))
    check("dv", dv[own, 7], (grads[1], grads[3]))


def test_attention_refusals():
    """Misuse raises on the host; nothing is launched."""
    parents, lens = [-1, 0], [20, 12]
    plan = ptp.tree_plan(parents, lens, 4)
    q, k, v, do = tensors(32, 4, 2, 64, torch.bfloat16)
    o, lse = ptp.tree_attention(q, k, v, plan, return_lse=True)
    with pytest.raises(ValueError):
        ptp.tree_attention(q[:31], k[:31], v[:31], plan)
    with pytest.raises(ValueError):
        ptp.tree_attention(q, k, v[:, :1], plan)
    with pytest.raises(ValueError):
        ptp.tree_attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, plan)  # a head's elements apart
    with pytest.raises(TypeError):
        ptp.tree_attention(q, k.float(), v, plan)
    with pytest.raises(TypeError):
        ptp.tree_attention(q.half(), k.half(), v.half(), plan)
    with pytest.raises(_lib.TreeError, match="multiple of h_kv"):
        ptp.tree_attention(q[:, :3].contiguous(), k, v, plan)
    with pytest.raises(_lib.TreeError, match="not compiled in"):
        ptp.tree_attention(q[:, :, :48].contiguous(), k[:, :, :48].contiguous(), v[:, :, :48].contiguous(), plan)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(_lib.TreeError, match="scale"):
            ptp.tree_attention(q, k, v, plan, scale=scale)
    with pytest.raises(_lib.TreeError, match="alias"):
        ptp.tree_attention(q, k, v, plan, out=q)
    wide = torch.zeros(32, 4 * 64 + 4, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(_lib.TreeError, match="16 bytes"):
        ptp.tree_attention(wide[:, 4:].unflatten(1, (4, 64)), k, v, plan)
    with pytest.raises(ValueError, match="workspace"):
        ptp.tree_attention_backward(q, k, v, o, lse, do, plan,
                                    workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        ptp.tree_attention_backward(q, k, v, o, lse.bfloat16(), do, plan)
    # A device copy that was not made from this trie's tables.
    lib, a = _lib.load(), plan.attention()
    other = ptp.tree_plan([-1], [32], 4).attention()
    stale = other.on_device(DEV)
    out = torch.empty_like(q)
    big = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    for buf in (big, stale):
        rc = lib.tree_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None, None, 32, 4, 2,
                                64, 0.125, 1, a.handle, buf.data_ptr(), max(buf.numel(), a.device_bytes()), None, 0,
                                None)
        assert rc == -1 and b"not an upload" in lib.tree_last_error()
