"""The root-mean-square error of the attention oracle, pinned on the CPU:
arithmetic that rounds its operands to bf16 passes at twice its size, and
gradients with a lost tile, a lost part or a wrong delta do not."""
import numpy as np
import pytest
import torch

from oracle.attention import rms_ratio, tree_attention_reference, tree_attention_rms

MOST = 2.0  # roundings average u / sqrt(3) at most: 1 is expected at most, 64 rows of one head vary by some 20%


def bf16(x):
    return torch.tensor(x).to(torch.bfloat16).double().numpy()


def case(parents, lens, hq, hkv, d, seed):
    n = int(sum(lens))
    rng = np.random.default_rng(seed)
    q, k, v, do = (bf16(rng.standard_normal((n, h, d))) for h in (hq, hkv, hkv, hq))
    ref = {x: y[0] for x, y in tree_attention_reference(parents, lens, q, k, v, d ** -0.5, do=do).items()}
    return q, k, v, do, ref, tree_attention_rms(parents, lens, q, k, v, d ** -0.5, do)


def gradients(q, k, v, do, scale, rounded=lambda x: x, delta=1.0, keep=None):
    """One chain; `keep` [N, N] pairs that take part in dk."""
    n, hq, d = q.shape
    grp = hq // k.shape[1]
    out = {"o": np.zeros_like(q), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    for h in range(hq):
        kk, vv, qq, dd = k[:, h // grp], v[:, h // grp], q[:, h], do[:, h]
        w = np.where(np.tri(n, dtype=bool), qq @ kk.T * scale, -np.inf)
        e = np.exp(w - w.max(1, keepdims=True))
        z = e.sum(1, keepdims=True)
        o = rounded(rounded(e) @ vv / z)
        p = e / z
        ds = rounded(p * (dd @ vv.T - delta * (dd * o).sum(1, keepdims=True)))
        p = rounded(p)
        out["o"][:, h], out["dq"][:, h] = o, rounded(scale * ds @ kk)
        if keep is not None:
            p, ds = p * keep, ds * keep
        out["dk"][:, h // grp] += scale * ds.T @ qq
        out["dv"][:, h // grp] += p.T @ dd
    out["dk"], out["dv"] = rounded(out["dk"]), rounded(out["dv"])
    return out


@pytest.mark.parametrize("heads,n,d", [((1, 1), 700, 64), ((4, 1), 300, 32), ((1, 1), 130, 128)])
def test_bf16_operands_pass(heads, n, d):
    q, k, v, do, ref, rms = case([-1], [n], *heads, d, 1)
    got = gradients(q, k, v, do, d ** -0.5, bf16)
    for x in rms:
        ratio = rms_ratio(got[x] - ref[x], rms[x])
        print(x, ratio)
        assert 0.2 < ratio <= MOST, x


def test_the_roundings_of_a_trie_are_those_of_its_paths():
    """Every row's o and dq, and a leaf's dk and dv, as on its path alone."""
    parents, lens = [-1, 0, 0], [20, 15, 9]
    q, k, v, do, _, rms = case(parents, lens, 2, 1, 32, 2)
    rows = np.r_[0:20, 35:44]
    alone = tree_attention_rms([-1], [29], q[rows], k[rows], v[rows], 32 ** -0.5, do[rows])
    for x in ("o", "dq"):
        np.testing.assert_allclose(rms[x][rows], alone[x], rtol=1e-9)
    for x in ("dk", "dv"):
        np.testing.assert_allclose(rms[x][35:], alone[x][20:], rtol=1e-9)


def test_lost_tiles_do_not_pass():
    """A 64 x 64 tile of pairs lost at the far end of a 2100-token list, and 32
    keys without the last query tile."""
    n, d = 2100, 64
    q, k, v, do, ref, rms = case([-1], [n], 1, 1, d, 3)
    for rows, keys in ((slice(n - 64, n), slice(0, 64)), (slice(n - 52, n), slice(320, 352))):
        keep = np.ones((n, n))
        keep[rows, keys] = 0
        got = gradients(q, k, v, do, d ** -0.5, keep=keep)
        for x in ("dk", "dv"):
            ratio = rms_ratio(got[x] - ref[x], rms[x])
            print(x, ratio)
            assert ratio > MOST, x


def test_a_wrong_delta_does_not_pass():
    n, d = 300, 64
    q, k, v, do, ref, rms = case([-1], [n], 1, 1, d, 4)
    got = gradients(q, k, v, do, d ** -0.5, delta=0.9)
    for x in ("dq", "dk"):
        ratio = rms_ratio(got[x] - ref[x], rms[x])
        print(x, ratio)
        assert ratio > MOST, x
