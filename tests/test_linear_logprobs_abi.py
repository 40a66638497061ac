"""Argument checks of the hidden-state log probability entry points that need no
device, and what their workspaces count."""
import ctypes

import numpy as np

from prefix_tree_packed_plan_amd import _lib

P, P2, P3 = (ctypes.c_void_p(0x1000 * i) for i in (1, 2, 3))  # never dereferenced
ODD = ctypes.c_void_p(0x1008)
BIG = 1 << 50
NAN, INF = float("nan"), float("inf")


def plan_of(parents=(-1, 0, 0), lens=(100, 60, 70)):
    return _lib.TreePlan(np.array(parents, np.int32), np.array(lens, np.int32), 4)


def test_refusals_need_no_device():
    plan, lib = plan_of(), _lib.load()
    need = lib.tree_linear_logprobs_workspace_bytes(230, 5000, 64, 1)
    assert need > 0
    good = dict(h=P, w=P2, tok=P, logp=P, ent=P, lse=P, ld=64, n=230, first=0, rows=230, vocab=5000, width=64, tb=8,
                temp=1.0, dtype=1, plan=plan.handle, dplan=P, bytes=BIG, ws=P, ws_bytes=need, stream=None)

    def call(**kw):
        return lib.tree_linear_logprobs(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    for name in ("h", "w", "tok", "logp", "ent", "lse", "plan", "dplan"):
        assert call(**{name: None}) == -1 and b"null" in lib.tree_last_error()
    assert call(n=229) == -3
    for bad in (dict(first=-1), dict(first=1), dict(rows=0), dict(rows=231), dict(vocab=0), dict(ld=63), dict(ld=68),
                dict(ld=(1 << 20) + 8), dict(tb=3), dict(dtype=2), dict(width=0), dict(h=ODD), dict(w=ODD), dict(ws=ODD)):
        assert call(**bad) == -1, bad
    for bad in (dict(width=60), dict(width=4), dict(vocab=(1 << 22) + 1), dict(width=65544, ld=65544)):
        assert call(**bad) == -4, bad
    assert call(width=60, ld=60, dtype=0) == -1 and b"not an upload" in lib.tree_last_error()  # 4 fp32 are 16 bytes
    assert call(width=62, ld=64, dtype=0) == -4
    for t in (0.0, -1.0, NAN, INF, 1e-31, 1e31):
        assert call(temp=t) == -1 and b"temperature" in lib.tree_last_error()
    assert call(ws=None) == -5 and call(ws_bytes=need - 1) == -5 and call(bytes=8) == -5


def test_backward_refusals_need_no_device():
    plan, lib = plan_of(), _lib.load()
    need = lib.tree_linear_logprobs_backward_workspace_bytes(230, 5000, 64, 1)
    assert need >= 256 * 5000 * 2
    good = dict(h=P, w=P, tok=P, lse=P, ent=P, dlogp=P, dent=P, dh=P2, dw=P3, ld=64, n=230, first=0, rows=230,
                vocab=5000, width=64, tb=8, temp=1.0, dtype=1, plan=plan.handle, dplan=P, bytes=BIG, ws=P,
                ws_bytes=need, stream=None)

    def call(**kw):
        return lib.tree_linear_logprobs_backward(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    assert call(dent=None, ent=None) == -1 and b"not an upload" in lib.tree_last_error()
    for name in ("h", "w", "tok", "lse", "ent", "dlogp", "dh", "dw", "plan", "dplan"):
        assert call(**{name: None}) == -1 and b"null" in lib.tree_last_error()
    assert call(n=1) == -3 and call(rows=300) == -1 and call(width=63, ld=64) == -4 and call(temp=0.0) == -1
    assert call(ws=None) == -5 and call(ws_bytes=need - 1) == -5 and call(bytes=8) == -5
    assert call(dh=ODD) == -1 and call(dw=ODD) == -1
    assert call(dh=P) == -1 and call(dw=P) == -1 and call(dw=P2) == -1 and b"alias" in lib.tree_last_error()


def test_workspaces_are_bounded():
    """Neither grows with rows x vocabulary: that is what keeping no logits is for."""
    lib = _lib.load()
    fwd, bwd = lib.tree_linear_logprobs_workspace_bytes, lib.tree_linear_logprobs_backward_workspace_bytes
    for f in (fwd, bwd):
        assert f(0, 5000, 64, 1) == 0 and f(5, 0, 64, 1) == 0 and f(5, 5000, 60, 1) == 0 and f(5, 5000, 64, 5) == 0
        assert f(5, (1 << 22) + 1, 64, 1) == 0 and f(5, 5000, 65544, 1) == 0
    for rows in (428843, 2 ** 31 - 1):
        assert fwd(rows, 131072, 4096, 1) <= 1 << 30
        # D, the weight's gradient and one of the rows at a time in fp32, and no more.
        assert bwd(rows, 131072, 4096, 1) <= (2 << 28) + 131072 * 4096 * 4 + 16384 * 4096 * 4 + (1 << 21)
    assert fwd(428843, 1 << 22, 65536, 0) <= (1 << 30) + 256 * 32768 * 16
    assert bwd(8192, 131072, 4096, 1) < bwd(428843, 131072, 4096, 1)
