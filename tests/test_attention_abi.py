"""Argument checks of the attention and log probability entry points that need
no device: every refusal comes before any device work."""
import ctypes

import numpy as np
import pytest

from prefix_tree_packed_plan_amd import _lib

P, P2, P3, P4 = (ctypes.c_void_p(0x1000 * i) for i in (1, 2, 3, 4))  # never dereferenced
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def strides(x):
    return ctypes.cast((ctypes.c_int64 * len(x))(*x), ctypes.c_void_p)


def plan_of(parents=(-1, 0, 0), lens=(100, 60, 70)):
    return _lib.TreePlan(np.array(parents, np.int32), np.array(lens, np.int32), 4)


def test_attention_plan_is_built_on_the_host():
    plan = plan_of()
    a = plan.attention()
    assert a is plan.attention()
    lib = _lib.load()
    assert a.device_bytes() >= 2 * 230 * 4
    h = ctypes.c_void_p()
    assert lib.tree_attention_plan(None, ctypes.byref(h)) == -1
    assert lib.tree_attention_plan(plan.handle, None) == -1
    assert lib.tree_attention_plan_device_bytes(None) == 0
    lib.tree_attention_plan_free(None)
    assert lib.tree_attention_plan_upload(a.handle, None, BIG, None) == -1
    assert lib.tree_attention_plan_upload(a.handle, P, a.device_bytes() - 1, None) == -5
    assert lib.tree_attention_plan_upload(a.handle, ctypes.c_void_p(0x1010), BIG, None) == -1


def test_attention_refusals_need_no_device():
    a = plan_of().attention()
    lib = _lib.load()
    good = dict(q=P, k=P, v=P, o=P2, lse=None, st=None, n=230, hq=4, hkv=2, d=128, scale=0.1,
                dtype=1, aplan=a.handle, dplan=P, bytes=BIG, stream=None)

    def call(**kw):
        return lib.tree_attention(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    assert call(bytes=a.device_bytes() - 1) == -5
    for name in ("q", "k", "v", "o", "aplan", "dplan"):
        assert call(**{name: None}) == -1
    assert call(n=229) == -3
    assert call(hq=0) == -1 and call(hkv=0) == -1 and call(d=0) == -1 and call(dtype=2) == -1
    assert call(hq=3) == -4 and call(d=48) == -4 and call(d=256) == -4
    for scale in (0.0, -0.1, NAN, INF):
        assert call(scale=scale) == -1
    ok = [512, 128, 256, 128, 256, 128]
    assert call(st=strides(ok)) == -1 and b"not an upload" in lib.tree_last_error()
    for i in range(6):  # negative, not on 16 bytes, absurd
        for x in (-512, ok[i] + 4, 1 << 50):
            assert call(st=strides(ok[:i] + [x] + ok[i + 1:])) == -1
            assert b"of q" in lib.tree_last_error() or b"not aligned" in lib.tree_last_error() or \
                b"bad strides" in lib.tree_last_error()
    assert call(q=ctypes.c_void_p(0x1008)) == -1 and call(o=ctypes.c_void_p(0x2004)) == -1
    assert call(o=P) == -1


def test_attention_backward_refusals_need_no_device():
    a = plan_of().attention()
    lib = _lib.load()
    need = lib.tree_attention_backward_workspace_bytes(a.handle, 4, 2, 128)
    assert need >= 230 * 4 * 4
    assert lib.tree_attention_backward_workspace_bytes(None, 4, 2, 128) == 0
    assert lib.tree_attention_backward_workspace_bytes(a.handle, 3, 2, 128) == 0
    good = dict(q=P, k=P, v=P, o=P, lse=P, do=P, dq=P2, dk=P3, dv=P4, st=None, n=230, hq=4, hkv=2, d=128, scale=0.1, dtype=1, aplan=a.handle, dplan=P, bytes=BIG, ws=P, ws_bytes=need,
                stream=None)

    def call(**kw):
        return lib.tree_attention_backward(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    for name in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv", "aplan", "dplan"):
        assert call(**{name: None}) == -1
    assert call(ws=None) == -5 and call(ws_bytes=need - 1) == -5
    assert call(n=231) == -3 and call(hq=5) == -4 and call(d=96) == -4 and call(scale=0.0) == -1
    ok = [512, 128, 256, 128, 256, 128, 512, 128, 128, 230 * 128]
    assert call(st=strides(ok)) == -1 and b"not an upload" in lib.tree_last_error()
    for i in range(10):
        assert call(st=strides(ok[:i] + [ok[i] + 1] + ok[i + 1:])) == -1 and b"not aligned" in lib.tree_last_error()
    assert call(dk=ctypes.c_void_p(0x3008)) == -1 and call(ws=ctypes.c_void_p(0x1008)) == -1
    assert call(dq=P) == -1 and call(dk=P2) == -1 and call(dv=P3) == -1


def test_attention_workspace_counts_split_work():
    """One part per key tile and heads enough: only delta; few tiles: partial
    sums for every head of the group; more than 2048 rows below a key tile:
    partial sums for its parts."""
    lib = _lib.load()
    many = plan_of([-1] * 600, [128] * 600).attention()
    assert lib.tree_attention_backward_workspace_bytes(many.handle, 2, 1, 64) == 2 * 600 * 128 * 2 * 4
    few = plan_of([-1], [128]).attention()
    assert lib.tree_attention_backward_workspace_bytes(few.handle, 4, 1, 64) == 2 * 128 * 4 * 4 + 4 * 2 * 128 * 64 * 4
    part = plan_of([-1] + [-1] * 600, [4096] + [128] * 600).attention()  # tiles 0..15 have two parts
    delta = 2 * (4096 + 600 * 128) * 4
    assert lib.tree_attention_backward_workspace_bytes(part.handle, 1, 1, 64) == delta + 32 * 2 * 128 * 64 * 4


def test_logprobs_refusals_need_no_device():
    plan = plan_of()
    lib = _lib.load()
    need = lib.tree_logprobs_workspace_bytes(230, 5000, 8)
    assert need > 0 and lib.tree_logprobs_workspace_bytes(512, 5000, 8) == 0
    assert lib.tree_logprobs_workspace_bytes(0, 5000, 8) == 0 and lib.tree_logprobs_workspace_bytes(230, 5000, 65) == 0
    good = dict(x=P, tok=P, logp=P, ent=P, lse=P, tl=P, ti=P, ld=5000, n=230, first=0, rows=230, vocab=5000, tb=8,
                temp=1.0, k=8, dtype=1, plan=plan.handle, dplan=P, bytes=BIG, ws=P, ws_bytes=need, stream=None)

    def call(**kw):
        return lib.tree_logprobs(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    for name in ("x", "tok", "logp", "ent", "lse", "tl", "ti", "plan", "dplan"):
        assert call(**{name: None}) == -1
    assert call(n=229) == -3
    assert call(first=-1) == -1 and call(first=1) == -1 and call(rows=0) == -1 and call(rows=231) == -1
    assert call(vocab=0) == -1 and call(ld=4999) == -1 and call(tb=2) == -1 and call(dtype=7) == -1
    for t in (0.0, -1.0, NAN, INF):
        assert call(temp=t) == -1
    assert call(k=-1) == -1 and call(k=65) == -1 and call(vocab=4, ld=4, k=5) == -1
    assert call(ws=None) == -5 and call(ws_bytes=need - 1) == -5 and call(bytes=8) == -5

    good = dict(x=P, tok=P, lse=P, ent=P, dlogp=P, dent=P, dx=P, ld=5000, ldd=5000, n=230, first=0, rows=230,
                vocab=5000, tb=8, temp=1.0, dtype=1, plan=plan.handle, dplan=P, bytes=BIG, stream=None)

    def back(**kw):
        return lib.tree_logprobs_backward(*{**good, **kw}.values())

    assert back() == -1 and b"not an upload" in lib.tree_last_error()
    for name in ("x", "tok", "lse", "ent", "dlogp", "dx", "plan", "dplan"):
        assert back(**{name: None}) == -1
    assert back(dent=None, ent=None) == -1 and b"not an upload" in lib.tree_last_error()
    assert back(n=1) == -3 and back(ldd=5001) == -1 and back(ldd=4000) == -1 and back(rows=300) == -1
    assert back(temp=0.0) == -1 and back(bytes=8) == -5


def test_python_entry_points_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import prefix_tree_packed_plan_amd as ptp
    plan = plan_of()
    q = torch.zeros(230, 2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        ptp.tree_attention(q, q, q, plan)
    with pytest.raises(ValueError, match="device tensor"):
        ptp.tree_logprobs(torch.zeros(230, 8), torch.zeros(230, dtype=torch.int64), plan)
