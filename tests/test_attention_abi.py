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
                dtype=1, aplan=a.handle, dplan=P, bytes=BIG, ws=None, ws_bytes=0, stream=None)

    def call(**kw):
        return lib.tree_attention(*{**good, **kw}.values())

    assert call() == -1 and b"not an upload" in lib.tree_last_error()
    assert call(bytes=a.device_bytes() - 1) == -5
    for name in ("q", "k", "v", "o", "aplan", "dplan"):
        assert call(**{name: None}) == -1
    assert call(n=229) == -3
    assert call(hq=0) == -1 and call(hkv=0) == -1 and call(d=0) == -1 and call(dtype=2) == -1
    assert call(hq=3) == -4 and call(d=48) == -4 and call(d=256) == -4
    for scale in (0.0, -0.1, NAN, INF, 1e-31, 1e31):
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
    need = lib.tree_attention_backward_workspace_bytes(a.handle, 4, 2, 128, 1)
    assert need >= 230 * 4 * 4
    assert lib.tree_attention_backward_workspace_bytes(None, 4, 2, 128, 1) == 0
    assert lib.tree_attention_backward_workspace_bytes(a.handle, 3, 2, 128, 1) == 0
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


def test_attention_workspace_counts_cut_lists():
    """Lists are cut, and need a workspace, only where whole ones would leave
    the device idle: a long chain with few heads, one list much longer than the
    rest; not a short chain, nor many equal ones."""
    lib = _lib.load()
    fwd, bwd = lib.tree_attention_workspace_bytes, lib.tree_attention_backward_workspace_bytes
    part = (128 * 130 * 4, 128 * 64 * 4, 2 * 128 * 64 * 4)  # o with maxima and sums; dq; dk and dv, of 64-wide heads

    def delta(n, h):
        return (2 * n * h * 4 + 255) // 256 * 256

    assert fwd(None, 4, 64, 1) == 0 and bwd(None, 4, 1, 64, 1) == 0
    many = plan_of([-1] * 600, [128] * 600).attention()
    assert fwd(many.handle, 2, 64, 1) == 0 and bwd(many.handle, 2, 1, 64, 1) == delta(600 * 128, 2)
    short = plan_of([-1], [300]).attention()
    assert fwd(short.handle, 4, 64, 1) == 0 and bwd(short.handle, 1, 1, 64, 1) == delta(300, 1)
    one = plan_of([-1], [2048]).attention()  # 256 positions a part: 2 of the 16 lists are not cut
    f = fwd(one.handle, 1, 64, 1)
    assert f > 0 and f % (128 * 66 * 4) == 0
    assert f // (128 * 66 * 4) == sum(-(-128 * i // 256) for i in range(3, 17))
    b = bwd(one.handle, 8, 1, 64, 1) - delta(2048, 8)
    assert b > 0 and b % part[1] == 0
    assert fwd(one.handle, 1, 64, 0) > f and fwd(one.handle, 1, 64, 2) == 0  # fp32: finer parts
    rc = lib.tree_attention(P, P, P, P2, None, None, 2048, 1, 1, 64, 0.1, 1, one.handle, P, BIG, P, f - 1, None)
    assert rc == -5
    rc = lib.tree_attention(P, P, P, P2, None, None, 2048, 1, 1, 64, 0.1, 1, one.handle, P, BIG, None, BIG, None)
    assert rc == -5
    rc = lib.tree_attention(P, P, P, P2, None, None, 2048, 1, 1, 64, 0.1, 1, one.handle, P, BIG,
                            ctypes.c_void_p(0x1008), BIG, None)
    assert rc == -1 and b"workspace" in lib.tree_last_error()


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
    for t in (0.0, -1.0, NAN, INF, 1e-31, 1e31):
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
