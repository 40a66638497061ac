"""Argument checks of the embedding entry points that need no device: every
refusal comes before any device work."""
import ctypes

import pytest

from prefix_tree_packed_plan_amd import _lib

P, P2, P3 = (ctypes.c_void_p(0x1000 * i) for i in (1, 2, 3))  # never dereferenced
ODD = ctypes.c_void_p(0x1001)
NAN, INF = float("nan"), float("inf")
MOST = 1 << 30


def test_embedding_refusals_need_no_device():
    lib = _lib.load()
    good = dict(tok=P, table=P2, out=P3, n=5, vocab=10, width=8, tb=8, scale=1.0, dtype=1, stream=None)

    def call(**kw):
        return lib.tree_embedding(*{**good, **kw}.values())

    for name in ("tok", "table", "out"):
        assert call(**{name: None}) == -1 and b"null" in lib.tree_last_error()
    for bad in (dict(n=-1), dict(n=MOST + 1), dict(vocab=0), dict(vocab=-3), dict(vocab=MOST + 1), dict(width=0),
                dict(width=(1 << 24) + 1), dict(tb=2), dict(dtype=2), dict(dtype=-1)):
        assert call(**bad) == -1, bad
    for scale in (0.0, -1.0, NAN, INF, 1e-31, 1e31):
        assert call(scale=scale) == -1 and b"scale" in lib.tree_last_error()
    assert call(out=P2) == -1 and b"alias" in lib.tree_last_error()
    assert call(table=ODD) == -1 and call(out=ODD) == -1 and b"aligned" in lib.tree_last_error()
    assert call(table=ctypes.c_void_p(0x1002), dtype=0) == -1
    assert call(n=0, tok=None, out=None) == 0  # nothing to do


def test_embedding_backward_refusals_need_no_device():
    lib = _lib.load()
    size = lib.tree_embedding_backward_workspace_bytes
    need = size(5, 10, 8)
    assert need >= 4 * (11 + 5)
    assert size(-1, 10, 8) == 0 and size(5, 0, 8) == 0 and size(5, 10, 0) == 0 and size(MOST + 1, 10, 8) == 0
    # Lists of more than 64 tokens are cut: two fp32 rows for every 64 tokens.
    assert size(1000, 10, 8) - size(64, 10, 8) >= 16 * 2 * 8 * 4
    assert size(MOST, 1 << 22, 1 << 24) > (1 << 50)  # no overflow
    assert size(5, (1 << 22) + 1, 8) == 0  # all tokens are looked through for every 512 rows
    good = dict(tok=P, dout=P2, dtable=P3, n=5, vocab=10, width=8, tb=8, scale=1.0, dtype=1, ws=P, bytes=need,
                stream=None)

    def call(**kw):
        return lib.tree_embedding_backward(*{**good, **kw}.values())

    for name in ("tok", "dout", "dtable"):
        assert call(**{name: None}) == -1 and b"null" in lib.tree_last_error()
    for bad in (dict(n=-1), dict(n=MOST + 1), dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(width=0), dict(tb=1),
                dict(dtype=7)):
        assert call(**bad) == -1, bad
    for scale in (0.0, -2.0, NAN, INF, 1e-31, 1e31):
        assert call(scale=scale) == -1
    assert call(ws=None) == -5 and call(bytes=need - 1) == -5
    assert call(ws=ctypes.c_void_p(0x1008)) == -1 and b"workspace" in lib.tree_last_error()
    assert call(dtable=P2) == -1 and call(dout=ODD) == -1 and call(dtable=ODD) == -1
    assert call(n=0, ws=None) == -5  # the table's gradient is zeroed by the same kernels


def test_python_embedding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import prefix_tree_packed_plan_amd as ptp
    tok, x = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ptp.tree_embedding(tok, x)
    with pytest.raises(ValueError, match="device tensor"):
        ptp.tree_embedding_backward(tok, x[:3], 4)
    with pytest.raises(TypeError, match="Tensor"):
        ptp.tree_embedding([0, 1], [[1.0]])
