"""The attention's workspace sizes for arguments that its calls refuse: 0."""
import numpy as np
import pytest

from prefix_tree_packed_plan_amd import _lib


@pytest.mark.parametrize("d,dtype", [(48, 0), (48, 1), (256, 1), (0, 1), (-64, 0), (1 << 20, 0), (64, 2), (64, -1)])
def test_no_workspace_for_sizes_that_are_refused(d, dtype):
    lib = _lib.load()
    a = _lib.TreePlan(np.array([-1], np.int32), np.array([2048], np.int32), 4).attention()
    assert lib.tree_attention_workspace_bytes(a.handle, 1, 64, 0) > 0
    assert lib.tree_attention_workspace_bytes(a.handle, 1, d, dtype) == 0
    assert lib.tree_attention_backward_workspace_bytes(a.handle, 1, 1, d, dtype) == 0


@pytest.mark.parametrize("heads", [0, -1, 65536, 1 << 30])
def test_no_workspace_for_heads_that_are_refused(heads):
    lib = _lib.load()
    a = _lib.TreePlan(np.array([-1], np.int32), np.array([2048], np.int32), 4).attention()
    for dtype in (0, 1):
        assert lib.tree_attention_workspace_bytes(a.handle, heads, 64, dtype) == 0
        assert lib.tree_attention_backward_workspace_bytes(a.handle, heads, 1, 64, dtype) == 0
        assert lib.tree_attention_backward_workspace_bytes(a.handle, 4, heads, 64, dtype) == 0
