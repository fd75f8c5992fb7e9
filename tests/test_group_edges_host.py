"""Edges of the operators over rows in order of expert and of the clipping, without a GPU."""
import pytest
import torch

import swiglu_mlp_fwd_amd as S
import swiglu_mlp_fwd_amd.group_ops as ops


# ------------------------------------------------- how a tensor's elements lie

@pytest.mark.parametrize("t,apart", [
    (torch.zeros(5, 7, 8)[:, ::2, :3], True), (torch.zeros(5, 7, 8)[:, ::2, ::3], True), (torch.zeros(4, 9)[:, ::4], True),
    (torch.zeros(20).as_strided((3, 4), (4, 1)), True), (torch.zeros(20).as_strided((3, 4), (3, 1)), False),
    (torch.zeros(20).as_strided((4, 2, 2), (3, 2, 1)), False)])
def test_slices_that_end_inside_a_stride_are_apart(t, apart):
    """The steps behind a dimension's last element are nobody's: strides (56, 16, 1) of 5 x 4 x 3 elements share none."""
    assert ops._apart(t) == apart
    with pytest.raises(ValueError, match="GPU" if apart else "share memory"):
        S.clip_grads([t], 1.0)
