"""Edges of the operators over rows in order of expert and of the clipping, on the GPU: the tiles that large calls take,
the path of tokens past 32-bit offsets, what a row's result depends on, limits and layouts of clipped gradients.

Bounds as in test_gpu_group.py.
"""
import math

import numpy as np
import pytest
import torch

from oracle import group_oracle as G
from parity_util import U32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import swiglu_mlp_fwd_amd as S  # noqa: E402
from test_gpu_group import DEV, host, normal, within  # noqa: E402


# ------------------------------------------------------------------ clipping

def test_clip_refuses_strided_gradients_that_overlap():
    """As contiguous ones: nothing is written, the shared elements are not counted twice."""
    a = normal((12, 20), 1, "f32")
    keep = a.clone()
    for views in ([a[:, ::2], a[:, ::2]], [a, a[:, ::2]]):
        with pytest.raises(ValueError, match="overlap"):
            S.clip_grads(views, 0.1)
    with pytest.raises(ValueError, match="overlap"):
        S.clip_grads([keep[:, :10], keep[:, 10:]], 0.1, out=[a[:, ::2], a[:, :10]])
    assert torch.equal(a, keep)
    even, odd = a[:, ::2], a[:, 1::2]
    norm, f = G.clip([host(a)], 0.5)
    got = S.clip_grads([even, odd], 0.5)
    assert abs(got.item() - norm) <= 2 * U32 * norm
    within(a, f * host(keep), 3 * U32 * np.abs(host(keep)), "interleaved columns")
