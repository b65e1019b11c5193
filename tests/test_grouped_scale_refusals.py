"""Refusals of the tensor scale over owned rows, without a GPU (nothing is launched and no
pointer is read)."""

import ctypes

import pytest
import torch

import sparse_moe_transformer_route_b200 as M
from tests.test_abi import built_library  # noqa: F401
from tests.test_grouped_refusals import INVALID, NO_DEVICE, ODD, PTR, SHAPE, SMALL


def _call(sh, dt=0, x=PTR, off=PTR, scale=PTR, ws=PTR, nws=256):
    ref = None if sh is None else ctypes.byref(sh)
    return M.lib().moe_grouped_tensor_scale_microscaled(ref, dt, x, None, off, scale, ws, nws, None)


def test_refuses():
    sh = M.grouped_shape(64, 4, 8, 64)
    assert _call(None) == INVALID
    for bad in (dict(dt=2), dict(dt=-1), dict(x=None), dict(x=ODD), dict(off=None), dict(scale=None), dict(ws=None),
                dict(ws=PTR + 128)):
        assert _call(sh, **bad) == INVALID, bad
    assert _call(sh, nws=255) == SMALL
    for bad in ((-1, 4, 8, 64), ((1 << 28) + 1, 4, 8, 64), (64, 0, 8, 64), (64, 257, 8, 64), (64, 4, 8, 48), (64, 4, 12, 64),
                (64, 4, 8, 32800)):
        assert _call(M.grouped_shape(*bad)) == SHAPE, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would launch")
def test_accepted_calls_need_a_device():
    assert _call(M.grouped_shape(64, 4, 8, 64), dt=1) == NO_DEVICE
    assert _call(M.grouped_shape(0, 4, 8, 64), x=None) == NO_DEVICE


def test_binding_refuses():
    sh = M.grouped_shape(16, 2, 8, 64)
    x, off, ws = torch.zeros(16, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    g = torch.zeros(1)
    with pytest.raises(TypeError, match="x must be a torch.bfloat16 or torch.float32"):
        M.moe_grouped_tensor_scale_microscaled(sh, x.half(), None, off, g, ws)
    with pytest.raises(TypeError, match="x must be a torch.bfloat16 or torch.float32"):
        M.moe_grouped_tensor_scale_microscaled(sh, None, None, off, g, ws)
    with pytest.raises(ValueError, match="offsets must have shape"):
        M.moe_grouped_tensor_scale_microscaled(sh, x, None, off[:2], g, ws)
    with pytest.raises(ValueError, match="offsets must be a CUDA tensor"):
        M.moe_grouped_tensor_scale_microscaled(sh, x, None, off, g, ws)
