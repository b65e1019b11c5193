"""Refusals of the ragged products and the 4-bit operators: the C entry points return
a status before anything is launched (so no GPU is needed and no pointer is read), and
the Python layer checks tensors before it calls them."""

import ctypes

import pytest
import torch

import sparse_moe_transformer_route_b200 as M
from sparse_moe_transformer_route_b200 import binding as B
from tests.test_abi import built_library  # noqa: F401

OK, INVALID, SHAPE, SMALL, NO_DEVICE = 0, 1, 2, 3, 6
PTR = 1 << 20  # aligned and never read
ODD = PTR + 8


def _status(name):
    return next(code for code, text in B.STATUS_NAMES.items() if text == name)


def test_status_numbers():
    assert (_status("MOE_ERR_INVALID_ARG"), _status("MOE_ERR_UNSUPPORTED_SHAPE"),
            _status("MOE_ERR_WORKSPACE_TOO_SMALL"), _status("MOE_ERR_NO_DEVICE")) == (INVALID, SHAPE, SMALL, NO_DEVICE)


def _sh(rows=64, experts=4, n=64, k=64, dt=torch.bfloat16):
    return M.grouped_shape(rows, experts, n, k, dt)


def _product(fn, sh, a=PTR, b=PTR, c=PTR, off=PTR, ws=PTR, nws=256):
    ref = ctypes.byref(sh) if sh is not None else None
    if fn == "moe_grouped_gemm_wgrad":
        return getattr(M.lib(), fn)(ref, a, b, None, off, c, ws, nws, None)
    return getattr(M.lib(), fn)(ref, a, None, off, b, c, ws, nws, None)


PRODUCTS = ("moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad")


@pytest.mark.parametrize("fn", PRODUCTS)
def test_products_refuse(fn):
    assert _product(fn, None) == INVALID
    assert _product(fn, _sh(), off=None) == INVALID
    for who in ("a", "b", "c"):
        assert _product(fn, _sh(), **{who: None}) == INVALID
        assert _product(fn, _sh(), **{who: ODD}) == INVALID
    assert _product(fn, _sh(), ws=None) == INVALID
    assert _product(fn, _sh(), ws=PTR + 128) == INVALID
    assert _product(fn, _sh(), nws=255) == SMALL
    for bad in (dict(rows=-1), dict(rows=(1 << 28) + 1), dict(experts=0), dict(experts=257), dict(n=0), dict(n=12),
                dict(n=32776), dict(k=0), dict(k=4), dict(k=32776), dict(k=-8)):
        assert _product(fn, _sh(**bad)) == SHAPE, bad
    odd = _sh()
    odd.out_dtype = 2
    assert _product(fn, odd) == INVALID


def _fp4(sh, fmt, xc=PTR, xs=PTR, xg=None, wc=PTR, wsc=PTR, wg=None, y=PTR):
    return M.lib().moe_grouped_gemm_microscaled(ctypes.byref(sh), fmt, xc, xs, xg, None, PTR, wc, wsc, wg, y, PTR, 256,
                                                None)


def test_microscaled_product_refuses():
    assert _fp4(_sh(), 2) == INVALID and _fp4(_sh(), -1) == INVALID
    for who in ("xc", "xs", "wc", "wsc", "y"):
        assert _fp4(_sh(), M.MOE_NVFP4, **{who: None}) == INVALID
        assert _fp4(_sh(), M.MOE_NVFP4, **{who: ODD}) == INVALID
    assert _fp4(_sh(), M.MOE_MXFP4, xg=PTR) == INVALID
    assert _fp4(_sh(), M.MOE_MXFP4, wg=PTR) == INVALID
    for k in (8, 16, 48, 32784):
        assert _fp4(_sh(k=k), M.MOE_NVFP4) == SHAPE


def _convert(fn, fmt=1, g=1, r=4, c=64, dt=0, a=PTR, ts=PTR, b=PTR, d=PTR):
    lib = M.lib()
    if fn == "moe_quantize_microscaled":
        return lib.moe_quantize_microscaled(fmt, g, r, c, dt, a, ts, b, d, None)
    return lib.moe_dequantize_microscaled(fmt, g, r, c, dt, a, b, ts, d, None)


@pytest.mark.parametrize("fn", ["moe_quantize_microscaled", "moe_dequantize_microscaled"])
def test_conversions_refuse(fn):
    for fmt in (2, -1):
        assert _convert(fn, fmt=fmt) == INVALID
    for dt in (2, -1):
        assert _convert(fn, dt=dt) == INVALID
    assert _convert(fn, fmt=0) == INVALID  # a tensor scale with the format that has none
    for who in ("a", "b", "d"):
        assert _convert(fn, **{who: None}) == INVALID
        assert _convert(fn, **{who: ODD}) == INVALID
    for bad in (dict(g=0), dict(r=-1), dict(c=0), dict(c=16), dict(c=48), dict(c=(1 << 20) + 32),
                dict(g=1 << 20, r=1 << 20), dict(g=1 << 41), dict(r=1 << 41), dict(g=1 << 39, r=1 << 39)):
        assert _convert(fn, **bad) == SHAPE, bad


def test_tensor_scale_refuses():
    f = M.lib().moe_tensor_scale_microscaled
    assert f(1, 4, 64, 2, PTR, PTR, None) == INVALID
    assert f(1, 4, 64, 0, None, PTR, None) == INVALID
    assert f(1, 4, 64, 0, ODD, PTR, None) == INVALID
    assert f(1, 4, 64, 0, PTR, None, None) == INVALID
    assert f(0, 4, 64, 0, PTR, PTR, None) == SHAPE
    assert f(1, 4, 40, 0, PTR, PTR, None) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would launch")
def test_accepted_calls_need_a_device():
    for fn in PRODUCTS:
        assert _product(fn, _sh()) == NO_DEVICE
        assert _product(fn, _sh(rows=0), a=None) == NO_DEVICE  # a buffer of no rows may be NULL
    for fmt in (M.MOE_NVFP4, M.MOE_MXFP4):
        assert _fp4(_sh(), fmt) == NO_DEVICE
    assert _convert("moe_quantize_microscaled") == NO_DEVICE
    assert _convert("moe_dequantize_microscaled", fmt=0, ts=None) == NO_DEVICE
    assert M.lib().moe_tensor_scale_microscaled(1, 0, 64, 0, None, PTR, None) == NO_DEVICE


def test_binding_refuses():
    bf, u8 = torch.bfloat16, torch.uint8
    sh = _sh(16, 2, 64, 32)
    x, w, y = torch.zeros(16, 32, dtype=bf), torch.zeros(2, 64, 32, dtype=bf), torch.zeros(16, 64, dtype=bf)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=u8)
    with pytest.raises(ValueError, match="offsets must be a CUDA tensor"):
        M.moe_grouped_gemm(sh, x, None, off, w, y, ws)
    with pytest.raises(TypeError, match="offsets must be torch.int32"):
        M.moe_grouped_gemm(sh, x, None, off.long(), w, y, ws)
    with pytest.raises(ValueError, match="group_start must have shape"):
        M.moe_grouped_gemm_dgrad(sh, y, off[:2], off, w, x, ws)
    with pytest.raises(ValueError, match="out_dtype"):
        M.grouped_shape(16, 2, 64, 32, torch.float16)
    codes, scales = torch.zeros(16, 16, dtype=u8), torch.zeros(16, 2, dtype=u8)
    with pytest.raises(ValueError, match="format must be"):
        M.moe_quantize_microscaled(7, x, None, codes, scales)
    with pytest.raises(TypeError, match="x must be torch.bfloat16 or torch.float32"):
        M.moe_quantize_microscaled(M.MOE_NVFP4, x.half(), None, codes, scales)
    with pytest.raises(ValueError, match="two or three dimensions"):
        M.moe_tensor_scale_microscaled(x[0], off)
    with pytest.raises(ValueError, match="multiple of 32 columns"):
        M.moe_quantize_microscaled(M.MOE_NVFP4, x[:, :16].contiguous(), None, codes, scales)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        M.moe_quantize_microscaled(M.MOE_NVFP4, x, None, codes, scales)
    with pytest.raises(ValueError, match="x must be contiguous"):
        M.moe_quantize_microscaled(M.MOE_NVFP4, torch.zeros(32, 32, dtype=bf).t(), None, codes, scales)
