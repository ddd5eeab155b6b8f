"""The products grouped by expert and the row operators on the host: what the C ABI refuses before it touches a
device, and what the binding refuses before it calls."""
import ctypes

import pytest
import torch

import fine_grained_moe_gemm_b200 as moe

P = ctypes.c_void_p
BAD, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK
B16, H16, F32, E43 = moe.MOE_BF16, moe.MOE_F16, moe.MOE_F32, moe.MOE_E4M3
NO_GPU = not torch.cuda.is_available()


X, W, Y, Z, V = (i << 24 for i in range(1, 6))   # addresses far apart


def _mm(groups=4, rows=10, n=64, k=32, dtype=B16, x=X, ldx=32, w=W, tr=0, off=16, y=Y, ldy=64, out=B16, acc=0):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_grouped_mm(groups, rows, n, k, dtype, p(x), ldx, p(w), tr, p(off), p(y), ldy, out, acc, None)


SHAPES = [dict(groups=0), dict(groups=1025), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(n=0), dict(n=12), dict(k=4),
          dict(k=36), dict(n=65544), dict(k=65544), dict(off=None), dict(off=18), dict(acc=2), dict(out=17)]


@pytest.mark.parametrize("wrong", SHAPES + [
    dict(x=None), dict(w=None), dict(y=None), dict(x=24), dict(w=8), dict(y=4), dict(ldx=31), dict(ldx=36), dict(ldy=56),
    dict(ldy=68), dict(tr=2), dict(dtype=9), dict(ldy=66, out=F32)])
def test_mm_refuses(wrong):
    assert _mm(**wrong) == BAD


def test_mm_types_and_nothing_to_do():
    assert _mm(dtype=F32, out=F32) == UNS and _mm(dtype=E43) == UNS
    assert _mm(dtype=B16, out=H16) == UNS and _mm(dtype=H16, out=B16) == UNS
    assert _mm(out=E43) == BAD
    assert _mm(rows=0, x=None, w=None, y=None) == OK
    if NO_GPU:
        assert _mm() == UNS and _mm(groups=1, off=None) == UNS


def _wgrad(groups=4, rows=10, n=64, k=32, dtype=B16, dy=Y, lddy=64, x=X, ldx=32, off=16, dw=W, out=F32, acc=0):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_grouped_wgrad(groups, rows, n, k, dtype, p(dy), lddy, p(x), ldx, p(off), p(dw), out, acc, None)


@pytest.mark.parametrize("wrong", SHAPES + [dict(dy=None), dict(x=None), dict(dw=None), dict(dy=8), dict(dw=8),
                                            dict(lddy=60), dict(ldx=33), dict(rows=0, dw=None)])
def test_wgrad_refuses(wrong):
    assert _wgrad(**wrong) == BAD


def test_wgrad_types():
    assert _wgrad(dtype=F32) == UNS and _wgrad(dtype=H16, out=B16) == UNS
    if NO_GPU:
        assert _wgrad() == UNS and _wgrad(rows=0, dy=None, x=None) == UNS


def _mm8(groups=4, rows=10, n=64, k=32, q=X, sx=4, w=W, sw=4, off=16, y=Y, ldy=64, out=B16, acc=0):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_grouped_mm_int8(groups, rows, n, k, p(q), p(sx), p(w), p(sw), p(off), p(y), ldy, out, acc, None)


@pytest.mark.parametrize("wrong", SHAPES + [dict(k=8), dict(k=24), dict(q=None), dict(sx=None), dict(w=None),
                                            dict(sw=None), dict(y=None), dict(q=8), dict(sx=2), dict(ldy=60),
                                            dict(out=E43)])
def test_mm_int8_refuses(wrong):
    assert _mm8(**wrong) == BAD


def test_mm_int8_accepts():
    assert _mm8(rows=0, q=None, sx=None, w=None, sw=None, y=None) == OK
    if NO_GPU:
        for out in (B16, H16, F32):
            assert _mm8(out=out) == UNS


def _swiglu(rows=4, width=64, dtype=B16, gate=X, ldg=64, up=W, ldu=64, coef=None, n=None, h=Y, ldh=64):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_swiglu(rows, width, dtype, p(gate), ldg, p(up), ldu, p(coef), p(n), p(h), ldh, None)


def _swiglu_b(rows=4, width=64, dtype=B16, dh=X, gate=W, up=Y, coef=None, n=None, dgate=Z, dup=V, dcoef=None, ld=64):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_swiglu_backward(rows, width, dtype, p(dh), ld, p(gate), ld, p(up), ld, p(coef), p(n), p(dgate), ld,
                                         p(dup), ld, p(dcoef), None)


@pytest.mark.parametrize("wrong", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(width=0), dict(width=12),
                                   dict(width=65544), dict(dtype=9), dict(gate=None), dict(up=8), dict(coef=2),
                                   dict(n=2)])
def test_swiglu_refuses(wrong):
    assert _swiglu(**wrong) == BAD
    assert _swiglu_b(**wrong) == BAD


def test_swiglu_more():
    assert _swiglu(h=None) == BAD and _swiglu(ldg=56) == BAD and _swiglu(ldh=68) == BAD and _swiglu(dtype=E43) == UNS
    assert _swiglu_b(dh=None) == BAD and _swiglu_b(dgate=8) == BAD and _swiglu_b(dup=None) == BAD
    assert _swiglu_b(dcoef=2) == BAD and _swiglu_b(ld=60) == BAD and _swiglu_b(dtype=E43) == UNS
    assert _swiglu(rows=0, gate=None, up=None, h=None) == OK
    assert _swiglu_b(rows=0, dh=None, gate=None, up=None, dgate=None, dup=None) == OK
    if NO_GPU:
        assert _swiglu() == UNS and _swiglu(dtype=F32) == UNS and _swiglu_b(coef=16, dcoef=16) == UNS


def _quant(x=X, dtype=B16, ldx=64, rows=4, k=64, n=None, q=Y, sx=16):
    p = lambda v: None if v is None else P(v)
    return moe.lib().moe_quantize_int8(p(x), dtype, ldx, rows, k, p(n), p(q), p(sx), None)


@pytest.mark.parametrize("wrong", [dict(x=None), dict(q=None), dict(sx=None), dict(x=8), dict(q=8), dict(sx=2), dict(n=2),
                                   dict(rows=-1), dict(k=8), dict(k=72), dict(k=32784), dict(ldx=60), dict(dtype=9)])
def test_quantize_refuses(wrong):
    assert _quant(**wrong) == BAD


def test_quantize_more():
    assert _quant(dtype=E43) == UNS and _quant(rows=0, x=None, q=None, sx=None) == OK
    if NO_GPU:
        assert _quant() == UNS


def test_outputs_over_inputs():
    """Shared bytes are refused before a launch; disjoint columns of one buffer are not, nor the elementwise
    operators in place."""
    fine = UNS if NO_GPU else OK
    if not NO_GPU:
        pytest.skip("the accepted calls would launch on made-up addresses")
    row = 96 * 2                                                 # x: 32 columns, y: 64 columns of 96
    assert _mm(x=X, ldx=96, y=X + 64, ldy=96) == fine
    assert _mm(x=X + 128, ldx=96, y=X, ldy=96) == fine
    assert _mm(x=X, ldx=96, y=X + 48, ldy=96) == BAD             # y starts inside x
    assert _mm(x=X, ldx=96, y=X + 9 * row + 48, ldy=96) == BAD   # only the last row of x
    assert _mm(x=X, ldx=96, y=X + 10 * row, ldy=96) == fine
    assert _mm(x=X, ldx=96, y=X + 64, ldy=104) == BAD            # another distance of rows over the same bytes
    assert _mm(x=X, y=X) == BAD and _mm(y=W) == BAD and _mm(y=W + 4 * 64 * 32 * 2 - 16) == BAD
    assert _mm(y=W + 4 * 64 * 32 * 2) == fine
    assert _wgrad(dw=X) == BAD and _wgrad(dw=Y) == BAD and _wgrad(dw=X - 16) == BAD
    assert _mm8(y=X) == BAD and _mm8(y=W) == BAD
    assert _quant(q=X) == BAD and _quant(q=X + 4 * 64 * 2 - 16) == BAD and _quant(q=X + 4 * 64 * 2) == fine
    assert _swiglu(h=X) == fine and _swiglu(h=W) == fine and _swiglu(h=X + 16) == BAD
    assert _swiglu(h=X, ldh=72) == BAD
    assert _swiglu_b(dgate=W, dup=Y) == fine and _swiglu_b(dgate=Y, dup=W) == fine and _swiglu_b(dup=X) == fine
    assert _swiglu_b(dgate=W, dup=W) == BAD and _swiglu_b(dgate=W + 16) == BAD and _swiglu_b(dup=X + 32) == BAD


def test_outputs_over_vectors():
    """The offsets, scales, coefficients and counts are inputs too."""
    if not NO_GPU:
        pytest.skip("the accepted calls would launch on made-up addresses")
    assert _mm(off=Y + 16) == BAD and _mm(off=Y - 16) == BAD and _mm(off=Y - 20) == UNS   # five offsets
    assert _wgrad(off=W) == BAD and _wgrad(off=W + 4 * 64 * 32 * 4 - 4) == BAD and _wgrad(off=W + 4 * 64 * 32 * 4) == UNS
    assert _mm8(off=Y) == BAD and _mm8(sx=Y) == BAD and _mm8(sw=Y - 4 * 4 * 64 + 4) == BAD and _mm8(sw=Y - 4 * 4 * 64) == UNS
    assert _swiglu(coef=Y + 4 * 64 * 2 - 4) == BAD and _swiglu(n=Y) == BAD and _swiglu(coef=Y - 16, n=Y - 4) == UNS
    assert _swiglu_b(coef=Z) == BAD and _swiglu_b(n=V) == BAD and _swiglu_b(dcoef=V) == BAD and _swiglu_b(dcoef=Z) == BAD
    assert _swiglu_b(dcoef=X) == BAD and _swiglu_b(dcoef=W) == BAD and _swiglu_b(dcoef=Y) == BAD
    assert _swiglu_b(coef=16, dcoef=20) == BAD and _swiglu_b(n=16, dcoef=16) == BAD
    assert _swiglu_b(coef=16, dcoef=16) == UNS and _swiglu_b(coef=16, dcoef=32) == UNS
    assert _quant(sx=X) == BAD and _quant(sx=Y) == BAD and _quant(n=Y) == BAD and _quant(n=28) == BAD and _quant(n=32) == UNS


def test_binding_refuses_host_tensors():
    x, w, y = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 8, 16).bfloat16(), torch.zeros(4, 8)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: moe.moe_grouped_mm(x, w, off, y), lambda: moe.moe_grouped_wgrad(x, x, off, w),
                 lambda: moe.moe_swiglu(x, x, x), lambda: moe.moe_swiglu_backward(x, x, x, x, x),
                 lambda: moe.moe_quantize_int8(x, x.to(torch.int8), y[:, 0]),
                 lambda: moe.moe_grouped_mm_int8(x.to(torch.int8), y[:, 0], w.to(torch.int8), y[:2], off, y)):
        with pytest.raises(ValueError):
            call()


def test_enum_matches_the_header():
    text = open(moe.HEADER_PATH).read()
    assert "MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2, MOE_F16 = 3" in text
    assert (moe.MOE_F32, moe.MOE_BF16, moe.MOE_E4M3, moe.MOE_F16) == (0, 1, 2, 3)
