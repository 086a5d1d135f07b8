"""Refusals of the microscaled formats, their product and the norm: on the host, before any CUDA call."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A, BAD = P(0x1000), P(0x1008)
OK, NULL, SHAPE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import bit_quantized_gemm_quant_b200 as bq
    return bq.lib()


@pytest.mark.parametrize("name", ["mxfp4_quantize", "mxfp8_quantize"])
def test_quantize(L, name):
    def f(x=A, t=0, c=A, s=A, M=4, K=64):
        return getattr(L, name)(x, t, c, s, M, K, None)
    assert f(M=-1) == f(K=-32) == f(K=48) == f(K=31) == SHAPE
    assert f(M=2 ** 60) == SHAPE
    assert f(t=2) == f(t=-1) == UNSUPPORTED
    assert f(x=None) == f(c=None) == f(s=None) == NULL
    assert f(x=BAD) == f(c=BAD) == f(s=BAD) == ALIGN
    assert f(x=None, c=None, s=None, M=0) == f(x=None, c=None, s=None, K=0) == OK


@pytest.mark.parametrize("name", ["mxfp4_dequantize", "mxfp8_dequantize"])
def test_dequantize(L, name):
    def f(c=A, s=A, o=A, M=4, K=64):
        return getattr(L, name)(c, s, o, M, K, None)
    assert f(M=-1) == f(K=-32) == f(K=40) == f(M=2 ** 60) == SHAPE
    assert f(c=None) == f(s=None) == f(o=None) == NULL
    assert f(c=BAD) == f(s=BAD) == f(o=BAD) == ALIGN
    assert f(c=None, M=0) == f(o=None, K=0) == OK


def test_matmul(L):
    def f(x=A, xs=A, bits=8, w=A, ws=A, y=A, M=4, N=64, K=64, buf=None, n=0):
        return L.mx_matmul(x, xs, bits, w, ws, y, M, N, K, buf, n, None)
    assert f(M=-1) == f(N=-1) == f(K=-32) == f(K=48) == SHAPE
    assert f(M=2 ** 31) == f(N=2 ** 30) == SHAPE
    assert f(bits=5) == f(bits=16) == f(bits=0) == UNSUPPORTED
    for k in ("x", "xs", "w", "ws", "y"):
        assert f(**{k: None}) == NULL, k
        assert f(**{k: BAD}) == ALIGN, k
    assert f(buf=BAD) == ALIGN
    assert f(x=None, y=None, M=0) == f(w=None, y=None, N=0) == OK
    size = L.mx_matmul_workspace_size
    assert size(0, 64, 64, 8) == size(4, 0, 64, 8) == size(4, 64, 48, 8) == size(4, 64, 64, 5) == size(2 ** 31, 64, 64, 8) == 0


def test_matmul_backward(L):
    def f(dy=A, w=A, ws=A, dx=A, M=4, N=64, K=64, buf=None, n=0):
        return L.mx_matmul_backward(dy, w, ws, dx, M, N, K, buf, n, None)
    assert f(M=-1) == f(N=-1) == f(K=-32) == f(K=48) == f(M=2 ** 31) == f(N=2 ** 30) == SHAPE
    for k in ("dy", "w", "ws", "dx"):
        assert f(**{k: None}) == NULL, k
        assert f(**{k: BAD}) == ALIGN, k
    assert f(buf=BAD) == ALIGN
    assert f(dy=None, dx=None, M=0) == f(dx=None, K=0) == OK
    size = L.mx_matmul_backward_workspace_size
    assert size(0, 64, 64) == size(4, 0, 64) == size(4, 64, 48) == 0
    assert size(4, 64, 64) > 0


def test_norm(L):
    def f(x=A, r=None, w=A, eps=1e-5, out=0, y=A, s=None, q=None, h=None, rstd=None, M=4, K=64):
        return L.add_rms_norm(x, r, w, eps, out, y, s, q, h, rstd, M, K, None)
    assert f(M=-1) == f(K=-1) == f(M=2 ** 30) == f(K=2 ** 30) == f(K=0) == f(M=0, K=0) == SHAPE
    assert f(out=4) == f(out=-1) == f(eps=-1e-6) == f(eps=float("nan")) == f(eps=float("inf")) == UNSUPPORTED
    for out in (1, 2, 3):
        assert f(out=out, s=A, q=A, K=40) == SHAPE
        assert f(out=out, q=A) == NULL
    assert f(out=1, s=A) == NULL
    assert f(x=None) == f(w=None) == f(y=None) == NULL
    for k in ("x", "r", "w", "y", "s", "q", "h", "rstd"):
        assert f(**{k: BAD}) == ALIGN, k
    assert f(x=None, y=None, M=0) == OK


def test_norm_backward(L):
    def f(dy=A, h=A, w=A, rstd=A, dh=None, dx=A, dw=None, M=4, K=64, buf=None, n=0):
        return L.add_rms_norm_backward(dy, h, w, rstd, dh, dx, dw, M, K, buf, n, None)
    assert f(M=-1) == f(K=-1) == f(M=2 ** 30) == f(K=2 ** 30) == SHAPE
    for k in ("dy", "h", "w", "rstd", "dx"):
        assert f(**{k: None}) == NULL, k
        assert f(**{k: BAD}) == ALIGN, k
    assert f(dh=BAD) == f(dw=BAD) == f(buf=BAD) == ALIGN
    assert f(dy=None, dx=None, M=0) == f(K=0, dw=A) == OK
    size = L.add_rms_norm_backward_workspace_size
    assert size(0, 64) == size(4, 0) == 0
    assert size(2048, 64) >= 64 * 4 and size(2048, 77) >= 77 * 4


def test_binding_refusals():
    import bit_quantized_gemm_quant_b200 as bq
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: bq.mxfp4_quantize(x), lambda: bq.mxfp8_quantize(x), lambda: bq.mxfp4_dequantize(c, s),
                 lambda: bq.mxfp8_dequantize(c, s), lambda: bq.mx_matmul(c, s, c, s), lambda: bq.mx_matmul_backward(x, c, s),
                 lambda: bq.add_rms_norm(x, x[0]), lambda: bq.add_rms_norm_backward(x, x, x[0], f)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="quantize"):
        bq.add_rms_norm(x, x[0], quantize="fp8")
    with pytest.raises(TypeError, match="expected a tensor"):
        bq.mx_matmul(None, s, c, s)
