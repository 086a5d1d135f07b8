"""Refusals of the products with an epilogue, all on the host before any CUDA call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import bit_quantized_gemm_quant_b200 as bq
    return bq.lib()


P = ctypes.c_void_p
A, BAD = P(0x1000), P(0x1008)
VP = ctypes.c_void_p * 2
OK, NULL, SHAPE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4


def act(L, x=A, wq=A, s=A, b=None, ob=None, r=None, act=1, y=A, z=None, M=4, N=64, K=64, g=32, bits=4, ws=None, wsb=0):
    return L.quant_matmul_act(x, wq, s, b, ob, r, act, y, z, M, N, K, g, bits, ws, wsb, None)


def glu(L, x=A, wq=(0x1000, 0x1000), s=(0x1000, 0x1000), b=None, ob=None, act=4, h=A, g=None, u=None, M=4, N=64, K=64,
        gs=32, bits=4):
    return L.quant_matmul_glu(x, VP(*wq), VP(*s), None if b is None else VP(*b), ob, None, act, h, g, u, M, N, K, gs, bits,
                              None, 0, None)


def act_bwd(L, dy=A, z=A, wq=A, s=A, b=None, act=1, dx=A, dz=A, db=None, M=4, N=64, K=64, g=32, bits=4):
    return L.quant_matmul_act_backward(dy, z, wq, s, b, act, dx, dz, db, M, N, K, g, bits, None, 0, None)


def glu_bwd(L, dh=A, g=A, u=A, wq=(0x1000, 0x1000), s=(0x1000, 0x1000), b=None, act=4, dx=A, dg=A, du=A, M=4, N=64, K=64,
            gs=32, bits=4):
    return L.quant_matmul_glu_backward(dh, g, u, VP(*wq), VP(*s), None if b is None else VP(*b), act, dx, dg, du, None,
                                       None, M, N, K, gs, bits, None, 0, None)


@pytest.mark.parametrize("call", [act, glu, act_bwd, glu_bwd])
def test_shared_refusals(L, call):
    gs = "g" if call in (act, act_bwd) else "gs"
    assert call(L, M=-1) == call(L, N=-1) == call(L, K=-64) == SHAPE
    assert call(L, K=48) == SHAPE                                     # Q4_0 blocks of 32
    assert call(L, M=2 ** 31) == call(L, N=2 ** 30) == SHAPE
    assert call(L, act=5) == call(L, act=-1) == UNSUPPORTED
    assert call(L, bits=8) == UNSUPPORTED                             # Q4_0 is 4-bit, groups of 32
    assert call(L, **{gs: 64}) == UNSUPPORTED
    two = A if call in (act, act_bwd) else (0x1000, 0x1000)
    assert call(L, b=two, **{gs: 64}, bits=5) == UNSUPPORTED
    assert call(L, b=two, **{gs: 16}) == UNSUPPORTED
    assert call(L, b=two, **{gs: 128}, K=64) == SHAPE


def test_pointers(L):
    assert act(L, x=None) == act(L, wq=None) == act(L, s=None) == act(L, y=None) == NULL
    for k in ("x", "wq", "s", "ob", "r", "y", "z", "ws"):
        assert act(L, **{k: BAD}) == ALIGN, k
    assert act(L, b=BAD) == ALIGN
    assert glu(L, x=None) == glu(L, h=None) == NULL
    assert glu(L, wq=(0x1000, 0)) == glu(L, s=(0, 0x1000)) == NULL
    assert glu(L, b=(0x1000, 0), gs=64) == NULL                       # both affine or both Q4_0
    assert glu(L, g=A) == glu(L, u=A) == NULL                         # both saved or neither
    assert glu(L, wq=(0x1000, 0x1008)) == glu(L, h=BAD) == ALIGN
    assert L.quant_matmul_glu(A, None, None, None, None, None, 4, A, None, None, 4, 64, 64, 32, 4, None, 0, None) == NULL
    assert act_bwd(L, dy=None) == act_bwd(L, z=None) == act_bwd(L, dz=None) == act_bwd(L, dx=None) == NULL
    assert act_bwd(L, z=BAD) == act_bwd(L, db=BAD) == ALIGN
    assert glu_bwd(L, u=None) == glu_bwd(L, du=None) == glu_bwd(L, g=None) == NULL
    assert glu_bwd(L, dg=BAD) == ALIGN


def test_empty_problems_touch_nothing(L):
    assert act(L, x=None, wq=None, s=None, y=None, M=0) == act(L, x=None, wq=None, s=None, y=None, N=0) == OK
    assert glu(L, x=None, h=None, M=0) == glu(L, x=None, h=None, N=0) == OK
    assert act_bwd(L, dy=None, z=None, dx=None, dz=None, M=0) == OK
    assert glu_bwd(L, dh=None, dx=None, M=0) == glu_bwd(L, dh=None, dx=None, N=0, K=0) == OK


def test_workspace_sizes(L):
    size = L.quant_matmul_epilogue_workspace_size
    for op in range(4):
        for bad in ((0, 64, 64, 32, 4), (4, 0, 64, 32, 4), (4, 64, 48, 32, 4), (4, 64, 64, 16, 4), (4, 64, 64, 64, 5)):
            assert size(op, *bad) == 0, (op, bad)
    assert size(-1, 4, 64, 64, 32, 4) == size(4, 4, 64, 64, 32, 4) == 0
    # 2-, 3- and 6-bit weights go through a bf16 copy, gate and up through two
    for bits in (2, 3, 6):
        assert size(1, 4, 64, 128, 64, bits) >= 64 * 128 * 2 and size(3, 4, 64, 128, 64, bits) >= 2 * 64 * 128 * 2
        assert size(0, 40, 64, 128, 64, bits) >= 64 * 128 * 2 and size(2, 40, 64, 128, 64, bits) >= 2 * 64 * 128 * 2
    # without biases Q4_0 and affine 4-bit in groups of 32 are told apart by nothing: one size
    assert size(0, 1, 64, 128, 32, 4) == 0


def test_binding_refusals():
    import bit_quantized_gemm_quant_b200 as bq
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    wq, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16)
    for call in (lambda: bq.quant_matmul_act(x, wq, s), lambda: bq.quant_matmul_glu(x, (wq, s, None), (wq, s, None)),
                 lambda: bq.quant_matmul_act_backward(x, wq, s),
                 lambda: bq.quant_matmul_glu_backward(x, x, x, (wq, s, None), (wq, s, None))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
