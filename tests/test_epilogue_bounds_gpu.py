"""Tighter checks of quant_matmul_act, quant_matmul_glu and their gradients, beside
test_epilogue_gpu.py, whose formulas and cases they share.
"""
import pytest
import torch

import bit_quantized_gemm_quant_b200 as bq
from test_epilogue_gpu import EVAL, HALF, Case, check_act, check_glu, df, f, near

pytestmark = pytest.mark.gpu


def check_column_sums(got, terms, err, what):
    """got: the bf16 column sums of `terms` (64 bits), each of which the kernel has within err.

    An fp32 sum of M terms in any order errs by at most (M + 8) 2^-24 sum |terms| (+ 8 for the
    sums over warps and row blocks); the result is rounded once to bf16.  With these terms
    the tolerance has to be small enough that a gradient of 0 would fail in most columns."""
    want = terms.sum(0)
    slack = err.sum(0) + (terms.shape[0] + 8) * 2.0 ** -24 * terms.abs().sum(0)
    assert ((HALF * want.abs() + slack) < want.abs()).double().mean() > 0.6, what
    near(got, want, slack, what)


@pytest.mark.parametrize("fmt,N,K,M", [("q4_0", 40, 64, 1), ("affine4", 264, 64, 31), ("affine8", 4100, 128, 700),
                                       ("affine8", 777, 4096, 1100), ("q4_0", 640, 4096, 1999),
                                       ("affine3", 203, 128, 2048), ("affine4", 840, 6144, 2600), ("q4_0", 24, 32, 20011)])
def test_bias_gradients_over_many_row_blocks(fmt, N, K, M):
    """Column sums over one row to several hundred row blocks, in both forms."""
    two = Case(fmt, N, K, M, 2)
    for act in ("none", "silu", "gelu"):
        dy, z, u = two.rand(M, N), two.rand(M, N, scale=2.0), two.rand(M, N)
        D, Z, U = dy.double(), z.double(), u.double()
        err = EVAL * (1 + Z.abs()) * D.abs()
        got = bq.quant_matmul_act_backward(dy, *two.mats[0], preact=z, act=act, group_size=two.gs, bits=two.bits,
                                           need_dbias=True)
        check_column_sums(got[2], D * df(act, Z), 0 * err if act == "none" else err, f"dbias {act}")
        got = bq.quant_matmul_glu_backward(dy, z, u, two.mats[0], two.mats[1], act, two.gs, two.bits, True)
        check_column_sums(got[3], D * U * df(act, Z), (err + 2.0 ** -22 * D.abs()) * U.abs(), f"dgate_bias {act}")
        check_column_sums(got[4], D * f(act, Z), err + 2.0 ** -22 * D.abs() * Z.abs(), f"dup_bias {act}")
    assert bq.bq_device_status() == 0


# What each covers of the kernel up to 16 tokens (2048 columns a chunk, 16 rows of W a tile):
# 8-bit codes past 1024 columns are a stage's second panel; K > 2048 with 2, 3 and 6 bits, K > 8192
# and 9 to 16 tokens with K > 4096 load the activations again for every chunk; N = 2500 gives a CTA
# two tiles of 16 rows (three of 8 + 8); K with a number of groups that is not a multiple of 8
# loads the scales past the ring.
RING = ([("affine8", 2500, 2048, M) for M in (1, 8, 16)] + [("affine8", 2500, 4224, M) for M in (1, 8, 16)] +
        [(fmt, 2500, 4224, 16) for fmt in ("affine8_g32", "affine8_g128")] + [("affine8_g32", 2500, 4192, 9)] +
        [(fmt, 2500, K, M) for fmt in ("affine2", "affine3", "affine6") for K, M in ((4480, 5), (4480, 16), (4608, 13))] +
        [("q4_0", 2500, 8480, 3), ("q4_0", 2500, 4384, 13), ("q4_0", 2501, 8704, 16), ("affine4", 2500, 10304, 2),
         ("affine4_g128", 2500, 14336, 1), ("affine4", 4900, 192, 11)])


@pytest.mark.parametrize("fmt,N,K,M", RING)
def test_decode_sizes_over_panels_chunks_and_tiles(fmt, N, K, M):
    check_act(Case(fmt, N, K, M, 1), "silu", bias=True, res=True, save=True)
    check_glu(Case(fmt, N, K, M, 2), "gelu_tanh", bias=True, save=True)
    assert bq.bq_device_status() == 0
