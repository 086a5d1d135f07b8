"""Microscaled rows, their product and its gradient against their definitions in 64 bits.

Quantizers and dequantizers are exact.  A product's tolerance, counted before its first run:
its one rounding to bf16, half a step (2^-8 relative), and an fp32 sum of n terms, which errs by
at most (n + 8) 2^-23 sum |terms| (each addition by one fp32 step of a partial sum, + 8 for
split sums).
"""
import pytest
import torch

import _mx
import bit_quantized_gemm_quant_b200 as bq

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
QUANT = {4: bq.mxfp4_quantize, 8: bq.mxfp8_quantize}
DEQUANT = {4: bq.mxfp4_dequantize, 8: bq.mxfp8_dequantize}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def signs(codes):
    """The sign bits of stored codes."""
    if codes.dtype == torch.uint8:
        return torch.stack([codes & 8, codes & 128], 2).reshape(codes.shape[0], -1) != 0
    return codes.view(torch.uint8) >= 128


def check_quantize(x, bits):
    codes, scales = QUANT[bits](x)
    want, byte = _mx.quantized(x, bits)
    assert codes.dtype == (torch.float8_e4m3fn if bits == 8 else torch.uint8) and scales.dtype == torch.float8_e8m0fnu
    assert torch.equal(scales.view(torch.uint8), byte)
    assert torch.equal(_mx.elements(codes), want)
    finite = (byte != 255).repeat_interleave(32, 1)
    assert torch.equal(signs(codes)[finite], torch.signbit(x)[finite])
    assert not codes.view(torch.uint8).view(x.shape[0], -1, 4 * bits)[byte == 255].any()
    return codes, scales


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 96), (17, 4128), (1000, 64), (333, 2080)])
def test_quantize(bits, dtype, M, K):
    x = torch.randn(M, K, generator=gen(M + K), device="cuda")
    x *= torch.exp(4 * torch.randn(M, K // 32, generator=gen(1), device="cuda")).repeat_interleave(32, 1)
    check_quantize(x.to(dtype), bits)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_edges(bits):
    tiny, big = 2.0 ** -149, 3.4028234663852886e38
    rows = [torch.zeros(32), -torch.zeros(32)]
    rows += [torch.full((32,), v) for v in (tiny, -tiny, 2.0 ** -127, 1.5 * 2.0 ** -126, big, -big)]
    for v in (float("nan"), float("inf"), -float("inf")):
        r = torch.randn(32, generator=torch.Generator().manual_seed(0))
        r[7] = v
        rows.append(r)
    # every border of the element types' grids, and its neighbours, under an amax that fixes the scale
    mid = (_mx.GRID[1:] + _mx.GRID[:-1]).float() / 2 if bits == 4 else None
    if bits == 8:
        codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        mid = ((codes[1:] + codes[:-1]) / 2).float()
    top = torch.tensor([4.0 if bits == 4 else 256.0])
    for d in (-1, 0, 1):
        m = (mid.view(torch.int32) + d).view(torch.float32)
        m = m[m < 2 * top]
        for part in m.split(31):
            rows.append(torch.cat([top, part, torch.zeros(31 - len(part))]))
            rows.append(-rows[-1])
    # saturation: amax just below the next power of two
    rows.append(torch.cat([torch.tensor([1.9999999]), torch.linspace(-1.99, 1.99, 31)]))
    x = torch.stack(rows).cuda()
    codes, scales = check_quantize(x, bits)
    back = DEQUANT[bits](codes, scales).float()
    assert torch.isnan(back[8:11]).all() and torch.isfinite(back[:8]).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_dequantize_every_code_and_scale(bits):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)
    K = 256 if bits == 8 else 512
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].expand(256, K // 32).contiguous()
    if bits == 8:
        codes = codes.view(torch.float8_e4m3fn)
    got = DEQUANT[bits](codes, scales)
    e = _mx.elements(codes)
    # X * element in fp64, to bf16 once.  (fp64 to bf16 by way of fp32: exact but for subnormal results, of at most 4 bits)
    want = (e * _mx.power(scales).repeat_interleave(32, 1)).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine])
    assert torch.isnan(got[255]).all()
    out = torch.empty_like(got)
    assert DEQUANT[bits](codes, scales.view(torch.float8_e8m0fnu), out=out) is out
    assert torch.equal(out.view(torch.int16), got.view(torch.int16))


def bound(x, w):
    """(the product, its error bound) of fp64 values."""
    want = x @ w.t()
    return want, (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t()) * (1 + HALF)


def near(got, want, slack, what=""):
    assert got.shape == want.shape and got.dtype == torch.bfloat16
    got = got.double()
    assert torch.isfinite(got).all(), what
    excess = (got - want).abs() - HALF * want.abs() - slack
    assert excess.numel() == 0 or excess.max() <= 0, f"{what}: off by {float(excess.max()):.3e} at {int(excess.argmax())}"


def check_matmul(M, N, K, a, seed=0, spread=6):
    g = gen(seed + M + N + K)
    x, w = _mx.random_codes(M, K, a, g, spread), _mx.random_codes(N, K, 4, g, spread)
    y = bq.mx_matmul(*x, *w)
    near(y, *bound(_mx.values(*x), _mx.values(*w)), f"{M} x {N} x {K}, {a} bits")
    return x, w, y


SIZES = [(1, 1, 32), (1, 40, 96), (1, 2048, 8192), (2, 129, 256), (3, 250, 160), (5, 128, 128), (7, 1000, 512), (8, 256, 4096),
         (15, 333, 1056), (16, 384, 2048), (17, 127, 640), (31, 2048, 2048), (32, 255, 384), (33, 512, 1024), (64, 1111, 544),
         (65, 4096, 256), (100, 77, 8192), (127, 256, 2560), (129, 640, 768), (200, 1500, 1184), (256, 2048, 512),
         (300, 8192, 128), (511, 1024, 4096), (777, 2309, 224), (1999, 520, 1536), (4096, 64, 64)]


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, a):
    check_matmul(M, N, K, a)


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 12288, 4096), (2048, 12288, 4096), (4096, 8192, 2048)])
def test_matmul_large(M, N, K, a):
    check_matmul(M, N, K, a)


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M", [1, 20, 300])
def test_matmul_wide_scales(a, M):
    check_matmul(M, 200, 512, a, spread=30)


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (40, 200, 256), (300, 300, 640)])
def test_matmul_one_hot(a, M, N, K):
    """x = one element: y is W's column, exactly; every k and both matrices' layouts."""
    g = gen(3)
    w = _mx.random_codes(N, K, 4, g)
    W = _mx.values(*w)
    ks = torch.randint(0, K, (M,), generator=g, device="cuda")
    x = torch.zeros(M, K, device="cuda")
    x[torch.arange(M, device="cuda"), ks] = 1.0
    y = bq.mx_matmul(*QUANT[a](x), *w)
    assert torch.equal(y.double(), W[:, ks].t())


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M", [1, 9, 70, 400])
def test_matmul_nan_scale_stays_in_its_row(a, M):
    N, K = 300, 512
    g = gen(5)
    x, w = _mx.random_codes(M, K, a, g), _mx.random_codes(N, K, 4, g)
    w[1].view(torch.uint8)[17, 3] = 255
    w[1].view(torch.uint8)[N - 1, 15] = 255
    y = bq.mx_matmul(*x, *w)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[17] = bad[N - 1] = True
    assert torch.isnan(y[:, bad]).all() and torch.isfinite(y[:, ~bad]).all()
    w[1].view(torch.uint8)[17, 3] = w[1].view(torch.uint8)[N - 1, 15] = 127
    x[1].view(torch.uint8)[M // 2, 1] = 255
    y = bq.mx_matmul(*x, *w)
    rows = torch.arange(M, device="cuda") == M // 2
    assert torch.isnan(y[rows]).all() and torch.isfinite(y[~rows]).all()


@pytest.mark.parametrize("a", [4, 8])
@pytest.mark.parametrize("M,N,K", [(3, 300, 512), (150, 300, 512), (150, 301, 544)])
def test_matmul_neighbours_are_left_alone(a, M, N, K):
    """out inside a larger buffer, inputs as views behind others' bytes."""
    g = gen(6)
    x, w = _mx.random_codes(M + 2, K, a, g), _mx.random_codes(N, K, 4, g)
    x = (x[0][1:M + 1], x[1].view(torch.uint8)[1:M + 1].clone())
    if x[0].data_ptr() % 16:
        x = (x[0].clone(), x[1])
    buf = torch.full((M * N + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[32:32 + M * N].view(M, N)
    assert bq.mx_matmul(*x, *w, out=out) is out
    near(out, *bound(_mx.values(x[0], x[1]), _mx.values(*w)))
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


def test_matmul_same_bits_again():
    for a in (4, 8):
        x, w, y = check_matmul(150, 1000, 4096, a)
        for _ in range(3):
            assert torch.equal(bq.mx_matmul(*x, *w), y)


def test_matmul_empty_and_refused():
    w = _mx.random_codes(64, 64, 4, gen(0))
    x = _mx.random_codes(4, 64, 8, gen(0))
    assert bq.mx_matmul(x[0][:0], x[1][:0], *w).shape == (0, 64)
    assert bq.mx_matmul(*x, w[0][:0], w[1][:0]).shape == (4, 0)
    e = torch.empty(4, 0, dtype=torch.uint8, device="cuda")
    assert not bq.mx_matmul(e, e, torch.empty(5, 0, dtype=torch.uint8, device="cuda"), torch.empty(5, 0, dtype=torch.uint8, device="cuda")).any()
    with pytest.raises(ValueError, match="wq: shape"):
        bq.mx_matmul(*x, w[0][:, :16].contiguous(), w[1])
    with pytest.raises(ValueError, match="x_scales: shape"):
        bq.mx_matmul(x[0], x[1].view(torch.uint8)[:, :1].contiguous(), *w)
    with pytest.raises(TypeError, match="xq: expected"):
        bq.mx_matmul(x[0].view(torch.int8), x[1], *w)
    with pytest.raises(TypeError, match="w_scales: expected"):
        bq.mx_matmul(*x, w[0], w[1].view(torch.uint8).float())
    with pytest.raises(ValueError, match="contiguous"):
        bq.mx_matmul(*x, w[0].t().contiguous().t(), w[1])
    with pytest.raises(ValueError, match="not on the call's device"):
        bq.mx_matmul(*x, w[0].cpu(), w[1])
    with pytest.raises(ValueError, match="out: shares memory with xq"):
        big = torch.zeros(4 * 64, dtype=torch.uint8, device="cuda")
        bq.mx_matmul(big[:128].view(4, 32), x[1], w[0][:32], w[1][:32], out=big.view(torch.bfloat16).view(4, 32))
    with pytest.raises(bq.BqError, match="ALIGN"):
        flat = torch.zeros(64 * 32 + 8, dtype=torch.uint8, device="cuda")
        bq.mx_matmul(*x, flat[8:].view(64, 32), w[1])
    with pytest.raises(bq.BqError, match="SHAPE"):
        bq.mxfp4_quantize(torch.zeros(4, 40, device="cuda"))
    with pytest.raises(TypeError):
        bq.mxfp8_quantize(torch.zeros(4, 64, device="cuda", dtype=torch.float64))


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 2048, 512), (3, 250, 160), (8, 333, 96), (17, 129, 1056), (33, 1000, 256),
                                   (64, 40, 2048), (129, 641, 544), (300, 2048, 1024), (777, 1111, 640), (1999, 512, 512)])
def test_matmul_backward(M, N, K):
    g = gen(M + N)
    w = _mx.random_codes(N, K, 4, g)
    dy = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    dx = bq.mx_matmul_backward(dy, *w)
    near(dx, *bound(dy.double(), _mx.values(*w).t()))
    assert torch.equal(dx, bq.mx_matmul_backward(dy, *w))


def test_matmul_backward_empty():
    w = _mx.random_codes(64, 96, 4, gen(0))
    dy = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    assert bq.mx_matmul_backward(dy[:0], *w).shape == (0, 96)
    none = torch.zeros(4, 0, device="cuda", dtype=torch.bfloat16)
    assert not bq.mx_matmul_backward(none, w[0][:0], w[1][:0]).any()


def test_gradient_is_the_product_s_difference():
    """mx_matmul is linear in x: for a step of one element, the change of sum(dy * y) is dx there, in 64 bits."""
    M, N, K = 5, 64, 96
    g = gen(8)
    w = _mx.random_codes(N, K, 4, g, spread=2)
    dy = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    dx = bq.mx_matmul_backward(dy, *w).double()
    unit = torch.zeros(K, K, device="cuda")
    unit.fill_diagonal_(4.0)
    y = bq.mx_matmul(*bq.mxfp4_quantize(unit), *w).double()          # row k: 4 W[:, k], exact in bf16
    want = (dy.double() @ y.t()) / 4
    slack = (N + 8) * 2.0 ** -23 * (dy.double().abs() @ y.abs().t()) / 4
    assert ((dx - want).abs() <= HALF * want.abs() + slack * (1 + HALF)).all()
