"""add_rms_norm and its gradient against the formulas in 64 bits.

Tolerances, counted before their first run.  A thread adds 8 exact squares in fp32 (relative error
of the sum at most 8 2^-24, so of rstd half of that, 2^-22), the rest is fp64; y takes one more
rounding, so its relative error is below 2^-21.  Then one rounding to bf16, half a step (2^-8), or to the
quantized type: a code must be the rounding of some number within 2^-21 of y.  The gradient's sums are
fp32 sums of n terms, (n + 8) 2^-23 sum |terms|, with n = K or M.
"""
import pytest
import torch

import _mx
import bit_quantized_gemm_quant_b200 as bq

pytestmark = pytest.mark.gpu
HALF, NEAR = 2.0 ** -8, 2.0 ** -21
B16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(M, K, seed=0, res=True, scale=2.0):
    g = gen(seed + M + K)
    x = (scale * torch.randn(M, K, generator=g, device="cuda")).to(B16)
    r = (scale * torch.randn(M, K, generator=g, device="cuda")).to(B16) if res else None
    w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(B16)
    return x, r, w


def formula(x, r, w, eps):
    h = x if r is None else (x.double() + r.double()).float().to(B16)      # the sum of two bf16 near one another is exact in fp32
    hd = h.double()
    s = 1 / torch.sqrt(hd.square().mean(1) + eps)
    return h, s, hd * s[:, None] * w.double()


def check(x, r, w, eps=1e-5, quantize=None, **kw):
    y, h, rstd = bq.add_rms_norm(x, w, residual=r, eps=eps, quantize=quantize, save_rstd=True, **kw)
    if r is not None:
        want_h = (x.float() + r.float()).to(B16)
        assert torch.equal(h, want_h)
    hw, s, want = formula(h, None, w, eps)
    assert ((rstd.double() - s).abs() <= NEAR * s).all()
    lo, hi = want * (1 - NEAR), want * (1 + NEAR)
    if quantize is None:
        assert y.dtype == B16
        assert ((y.double() - want).abs() <= (HALF + NEAR) * want.abs() + 1e-40).all()
    elif quantize == "q8_1":
        q, d, qsum = y
        blocks = want.view(len(want), -1, 32)
        amax = blocks.abs().amax(2)
        assert ((d.double() - amax / 127).abs() <= 2 * NEAR * amax / 127).all()
        qd = q.double().view(blocks.shape)
        # half a unit, and the errors of y, d and 1 / d (below 4 NEAR of at most 127 units)
        assert ((qd * d.double()[..., None] - blocks).abs() <= d.double()[..., None] * (0.5 + 127 * 4 * NEAR)).all()
        assert torch.equal(qsum.long(), q.long().view(blocks.shape).sum(2))
    else:
        bits = int(quantize[-1])
        codes, scales = y
        byte = scales.view(torch.uint8)
        assert ((byte == _mx.scale_bytes(lo, bits)) | (byte == _mx.scale_bytes(hi, bits))).all()
        a, b = _mx.quantized(lo, bits, byte)[0], _mx.quantized(hi, bits, byte)[0]
        e = _mx.elements(codes)
        assert ((e >= torch.minimum(a, b)) & (e <= torch.maximum(a, b))).all()
    return y, h, rstd


SIZES = [(1, 8), (1, 1), (2, 7), (5, 33), (1, 256), (9, 264), (3, 512), (7, 520), (1, 1024), (5, 1032), (1, 2048), (33, 2056),
         (1, 4096), (2, 4104), (257, 4096), (3, 8192), (2, 8200), (1, 16384), (3, 16392), (2, 20000), (2, 16383), (1000, 96),
         (777, 2049)]


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(M, K, res):
    x, r, w = inputs(M, K, res=res)
    check(x, r, w)


@pytest.mark.parametrize("quantize", ["q8_1", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (17, 288), (5, 544), (9, 1056), (1, 2048), (70, 2080), (33, 4096), (5, 6176),
                                 (3, 8192), (2, 16384), (3, 16416), (2, 40000)])
def test_norm_quantized(M, K, quantize):
    x, r, w = inputs(M, K, seed=1)
    check(x, r, w, quantize=quantize)
    check(x, None, w, quantize=quantize)


@pytest.mark.parametrize("K", [32, 2048, 2049, 20000])
def test_norm_edges(K):
    x, r, w = inputs(6, K, seed=2)
    x[0], r[0] = 0, 0                                  # a row of zeros: rstd 1 / sqrt(eps), y 0
    x[1] = -r[1]                                       # cancels
    x[2], r[2] = 2.0 ** -60, 0                         # far below eps
    x[3], r[3] = 2.0 ** 50, 0
    y, h, rstd = check(x, r, w)
    assert not y[0].any() and not h[1].any()
    # a NaN or an infinity stays in its row
    x[4, K // 2] = float("nan")
    x[5, K - 1] = float("inf")
    r[5] = 1
    y, h, rstd = bq.add_rms_norm(x, w, residual=r, save_rstd=True)
    assert torch.isnan(y[4]).all() and torch.isnan(rstd[4])
    assert rstd[5] == 0 and torch.isnan(y[5, K - 1]) and not y[5, :K - 1].any()
    assert torch.isfinite(y[:4]).all()
    if K % 32 == 0:
        for bits, q in ((8, "mxfp8"), (4, "mxfp4")):
            codes, scales = bq.add_rms_norm(x, w, residual=r, quantize=q)[0]
            b = scales.view(torch.uint8)
            assert (b[4] == 255).all() and (b[:4] != 255).all() and b[5, -1] == 255 and not codes.view(torch.uint8)[0].any()


def test_norm_without_eps():
    x, _, w = inputs(3, 512, res=False)
    x[1] = 0
    y, _, rstd = bq.add_rms_norm(x, w, eps=0.0, save_rstd=True)
    assert rstd[1] == float("inf") and torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


@pytest.mark.parametrize("K", [512, 4096, 2049, 20000])
@pytest.mark.parametrize("quantize", [None, "mxfp8"])
def test_h_in_place(K, quantize):
    K = K // 32 * 32 if quantize else K
    x, r, w = inputs(9, K)
    want = bq.add_rms_norm(x, w, residual=r, quantize=quantize, save_rstd=True)
    flat = lambda t: [u for v in t for u in (v if isinstance(v, tuple) else (v,))]  # noqa: E731
    for which in ("residual", "x", "other"):
        a, b = x.clone(), r.clone()
        to = {"residual": b, "x": a, "other": torch.empty_like(a)}[which]
        got = bq.add_rms_norm(a, w, residual=b, quantize=quantize, save_rstd=True, h_out=to)
        assert got[1] is to
        for u, v in zip(flat(got), flat(want)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    copy = torch.empty_like(x)
    assert torch.equal(bq.add_rms_norm(x, w, h_out=copy)[1], x)


def test_norm_rows_do_not_depend_on_their_company():
    for K in (96, 2048, 4096, 2049):
        x, r, w = inputs(37, K)
        y = bq.add_rms_norm(x, w, residual=r)[0]
        for m in (0, 18, 36):
            assert torch.equal(bq.add_rms_norm(x[m:m + 1].clone(), w, residual=r[m:m + 1].clone())[0][0], y[m])


def test_norm_refusals():
    x, r, w = inputs(4, 64)
    with pytest.raises(ValueError, match="h_out: shares memory with residual"):
        big = torch.zeros(5 * 64, device="cuda", dtype=B16)
        bq.add_rms_norm(x, w, residual=big[:256].view(4, 64), h_out=big[64:].view(4, 64))
    with pytest.raises(ValueError, match="weight: shape"):
        bq.add_rms_norm(x, w[:32])
    with pytest.raises(TypeError, match="x: expected"):
        bq.add_rms_norm(x.float(), w)
    with pytest.raises(ValueError, match="contiguous"):
        bq.add_rms_norm(x, w, residual=r.t().contiguous().t())
    with pytest.raises(bq.BqError, match="SHAPE"):
        bq.add_rms_norm(x[:, :40].contiguous(), w[:40].clone(), quantize="mxfp8")
    with pytest.raises(bq.BqError, match="UNSUPPORTED"):
        bq.add_rms_norm(x, w, eps=-1.0)
    assert bq.add_rms_norm(x[:0], w, residual=r[:0], save_rstd=True)[2].shape == (0,)
    with pytest.raises(bq.BqError, match="SHAPE"):                 # a mean over nothing
        bq.add_rms_norm(x[:, :0].contiguous(), w[:0])
    dx, dw = bq.add_rms_norm_backward(x[:0], x[:0], w, torch.zeros(0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


def check_backward(M, K, dh, need=True, seed=3):
    x, r, w = inputs(M, K, seed=seed)
    g = gen(seed)
    dy = torch.randn(M, K, generator=g, device="cuda").to(B16)
    d = torch.randn(M, K, generator=g, device="cuda").to(B16) if dh else None
    _, h, rstd = bq.add_rms_norm(x, w, residual=r, save_rstd=True)
    dx, dw = bq.add_rms_norm_backward(dy, h, w, rstd, dh=d, need_dweight=need)
    hd, s, gd = h.double(), rstd.double()[:, None], dy.double() * w.double()
    dot, adot = (gd * hd).mean(1, keepdim=True), (gd * hd).abs().mean(1, keepdim=True)
    want = s * (gd - hd * s * s * dot) + (d.double() if dh else 0)
    err = s.pow(3) * hd.abs() * adot * (K + 16) * 2.0 ** -23 + s * gd.abs() * 2.0 ** -22 + (2.0 ** -23) * want.abs()
    assert ((dx.double() - want).abs() <= HALF * want.abs() + err * (1 + HALF)).all()
    if not need:
        assert dw is None
        return
    t = dy.double() * hd * s
    want = t.sum(0)
    err = (M + 8) * 2.0 ** -23 * t.abs().sum(0)
    assert ((dw.double() - want).abs() <= HALF * want.abs() + err * (1 + HALF)).all()
    again = bq.add_rms_norm_backward(dy, h, w, rstd, dh=d)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("M,K", SIZES + [(333, 2048), (2048, 512), (3000, 40), (1500, 1001)])
def test_norm_backward(M, K, dh):
    check_backward(M, K, dh)


def test_norm_backward_without_weight_gradient():
    for K in (64, 2048, 2049):
        check_backward(9, K, True, need=False)


def test_norm_gradient_is_its_difference():
    """Central differences in 64 bits of the formula, at the saved h; and autograd's of the same."""
    M, K = 3, 40
    x, r, w = inputs(M, K, seed=9)
    dy = torch.randn(M, K, generator=gen(4), device="cuda").to(B16)
    _, h, rstd = bq.add_rms_norm(x, w, residual=r, eps=1e-5, save_rstd=True)
    dx, dw = bq.add_rms_norm_backward(dy, h, w, rstd)

    def loss(hd, wd):
        return (hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-5) * wd * dy.double()).sum()
    hd, wd = h.double(), w.double()
    step = 1e-5
    num = torch.empty_like(hd)
    for m in range(M):
        for k in range(K):
            e = torch.zeros_like(hd)
            e[m, k] = step
            num[m, k] = (loss(hd + e, wd) - loss(hd - e, wd)) / (2 * step)
    assert ((dx.double() - num).abs() <= HALF * num.abs() + 1e-5).all()
    for k in range(K):
        e = torch.zeros_like(wd)
        e[k] = step
        n = (loss(hd, wd + e) - loss(hd, wd - e)) / (2 * step)
        assert abs(float(dw[k]) - float(n)) <= HALF * abs(float(n)) + 1e-5
    ha, wa = hd.clone().requires_grad_(), wd.clone().requires_grad_()
    loss(ha, wa).backward()
    assert ((dx.double() - ha.grad).abs() <= HALF * ha.grad.abs() + 1e-5).all()
    assert ((dw.double() - wa.grad).abs() <= HALF * wa.grad.abs() + 1e-5).all()
