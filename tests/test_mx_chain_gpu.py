"""The norm, the microscaled product and their gradients as they are used: one after the other, into
captured graphs, on streams of their own, beside one another, and in buffers of exactly their size.

Tolerances as in test_mx_gpu.py and test_norm_gpu.py; where a step takes a rounded result of the one before,
it is held to the formula at that result.
"""
import subprocess
import sys

import pytest
import torch

import _mx
import bit_quantized_gemm_quant_b200 as bq

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
B16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def layer(M, N, K, seed=0):
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(B16)
    r = torch.randn(M, K, generator=g, device="cuda").to(B16)
    w = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(B16)
    W = bq.mxfp4_quantize(0.05 * torch.randn(N, K, generator=g, device="cuda"))
    return x, r, w, W


def near(got, want, slack):
    excess = (got.double() - want).abs() - HALF * want.abs() - slack
    assert torch.isfinite(got).all() and excess.max() <= 0, float(excess.max())


def product(x, w):
    return x @ w.t(), (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t()) * (1 + HALF)


@pytest.mark.parametrize("quantize", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (7, 300, 544), (100, 640, 1024), (600, 257, 2080)])
def test_norm_into_product_and_back(M, N, K, quantize):
    x, r, w, W = layer(M, N, K)
    q, h, rstd = bq.add_rms_norm(x, w, residual=r, quantize=quantize, save_rstd=True)
    y = bq.mx_matmul(*q, *W)
    near(y, *product(_mx.values(*q), _mx.values(*W)))
    # what the codes stand for is the norm, to the type's half step (E4M3 2^-4; E2M1: a quarter of the block's
    # scale below 2, which is at least an eighth of its largest value, and 2 beyond 6, a third) of it
    hd = h.double()
    n = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-5) * w.double()
    amax = n.view(M, -1, 32).abs().amax(2, keepdim=True).expand(-1, -1, 32).reshape(M, K)
    assert ((_mx.values(*q) - n).abs() <= (0.5 if quantize == "mxfp4" else 0.126) * amax).all()
    # the way back: dy to the normed rows, and on to the residual stream beside dh
    g = gen(1)
    dy, dh = torch.randn(M, N, generator=g, device="cuda").to(B16), torch.randn(M, K, generator=g, device="cuda").to(B16)
    dn = bq.mx_matmul_backward(dy, *W)
    near(dn, *product(dy.double(), _mx.values(*W).t()))
    dx, dw = bq.add_rms_norm_backward(dn, h, w, rstd, dh=dh)
    hr, wr = hd.clone().requires_grad_(), w.double().requires_grad_()
    out = hr / torch.sqrt(hr.square().mean(1, keepdim=True) + 1e-5) * wr
    (out * dn.double()).sum().backward()
    s = rstd.double()[:, None]
    gd = (dn.double() * w.double()).abs()
    slack = s.pow(3) * hd.abs() * (gd * hd.abs()).mean(1, keepdim=True) * (K + 16) * 2.0 ** -23 + s * gd * 2.0 ** -20
    near(dx, hr.grad + dh.double(), slack + 2.0 ** -23 * (hr.grad.abs() + dh.double().abs()))
    near(dw, wr.grad, (M + 16) * 2.0 ** -21 * (dn.double() * hd * s).abs().sum(0))


def test_norm_into_q8_product():
    M, N, K = 5, 384, 1024
    x, r, w, _ = layer(M, N, K)
    wq, sc = bq.q4_0_quantize(0.05 * torch.randn(N, K, generator=gen(3), device="cuda"))
    (q, d, qsum), h = bq.add_rms_norm(x, w, residual=r, quantize="q8_1")
    y = bq.quant_matmul_q8(q, d, qsum, wq, sc)
    xv = (q.double().view(M, -1, 32) * d.double()[..., None]).view(M, K)
    b = wq.view(N, -1, 16)
    wv = ((torch.cat([b & 15, b >> 4], 2).double() - 8) * sc.double()[..., None]).view(N, K)
    near(y, *product(xv, wv))


def test_quantized_norm_is_the_quantizer_of_the_norm():
    """Where the norm's result is exact in bf16 (rows of +-1, weights of few bits, no eps), both ways agree bit for bit."""
    M, K = 6, 512
    x = torch.where(torch.rand(M, K, generator=gen(2), device="cuda") < 0.5, -1.0, 1.0).to(B16)
    w = (torch.randint(-48, 49, (K,), generator=gen(3), device="cuda").float() / 16).to(B16)
    y = bq.add_rms_norm(x, w, eps=0.0)[0]
    assert torch.equal(y.float(), x.float() * w.float())
    for name, f in (("mxfp8", bq.mxfp8_quantize), ("mxfp4", bq.mxfp4_quantize)):
        (c, s), _ = bq.add_rms_norm(x, w, eps=0.0, quantize=name)
        c2, s2 = f(y)
        assert torch.equal(s.view(torch.uint8), s2.view(torch.uint8))
        assert torch.equal(_mx.elements(c), _mx.elements(c2))
    (q, d, n), _ = bq.add_rms_norm(x, w, eps=0.0, quantize="q8_1")
    for a, b in zip((q, d, n), bq.q8_1_quantize(y)):
        assert torch.equal(a, b)


def forward(x, r, w, W):
    q, h, rstd = bq.add_rms_norm(x, w, residual=r, quantize="mxfp8", save_rstd=True)
    y = bq.mx_matmul(*q, *W)
    dn = bq.mx_matmul_backward(y, *W)
    dx, dw = bq.add_rms_norm_backward(dn, h, w, rstd, dh=h)
    return [q[0].view(torch.uint8), q[1].view(torch.uint8), h, rstd, y, dn, dx, dw]


SHAPES = [(3, 640, 1024), (70, 640, 1056), (700, 513, 2048)]


def test_captured_and_replayed():
    """Two graphs with their own inputs, replayed in turn and after the inputs changed: an eager call's bits."""
    for shape in SHAPES:
        graphs = []
        for seed in (0, 1):
            ins = layer(*shape, seed=seed)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                forward(*ins)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    outs = forward(*ins)
            torch.cuda.current_stream().wait_stream(side)
            graphs.append((ins, g, outs))
        for turn in range(3):
            for i, (ins, g, outs) in enumerate(graphs):
                ins[0].copy_(torch.randn(ins[0].shape, generator=gen(10 * turn + i), device="cuda").to(B16))
            for _, g, _ in graphs:
                g.replay()
            torch.cuda.synchronize()
            for ins, _, outs in graphs:
                for a, b in zip(outs, forward(*ins)):
                    assert torch.equal(a, b)


def test_first_call_in_a_capture():
    code = """
import torch, sys
sys.path.insert(0, %r)
import bit_quantized_gemm_quant_b200 as bq
b = torch.bfloat16
for M in (3, 300):
    x, w = torch.randn(M, 1024, device="cuda").to(b), torch.ones(1024, device="cuda", dtype=b)
    codes = torch.randint(0, 256, (256, 512), device="cuda", dtype=torch.uint8)
    scales = torch.full((256, 32), 120, device="cuda", dtype=torch.uint8)
    def f():
        q, h, rstd = bq.add_rms_norm(x, w, residual=x, quantize="mxfp8", save_rstd=True)
        y = bq.mx_matmul(*q, codes, scales)
        return [y, *bq.add_rms_norm_backward(bq.mx_matmul_backward(y, codes, scales), h, w, rstd)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = f()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, f()))
print("done")
""" % bq.__file__.rsplit("/", 2)[0]
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


def test_streams_at_once():
    """Calls of different shapes on two streams at once, and a call on a stream that is handed in: the same bits."""
    ins = [layer(*s, seed=i) for i, s in enumerate(SHAPES)]
    want = [forward(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[] for _ in ins]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(forward(*ins[i]))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        for outs in got[i]:
            for a, b in zip(outs, w):
                assert torch.equal(a, b)
    st = streams[0]
    x, r, w, W = ins[1]
    st.wait_stream(torch.cuda.current_stream())
    q, h, rstd = bq.add_rms_norm(x, w, residual=r, quantize="mxfp8", save_rstd=True, stream=st)
    y = bq.mx_matmul(*q, *W, stream=st)
    dn = bq.mx_matmul_backward(y, *W, stream=st)
    dx, dw = bq.add_rms_norm_backward(dn, h, w, rstd, dh=h, stream=st)
    back = bq.mxfp8_dequantize(*bq.mxfp8_quantize(x, stream=st), stream=st)
    st.synchronize()
    for a, b in zip([q[0].view(torch.uint8), q[1].view(torch.uint8), h, rstd, y, dn, dx, dw], want[1]):
        assert torch.equal(a, b)
    assert torch.equal(back, bq.mxfp8_dequantize(*bq.mxfp8_quantize(x)))


def test_products_of_every_kind_at_once():
    """Products on clusters, on pairs of SMs, and gradients, of one stage and of many, that meet on the SMs from
    streams of their own: each holds tensor memory, and those that wait for another SM's part keep apart."""
    def codes(rows, k, bits, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        return _mx.random_codes(rows, k, bits, g)

    sizes = [(1, 2048, 8192, 8), (16, 1024, 2048, 4), (300, 8192, 64, 4), (700, 2048, 1024, 8), (260, 4096, 4096, 4)]
    ins = [(codes(m, k, a, i), codes(n, k, 4, 20 + i), torch.randn(m, n, device="cuda").bfloat16())
           for i, (m, n, k, a) in enumerate(sizes)]
    calls = [lambda i=i: bq.mx_matmul(*i[0], *i[1]) for i in ins] + [lambda i=i: bq.mx_matmul_backward(i[2], *i[1]) for i in ins[2:4]]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(30):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w.view(torch.int16), o.view(torch.int16)) for o in outs)


@pytest.mark.parametrize("M,N,K,a", [(3, 300, 1056, 8), (200, 300, 1056, 8), (300, 700, 4096, 8), (130, 260, 4096, 4),
                                     (700, 520, 1024, 4)])
def test_workspaces_of_exactly_their_size(M, N, K, a):
    """Through the C ABI, in workspaces of the reported size filled with NaN patterns: nothing stale is read, nothing
    behind them written, and one byte less is refused."""
    L = bq.lib()
    g = gen(4)
    x, W = _mx.random_codes(M, K, a, g), _mx.random_codes(N, K, 4, g)
    st = torch.cuda.current_stream().cuda_stream

    def space(n):
        return torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(n, call):
        ws = space(n)
        assert call(ws.data_ptr(), n) == 0
        assert (ws[n:] == 0xFF).all()
        if n:
            assert call(ws.data_ptr(), n - 1) == 7
    y = torch.empty(M, N, dtype=B16, device="cuda")
    run(L.mx_matmul_workspace_size(M, N, K, a),
        lambda p, n: L.mx_matmul(x[0].data_ptr(), x[1].data_ptr(), a, W[0].data_ptr(), W[1].data_ptr(), y.data_ptr(), M, N, K, p, n, st))
    assert torch.equal(y, bq.mx_matmul(*x, *W))
    # the library's own buffer
    y2 = torch.empty_like(y)
    assert L.mx_matmul(x[0].data_ptr(), x[1].data_ptr(), a, W[0].data_ptr(), W[1].data_ptr(), y2.data_ptr(), M, N, K, None, 0, st) == 0
    assert torch.equal(y, y2)
    dy, dx = torch.randn(M, N, generator=g, device="cuda").to(B16), torch.empty(M, K, dtype=B16, device="cuda")
    run(L.mx_matmul_backward_workspace_size(M, N, K),
        lambda p, n: L.mx_matmul_backward(dy.data_ptr(), W[0].data_ptr(), W[1].data_ptr(), dx.data_ptr(), M, N, K, p, n, st))
    assert torch.equal(dx, bq.mx_matmul_backward(dy, *W))
    h, w = dx, torch.ones(K, dtype=B16, device="cuda")
    rstd = torch.ones(M, device="cuda")
    d2, dw = torch.empty_like(dx), torch.empty(K, dtype=B16, device="cuda")
    run(L.add_rms_norm_backward_workspace_size(M, K),
        lambda p, n: L.add_rms_norm_backward(dx.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(), None, d2.data_ptr(),
                                             dw.data_ptr(), M, K, p, n, st))
    want = bq.add_rms_norm_backward(dx, h, w, rstd)
    assert torch.equal(d2, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 2080), (77, 4128), (301, 512)])
def test_nothing_beside_the_outputs_is_written(M, K):
    """Outputs inside larger buffers, by the C ABI, of the quantizers, the dequantizers, the norm and its gradient."""
    L = bq.lib()
    st = torch.cuda.current_stream().cuda_stream
    x, r, w, _ = layer(M, 8, K)
    bufs = []

    def out(n):
        b = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        bufs.append((b, n))
        return b.data_ptr() + 256
    for bits, q, d in ((4, L.mxfp4_quantize, L.mxfp4_dequantize), (8, L.mxfp8_quantize, L.mxfp8_dequantize)):
        c, s = out(M * K * bits // 8), out(M * K // 32)
        assert q(x.data_ptr(), 0, c, s, M, K, st) == 0
        assert d(c, s, out(2 * M * K), M, K, st) == 0
    for fmt, size, scale in ((0, 2 * M * K, 0), (1, M * K, M * K // 8), (2, M * K, M * K // 32), (3, M * K // 2, M * K // 32)):
        assert L.add_rms_norm(x.data_ptr(), r.data_ptr(), w.data_ptr(), 1e-5, fmt, out(size), out(scale) if scale else None,
                              out(M * K // 8) if fmt == 1 else None, out(2 * M * K), out(4 * M), M, K, st) == 0
    rstd = torch.ones(M, device="cuda")
    for k in (K, K - 1):
        ws = torch.empty(max(16, L.add_rms_norm_backward_workspace_size(M, k)), dtype=torch.uint8, device="cuda")
        assert L.add_rms_norm_backward(x.data_ptr(), r.data_ptr(), w.data_ptr(), rstd.data_ptr(), None, out(2 * M * k), out(2 * k), M, k,
                                       ws.data_ptr(), ws.numel(), st) == 0
        assert L.add_rms_norm(x.data_ptr(), r.data_ptr(), w.data_ptr(), 1e-5, 0, out(2 * M * k), None, None, out(2 * M * k), out(4 * M), M,
                              k, st) == 0
    torch.cuda.synchronize()
    for b, n in bufs:
        assert (b[:256] == 0xA5).all() and (b[256 + n:] == 0xA5).all()


def test_bit_patterns_and_dtypes():
    """bf16 operands as 16-bit patterns and scales as bytes, as everywhere in the package."""
    x, r, w, W = layer(4, 128, 256)
    i16 = lambda t: t.view(torch.int16)  # noqa: E731
    want = bq.add_rms_norm(x, w, residual=r, quantize="mxfp8")[0]
    got = bq.add_rms_norm(i16(x), i16(w), residual=i16(r), quantize="mxfp8")[0]
    assert torch.equal(want[0].view(torch.uint8), got[0].view(torch.uint8))
    y = bq.mx_matmul(*want, *W)
    out = torch.empty(4, 128, dtype=torch.int16, device="cuda")
    assert bq.mx_matmul(want[0], want[1].view(torch.uint8), W[0], W[1].view(torch.uint8), out=out) is out
    assert torch.equal(out.view(B16), y)
    assert torch.equal(bq.mx_matmul_backward(i16(y), *W), bq.mx_matmul_backward(y, *W))
    assert torch.equal(bq.mxfp4_quantize(i16(x))[0], bq.mxfp4_quantize(x)[0])


def test_large_offsets():
    """Outputs and inputs past 2^31 elements: the last rows are those of a small call."""
    M, K = 300_000, 8192                                 # 2.5e9 elements
    x = torch.ones(1, K, device="cuda", dtype=B16).repeat(M, 1)
    x[-3:] = torch.randn(3, K, generator=gen(0), device="cuda").to(B16)
    w = torch.ones(K, device="cuda", dtype=B16)
    (c, s), h, rstd = bq.add_rms_norm(x, w, quantize="mxfp8", save_rstd=True)
    (c2, s2), _, rstd2 = bq.add_rms_norm(x[-3:].clone(), w, quantize="mxfp8", save_rstd=True)
    assert torch.equal(c[-3:].view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s[-3:].view(torch.uint8), s2.view(torch.uint8))
    assert torch.equal(rstd[-3:], rstd2)
    q4 = bq.mxfp4_quantize(x)
    assert torch.equal(q4[0][-3:], bq.mxfp4_quantize(x[-3:].clone())[0])
    back = bq.mxfp8_dequantize(c, s)
    assert torch.equal(back[-3:], bq.mxfp8_dequantize(c2, s2))
    del back, q4
    # a product whose output passes 2^31 elements
    W = bq.mxfp4_quantize(torch.randn(8192, 64, generator=gen(1), device="cuda"))
    cx, sx = c[:, :64].contiguous(), s.view(torch.uint8)[:, :2].contiguous()
    del x, c, s, h
    y = bq.mx_matmul(cx, sx, *W)
    assert torch.equal(y[-200:], bq.mx_matmul(cx[-200:].clone(), sx[-200:].clone(), *W)) or \
        ((y[-200:].double() - _mx.values(cx[-200:], sx[-200:]) @ _mx.values(*W).t()).abs() <=
         HALF * y[-200:].double().abs() + 72 * 2.0 ** -23 * (_mx.values(cx[-200:], sx[-200:]).abs() @ _mx.values(*W).abs().t()) * 1.01).all()
