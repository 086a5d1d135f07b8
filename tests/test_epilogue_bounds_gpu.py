"""Tighter checks of quant_matmul_act, quant_matmul_glu and their gradients, beside
test_epilogue_gpu.py, whose formulas and cases they share.
"""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import bit_quantized_gemm_quant_b200 as bq
from test_epilogue_gpu import EVAL, HALF, Case, check_act, check_glu, df, f, near, sums

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


FORMS = ["act", "act_backward", "glu", "glu_backward"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt,N,K", [("q4_0", 520, 1024), ("affine4", 777, 640), ("affine8", 203, 4160), ("affine3", 777, 640),
                                     ("affine6", 264, 384)])
def test_nothing_of_the_workspace_is_read_before_it_is_written(form, fmt, N, K):
    """A workspace of exactly the reported size, filled with NaN patterns (0xFF bytes: NaN as
    bf16 and as fp32), gives the bits of a call with its own, and the bytes behind it stay."""
    P = ctypes.c_void_p
    L = bq.lib()
    for M in (17, 40, 300, 1100):
        c = Case(fmt, N, K, M, 2)
        (wq, s, b), (wq2, s2, b2) = c.mats
        kw = dict(group_size=c.gs, bits=c.bits)
        need = bq.quant_matmul_epilogue_workspace_size(FORMS.index(form), M, N, K, c.gs, c.bits)
        assert need > 0
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        tail = (M, N, K, c.gs, c.bits, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)

        def ptr(t):
            return None if t is None else t.data_ptr()

        def pair(x, y):
            return None if x is None else (P * 2)(x.data_ptr(), y.data_ptr())

        def out(*shape):
            return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")

        if form == "act":
            x, r = c.rand(M, K), c.rand(M, N)
            want = bq.quant_matmul_act(x, wq, s, b, act="gelu", residual=r, save_preact=True, **kw)
            got = out(M, N), out(M, N)
            st = L.quant_matmul_act(ptr(x), ptr(wq), ptr(s), ptr(b), None, ptr(r), 2, ptr(got[0]), ptr(got[1]), *tail)
        elif form == "act_backward":
            dy, z = c.rand(M, N), c.rand(M, N)
            want = bq.quant_matmul_act_backward(dy, wq, s, b, z, "silu", need_dbias=True, **kw)
            got = out(M, K), out(M, N), out(N)
            st = L.quant_matmul_act_backward(ptr(dy), ptr(z), ptr(wq), ptr(s), ptr(b), 4, *map(ptr, got), *tail)
        elif form == "glu":
            x = c.rand(M, K)
            want = bq.quant_matmul_glu(x, *c.mats, act="silu", save_preact=True, **kw)
            got = out(M, N), out(M, N), out(M, N)
            st = L.quant_matmul_glu(ptr(x), pair(wq, wq2), pair(s, s2), pair(b, b2), None, None, 4, *map(ptr, got), *tail)
        else:
            dh, g, u = c.rand(M, N), c.rand(M, N), c.rand(M, N)
            want = bq.quant_matmul_glu_backward(dh, g, u, *c.mats, act="relu", need_dbias=True, **kw)
            got = out(M, K), out(M, N), out(M, N), out(N), out(N)
            st = L.quant_matmul_glu_backward(ptr(dh), ptr(g), ptr(u), pair(wq, wq2), pair(s, s2), pair(b, b2), 1,
                                             *map(ptr, got), *tail)
        assert st == 0
        for a, w in zip(got, want):
            assert torch.isfinite(w).all() and torch.equal(a, w), (form, M)
        assert (ws[need:] == 0xFF).all()
    assert bq.bq_device_status() == 0


# act and act' far left of 0, without the cancellation of 1 + tanh and 1 + erf: the factor p that
# multiplies z, the two terms of the derivative, and the argument a of p's exponential.
def tail_terms(act, z):
    if act == "silu":
        p = torch.sigmoid(z)
        return p, z * p * torch.sigmoid(-z), z.abs()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), z * z / 2
    c = 2 * math.sqrt(2 / math.pi)
    a = c * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(a)
    return p, z * p * torch.sigmoid(-a) * c * (1 + 3 * 0.044715 * z * z), a.abs()


@pytest.mark.parametrize("act,left", [("gelu", -12.9), ("gelu_tanh", -9.9), ("silu", -85.0)])
def test_tails_of_the_activations(act, left):
    """act(z) and act'(z) for z from -3 to `left`, where both vanish (1e-35), relative to themselves.

    W is 0, so that z is the bias.  e^-a in fp32 is within (a + 4) 2^-23 of itself; the
    roundings of a itself add 2 a 2^-24 (gelu: half of z z and its product with log2 e),
    or 6 (gelu_tanh, with those of its constants); gelu's polynomial may be as far off as
    its exponential; the reciprocal and the products are a few steps of 2^-24."""
    N, K = 264, 64
    z = torch.linspace(-3, left, N, device="cuda").to(torch.bfloat16)
    Z = z.double()
    p, q, a = tail_terms(act, Z)
    rel = ({"silu": 1, "gelu": 3, "gelu_tanh": 4}[act] * a + 16) * 2.0 ** -23

    def hold(got, want, terms, what):
        off = (got.double() - want).abs() - HALF * want.abs() - rel * terms
        i = int(off.max(0).values.argmax())
        assert (off <= 0).all(), f"{what}: z = {float(Z[i])}, {got[0, i].item()} for {float(want[i])}"

    one = torch.ones_like(z)
    for fmt in ("q4_0", "affine4", "affine3"):
        for M in (2, 40):
            c = Case(fmt, N, K, M, 1)
            wq, s, b = c.mats[0]
            w = (wq, torch.zeros_like(s), None if b is None else torch.zeros_like(b))
            x, kw = c.rand(M, K), dict(group_size=c.gs, bits=c.bits)
            hold(bq.quant_matmul_act(x, *w, out_bias=z, act=act, **kw), Z * p, (Z * p).abs(), "act")
            hold(bq.quant_matmul_glu(x, w, w, z, one, act, **kw), Z * p, (Z * p).abs(), "glu")
            rows, ones = z.expand(M, N).contiguous(), one.expand(M, N).contiguous()
            dz = bq.quant_matmul_act_backward(ones, *w, preact=rows, act=act, **kw)[1]
            hold(dz, p + q, p + q.abs(), "dz")
            _, dg, du = bq.quant_matmul_glu_backward(ones, rows, ones, w, w, act, **kw)
            hold(dg, p + q, p + q.abs(), "dg")
            hold(du, Z * p, (Z * p).abs(), "du")


def test_out_of_memory_is_pytorchs_error():
    """An output of 2 TB: the error type that quant_matmul's own allocation gives, and the next call runs."""
    n = 1 << 20
    x = torch.zeros(n, 32, dtype=torch.bfloat16, device="cuda")
    wq, s = torch.zeros(n, 16, dtype=torch.uint8, device="cuda"), torch.zeros(n, 1, dtype=torch.float16, device="cuda")
    for call in (bq.quant_matmul, bq.quant_matmul_act, lambda x, wq, s: bq.quant_matmul_glu(x, (wq, s, None), (wq, s, None))):
        with pytest.raises(torch.OutOfMemoryError):
            call(x, wq, s)
    assert not bq.quant_matmul_act(x[:4], wq[:8], s[:8]).any()


def test_out_that_shares_memory_with_an_input_is_refused():
    """Square weights make out = x fit; a residual is taken whole or not at all."""
    M, N = 24, 128
    c = Case("affine4", N, N, M, 2)
    kw = dict(group_size=c.gs, bits=c.bits)
    wq, s, b = c.mats[0]
    buf = torch.zeros(2 * M, N, dtype=torch.bfloat16, device="cuda")
    x, out, bias = buf[:M].copy_(c.rand(M, N)), buf[M:], c.rand(M, N)
    act = lambda **k: bq.quant_matmul_act(k.pop("x", x), wq, s, b, **kw, **k)
    glu = lambda **k: bq.quant_matmul_glu(k.pop("x", x), *c.mats, **kw, **k)
    want, want_glu = act(residual=bias).clone(), glu().clone()
    for call in (act, glu):
        for o in (x, buf[1:M + 1], buf[M - 1:2 * M - 1]):
            with pytest.raises(ValueError, match="shares memory with x"):
                call(out=o)
    with pytest.raises(ValueError, match="residual"):
        act(residual=buf[M - 8:2 * M - 8], x=bias, out=out)
    with pytest.raises(ValueError, match="out_bias"):
        act(out_bias=out[3], out=out)
    with pytest.raises(ValueError, match="up_bias"):
        glu(up_bias=out[M - 1], out=out)
    words = torch.zeros(N * N // 8 + M * N // 2, dtype=torch.int32, device="cuda")     # codes, then an output's place
    codes = words[:N * N // 8].view(N, N // 8)
    place = words.view(torch.bfloat16)[:M * N].view(M, N)
    with pytest.raises(ValueError, match="w.wq"):
        bq.quant_matmul_act(x, codes, s, b, out=place, **kw)
    with pytest.raises(ValueError, match="up"):
        bq.quant_matmul_glu(x, c.mats[0], (codes, s, b), out=place, **kw)
    # beside an input is apart
    assert act(residual=bias, out=out) is out and torch.equal(out, want)
    assert glu(out=out) is out and torch.equal(out, want_glu)
    assert torch.equal(act(residual=out.copy_(bias), out=out), want)
    # nothing to write: nothing shared
    e = x[:0]
    assert act(x=e, out=e) is e


@pytest.mark.parametrize("bits", [torch.int16, torch.uint16])
def test_bit_patterns_stand_for_bf16_in_every_operand(bits):
    """int16 and uint16 tensors, as quant_matmul takes them: the results are those of the bf16 tensors."""
    M, N, K = 20, 72, 64
    c = Case("affine4", N, K, M, 2)
    kw = dict(group_size=c.gs, bits=c.bits)
    raw = lambda t: t.view(bits)
    mats = [(wq, raw(s), raw(b)) for wq, s, b in c.mats]
    x, bias, r, y = c.rand(M, K), c.rand(N), c.rand(M, N), c.rand(M, N)
    for call in (lambda t, m, o: bq.quant_matmul_act(t(x), *m[0], out_bias=t(bias), act="gelu", residual=t(r), out=o, **kw),
                 lambda t, m, o: bq.quant_matmul_glu(t(x), *m, t(bias), t(bias), out=o, **kw)):
        out = torch.empty(M, N, dtype=bits, device="cuda")
        assert call(raw, mats, out) is out
        assert torch.equal(out.view(torch.bfloat16), call(lambda t: t, c.mats, None))
    for call in (lambda t, m: bq.quant_matmul_act_backward(t(y), *m[0], preact=t(r), act="silu", need_dbias=True, **kw),
                 lambda t, m: bq.quant_matmul_glu_backward(t(y), t(r), t(y), *m, need_dbias=True, **kw)):
        for a, b in zip(call(raw, mats), call(lambda t: t, c.mats)):
            assert torch.equal(a, b)
    dy = raw(y)
    dx, dz = bq.quant_matmul_act_backward(dy, *mats[0], **kw)
    assert dz is dy and torch.equal(dx, bq.quant_matmul_act_backward(y, *c.mats[0], **kw)[0])
    with pytest.raises(TypeError, match="dy"):
        bq.quant_matmul_act_backward(y.to(torch.float16), *mats[0], **kw)


def test_a_product_of_seconds_is_no_timeout():
    """2.5 s of tensor-core work in one kernel (2 x 81920 x 81920, 131072 tokens): every wait in it
    is short, so the limit on waits (2e9 clocks, 1 to 1.5 s) is not met."""
    M, N = 131072, 81920
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    wq = torch.randint(0, 256, (N, N // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand(N, N // 32, generator=g, device="cuda", dtype=torch.float16) * 0.002 + 0.001
    x = torch.empty(M, N, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert bq.bq_device_status() == 0
    h = bq.quant_matmul_glu(x, (wq, s, None), (wq, s, None))
    assert bq.bq_device_status() == 0
    rows = torch.tensor([0, 1, 77777, M - 1], device="cuda")
    for cols in (slice(0, 48), slice(N - 48, N)):
        z, t = sums(x[rows], bq.q4_0_dequantize(wq[cols].contiguous(), s[cols].contiguous()).double(), None)
        a = f("silu", z)
        near(h[rows, cols], a * z, ((1.13 * t + EVAL * (1 + z.abs())) * (z.abs() + t) + a.abs() * t) * (1 + HALF), "h")


def test_calls_on_two_streams_at_once_and_in_forked_captures():
    """A gated forward and a gradient of other weights side by side: on two streams without order
    between them, and as two branches of one captured graph that join before a third call."""
    a, b, down = Case("affine4", 1024, 2048, 300, 2), Case("affine8", 768, 1024, 300, 2, seed=4), Case("q4_0", 2048, 1024, 300, 1, seed=8)
    kw, kb = dict(group_size=a.gs, bits=a.bits), dict(group_size=b.gs, bits=b.bits)
    x, dh, g, u, r = a.rand(300, 2048), b.rand(300, 768), b.rand(300, 768), b.rand(300, 768), a.rand(300, 2048)

    def one():
        return bq.quant_matmul_glu(x, *a.mats, save_preact=True, **kw)

    def two():
        return bq.quant_matmul_glu_backward(dh, g, u, *b.mats, act="gelu", need_dbias=True, **kb)

    def three(h):
        return bq.quant_matmul_act(h, *down.mats[0], residual=r, act="gelu_tanh")

    want1, want2 = one(), two()
    want3 = three(want1[0])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            got.append((one(), want1))
        with torch.cuda.stream(s2):
            got.append((two(), want2))
    torch.cuda.synchronize()
    for t, w in got:
        assert all(torch.equal(p, q) for p, q in zip(t, w))
    del got
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        s2.wait_stream(main)
        with torch.cuda.stream(s2):
            t2 = two()
        t1 = one()
        main.wait_stream(s2)
        t3 = three(t1[0])
    for _ in range(5):
        for t in (*t1, *t2, t3):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*t1, *t2, t3), (*want1, *want2, want3)))
    assert bq.bq_device_status() == 0


FIRST = """
import sys; sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
import bit_quantized_gemm_quant_b200 as bq
from test_epilogue_gpu import Case, feed_forward
torch.cuda.init()
c, down = Case("affine4", 256, 192, {M}, 2), Case("affine4", 192, 256, {M}, 1, seed=9)
x, h0 = c.rand({M}, 192), c.rand({M}, 192)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = feed_forward(c, down, x, h0)
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, feed_forward(c, down, x, h0)))
assert bq.bq_device_status() == 0
"""


@pytest.mark.parametrize("M", [3, 600])
def test_the_first_calls_of_a_process_may_be_captured(M):
    tests = os.path.dirname(os.path.abspath(__file__))
    script = FIRST.format(root=os.path.dirname(tests), tests=tests, M=M)
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("fmt,N,K", [("q4_0", 203, 96), ("affine4", 17, 192), ("affine8", 521, 320), ("affine3", 35, 128)])
def test_nothing_is_written_beside_an_output(fmt, N, K):
    """Every output between 4 KB of a pattern, which stays; gate and up are halves of one matrix."""
    P = ctypes.c_void_p

    def between(*shape):
        n = math.prod(shape)
        buf = torch.full((n + 4096,), -7.0, dtype=torch.bfloat16, device="cuda")
        return buf[2048:2048 + n].view(shape), buf

    for M in (1, 7, 16, 17, 300):
        both = Case(fmt, 8 * N, K, M, 1)
        wq, s, b = both.mats[0]
        at = 7 * N // 8 * 8                                    # every eighth row starts on 16 bytes in every array
        mats = [tuple(None if t is None else t[o:o + N] for t in (wq, s, b)) for o in (0, at)]
        dense = [both.W[0][o:o + N] for o in (0, at)]
        kw = dict(group_size=both.gs, bits=both.bits)
        x, y = both.rand(M, K), both.rand(M, N)
        outs = []
        for call, want in ((lambda o: bq.quant_matmul_act(x, *mats[1], act="relu", out=o, **kw), None),
                           (lambda o: bq.quant_matmul_glu(x, *mats, out=o, **kw), None)):
            o, buf = between(M, N)
            assert torch.equal(call(o), call(None))
            outs.append((o, buf))
        (g, tg), (u, tu) = (sums(x, w, None) for w in dense)
        a = f("silu", g)
        near(outs[1][0], a * u, ((1.13 * tg + EVAL * (1 + g.abs())) * (u.abs() + tu) + a.abs() * tu) * (1 + HALF), "h")
        (dx, b0), (dg, b1), (du, b2), (db0, b3), (db1, b4) = (between(M, K), between(M, N), between(M, N), between(N), between(N))
        pair = [None if p[0] is None else (P * 2)(*(t.data_ptr() for t in p)) for p in zip(*mats)]
        need = bq.quant_matmul_epilogue_workspace_size(bq.OP_GLU_BACKWARD, M, N, K, both.gs, both.bits)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        ptr = [t.data_ptr() for t in (dx, dg, du, db0, db1)]
        st = bq.lib().quant_matmul_glu_backward(y.data_ptr(), y.data_ptr(), y.data_ptr(), *pair, 4, *ptr, M, N, K, both.gs, both.bits,
                                                ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for t, w in zip((dx, dg, du, db0, db1), bq.quant_matmul_glu_backward(y, y, y, *mats, need_dbias=True, **kw)):
            assert torch.equal(t, w)
        for t, buf in (*outs, (dx, b0), (dg, b1), (du, b2), (db0, b3), (db1, b4)):
            assert (buf[:2048] == -7).all() and (buf[2048 + t.numel():] == -7).all(), (M, t.shape)
    assert bq.bq_device_status() == 0
