"""quant_matmul_act, quant_matmul_glu and their gradients against the formulas in 64
bits, over the oracle's bf16 weights.

Tolerances (|.| elementwise, all counted before the first run):
  - an output is rounded once to bf16: half a step, 2^-8 relative;
  - an fp32 sum of n products errs by at most (n + 8) 2^-23 sum |terms| (each addition
    by at most one fp32 step of a partial sum; + 8 for the bias and split additions);
  - act and act' in fp32: an exponential of argument a errs by at most (|a| + 4) 2^-23
    relative, times at most |z| where the sigmoid's slope multiplies it; for the
    arguments here (|a| < 60 wherever the slope is not 0) 2^-17 (1 + |z|) bounds both;
    the slope |act'| is at most 1.13;
  - dx is held to the product of the returned dz (dg, du), dz to the formula.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_gemm_quant_b200 as bq
from _helpers import Problem

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
HALF = 2.0 ** -8
EVAL = 2.0 ** -17


def f(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def df(act, z):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a, da = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        return 0.5 * (1 + torch.tanh(a)) + 0.5 * z * da / torch.cosh(a.clamp(-300, 300)) ** 2
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def near(got, want, slack, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    excess = (got - want).abs() - (HALF * want.abs() + slack + 1e-30)
    assert excess.numel() == 0 or excess.max() <= 0, \
        f"{what}: off by {float(excess.max()):.3e} beyond the tolerance at {int(excess.argmax())}"


class Case:
    """Weights (one or two of one format), their bf16 values in 64 bits, and tokens."""

    def __init__(self, fmt, N, K, M, mats, seed=0):
        self.M, self.N, self.K = M, N, K
        p = [Problem(fmt, N, K, seed=seed + i) for i in range(mats)]
        self.gs, self.bits = p[0].group_size, p[0].bits
        self.mats = [q.device() for q in p]
        self.W = [torch.from_numpy((q.wb.astype(np.uint32) << 16).view(np.float32)).cuda().double() for q in p]
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed + 77)

    def rand(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(torch.bfloat16)


def sums(x, W, bias):
    """(the sum, its error bound) in 64 bits."""
    z, a = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    if bias is not None:
        z, a = z + bias.double(), a + bias.double().abs()
    return z, (W.shape[1] + 8) * 2.0 ** -23 * a


def check_act(c, act, bias=True, res=True, save=False, seed_x=1.0):
    x = c.rand(c.M, c.K, scale=seed_x)
    b = c.rand(c.N) if bias else None
    r = c.rand(c.M, c.N) if res else None
    got = bq.quant_matmul_act(x, *c.mats[0], out_bias=b, act=act, residual=r, group_size=c.gs, bits=c.bits,
                              save_preact=save)
    y, z = got if save else (got, None)
    zr, tz = sums(x, c.W[0], b)
    want = f(act, zr) + (r.double() if res else 0)
    near(y, want, (1.13 * tz + EVAL * (1 + zr.abs())) * (1 + HALF), f"y {act}")
    if save:
        near(z, zr, tz * (1 + HALF), "z")


def check_glu(c, act, bias=False, save=False):
    x = c.rand(c.M, c.K)
    b = [c.rand(c.N) if bias else None for _ in range(2)]
    got = bq.quant_matmul_glu(x, c.mats[0], c.mats[1], b[0], b[1], act, c.gs, c.bits, save)
    h, g, u = got if save else (got, None, None)
    (gr, tg), (ur, tu) = (sums(x, w, v) for w, v in zip(c.W, b))
    fa = f(act, gr)
    slack = (1.13 * tg + EVAL * (1 + gr.abs())) * (ur.abs() + tu) + fa.abs() * tu
    near(h, fa * ur, slack * (1 + HALF), f"h {act}")
    if save:
        near(g, gr, tg * (1 + HALF), "g")
        near(u, ur, tu * (1 + HALF), "u")


def product_bound(ds, Ws):
    want = sum(d.double() @ w for d, w in zip(ds, Ws))
    mags = sum(d.double().abs() @ w.abs() for d, w in zip(ds, Ws))
    return want, (len(ds) * Ws[0].shape[0] + 8) * 2.0 ** -23 * mags * (1 + HALF)


def check_act_bwd(c, act, db=True):
    dy, z = c.rand(c.M, c.N), c.rand(c.M, c.N, scale=2.0)
    got = bq.quant_matmul_act_backward(dy, *c.mats[0], preact=z, act=act, group_size=c.gs, bits=c.bits, need_dbias=db)
    dx, dz = got[:2]
    want = dy.double() * df(act, z.double())
    slack = EVAL * (1 + z.double().abs()) * dy.double().abs()
    near(dz, want, 0 * slack if act in ("none", "relu") else slack, f"dz {act}")
    w, t = product_bound([dz], c.W)
    near(dx, w, t, "dx")
    if db:
        near(got[2], want.sum(0), (slack + (c.M + 8) * 2.0 ** -24 * want.abs().sum(0)).sum(0) if c.M else slack.sum(0),
             "dbias")


def check_glu_bwd(c, act, db=True):
    dh, g, u = c.rand(c.M, c.N), c.rand(c.M, c.N, scale=2.0), c.rand(c.M, c.N)
    got = bq.quant_matmul_glu_backward(dh, g, u, c.mats[0], c.mats[1], act, c.gs, c.bits, db)
    dx, dg, du = got[:3]
    D, G, U = dh.double(), g.double(), u.double()
    wg, wu = D * U * df(act, G), D * f(act, G)
    ev = EVAL * (1 + G.abs()) * D.abs()
    near(dg, wg, ev * U.abs() + 2.0 ** -22 * wg.abs(), "dg")
    near(du, wu, ev, "du")
    w, t = product_bound([dg, du], c.W)
    near(dx, w, t, "dx")
    if db:
        for o, v, e, name in ((got[3], wg, ev * U.abs(), "dgate_bias"), (got[4], wu, ev, "dup_bias")):
            near(o, v.sum(0), e.sum(0) + (c.M + 8) * 2.0 ** -24 * v.abs().sum(0), name)


FMTS = ["q4_0", "affine4", "affine8", "affine4_g32", "affine4_g128", "affine8_g32", "affine8_g128", "affine2", "affine3",
        "affine6", "affine3_g128"]
MS = [1, 2, 5, 8, 9, 16, 20, 21, 33, 64, 129, 300]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(1, 128), (17, 256), (200, 384), (264, 640)])
def test_forms_over_formats_and_tokens(fmt, N, K):
    for i, M in enumerate(MS):
        act = ACTS[(i + N) % 5]
        one, two = Case(fmt, N, K, M, 1, seed=i), Case(fmt, N, K, M, 2, seed=i)
        check_act(one, act, bias=i % 2 == 0, res=i % 3 != 0, save=i % 4 == 1)
        check_glu(two, act, bias=i % 3 == 0, save=i % 2 == 1)
        check_act_bwd(one, act, db=i % 2 == 0)
        check_glu_bwd(two, act, db=i % 3 == 0)
    assert bq.bq_device_status() == 0


@pytest.mark.parametrize("fmt,K", [("q4_0", 32), ("q4_0", 96), ("q4_0", 160), ("affine4", 64), ("affine8", 192), ("affine8_g32", 32),
                                   ("affine2_g32", 32), ("affine3_g32", 32), ("affine6_g32", 96), ("affine4_g32", 224)])
def test_shortest_and_odd_reductions(fmt, K):
    """One block or group of columns and counts that fill no stage, chunk or 16-byte row of scales."""
    for i, M in enumerate((1, 16, 17, 70)):
        for N in (3, 136):
            check_act(Case(fmt, N, K, M, 1, seed=i), ACTS[i + 1], save=True)
            check_glu(Case(fmt, N, K, M, 2, seed=i), "silu", bias=True, save=True)
            check_act_bwd(Case(fmt, N, K, M, 1, seed=i), ACTS[i])
            check_glu_bwd(Case(fmt, N, K, M, 2, seed=i), ACTS[i + 1])
    assert bq.bq_device_status() == 0


def test_outputs_past_32_bit_offsets():
    """70000 x 32768 outputs (2.3e9 elements): the last rows and columns against the formula."""
    M, N, K = 70000, 32768, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    wq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    s = (torch.rand(N, K // 32, generator=g, device="cuda") * 0.02 + 0.01).to(torch.float16)
    W = bq.q4_0_dequantize(wq, s).double()
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    y = bq.quant_matmul_act(x, wq, s, act="silu")
    rows = torch.tensor([0, 1, 65535, 65536, M - 2, M - 1], device="cuda")
    z, t = sums(x[rows], W, None)
    near(y[rows], f("silu", z), (1.13 * t + EVAL * (1 + z.abs())) * (1 + HALF), "y")
    dx, dz = bq.quant_matmul_act_backward(y, wq, s, preact=y, act="relu")
    assert torch.equal(dz[rows], torch.where(y[rows] > 0, y[rows], torch.zeros_like(y[rows])))
    want, t = product_bound([dz[rows]], [W])
    near(dx[rows], want, t, "dx")
    assert bq.bq_device_status() == 0


@pytest.mark.parametrize("act", ACTS)
def test_every_activation_each_way(act):
    for M in (3, 40):
        one, two = Case("q4_0", 96, 160, M, 1), Case("q4_0", 96, 160, M, 2)
        check_act(one, act, save=True)
        check_glu(two, act, bias=True, save=True)
        check_act_bwd(one, act)
        check_glu_bwd(two, act)


@pytest.mark.parametrize("fmt,N,K,M", [("q4_0", 2048, 8192, 1), ("affine4", 1500, 4096, 7), ("affine8", 4100, 2048, 700),
                                       ("q4_0", 8192, 2048, 512), ("affine4", 640, 4096, 1999), ("affine6", 520, 2048, 513)])
def test_larger_products(fmt, N, K, M):
    one, two = Case(fmt, N, K, M, 1), Case(fmt, N, K, M, 2)
    check_act(one, "gelu", save=True)
    check_glu(two, "silu", save=True)
    check_act_bwd(one, "silu")
    check_glu_bwd(two, "gelu_tanh")
    assert bq.bq_device_status() == 0


@pytest.mark.parametrize("fmt", ["q4_0", "affine4", "affine8", "affine8_g32"])
@pytest.mark.parametrize("N,K,M", [(777, 4096, 1100), (640, 4096, 1025), (840, 6144, 2600)])
def test_gradients_with_two_token_tiles_per_unit(fmt, N, K, M):
    """Sizes whose gradient takes both accumulators for one weight tile: a single unit per
    pair of SMs and several, a second tile cut short, rows of dz with and without padding."""
    check_act_bwd(Case(fmt, N, K, M, 1), "silu")
    check_glu_bwd(Case(fmt, N, K, M, 2), "gelu", db=False)
    assert bq.bq_device_status() == 0


@pytest.mark.parametrize("M", [4, 70])
def test_residual_added_in_place(M):
    c = Case("affine4", 200, 256, M, 1)
    x, r = c.rand(M, c.K), c.rand(M, c.N)
    want = bq.quant_matmul_act(x, *c.mats[0], residual=r, group_size=c.gs, bits=c.bits)
    h = r.clone()
    got = bq.quant_matmul_act(x, *c.mats[0], residual=h, group_size=c.gs, bits=c.bits, out=h)
    assert got is h and torch.equal(h, want)


def test_gradients_match_differences_of_the_formula():
    """d/de of sum(v * forward(x + e p)) in 64 bits against the returned gradients."""
    c = Case("affine8", 72, 128, 24, 2)
    x, p = c.rand(c.M, c.K).double(), c.rand(c.M, c.K).double()
    v = c.rand(c.M, c.N)
    for act in ACTS:
        gu = [x @ w.t() for w in c.W]
        g, u = (t.to(torch.bfloat16) for t in gu)
        # the saved factors are rounded: differences of the forward from exactly those values
        step, e = [p @ w.t() for w in c.W], 1e-5
        def loss(s):
            return (v.double() * f(act, g.double() + s * step[0]) * (u.double() + s * step[1])).sum()
        slope = float((loss(e) - loss(-e)) / (2 * e))
        dx, dg, du = bq.quant_matmul_glu_backward(v, g, u, c.mats[0], c.mats[1], act, c.gs, c.bits)
        # dg, du and dx are each off by half a bf16 step of themselves
        room = HALF * ((dx.double() * p).abs().sum() + (dg.double() * step[0]).abs().sum() + (du.double() * step[1]).abs().sum())
        if act == "relu":   # where g +- e step crosses 0 the difference of relu lies in [0, 1] step, the derivative is 0 or 1
            room += ((v.double() * u.double() * step[0]).abs() * (g.double().abs() <= e * step[0].abs())).sum()
        assert abs(float((dx.double() * p).sum()) - slope) <= float(room) + 1e-3 * abs(slope), act


def test_large_and_non_finite_arguments():
    """Saturated activations give their limits, and a non-finite activation stays in its row."""
    N = K = 64
    M = 40
    c = Case("affine8", N, K, M, 2)
    z = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    vals = [0.0, -0.0, 1e-30, 30.0, -30.0, 200.0, -200.0, 3e38, -3e38, float("inf"), float("-inf")]
    z[0, :len(vals)] = torch.tensor(vals)
    dy = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    for act in ACTS[1:]:
        dx, dz = bq.quant_matmul_act_backward(dy, *c.mats[0], preact=z, act=act, group_size=c.gs, bits=c.bits)
        lim = dz[0, :len(vals)].float().tolist()
        at0 = 0.0 if act == "relu" else 0.5
        assert lim[0] == lim[1] == at0 and abs(lim[3] - 1) < 1e-2 and abs(lim[4]) < 1e-2, (act, lim)
        assert lim[5] == lim[7] == lim[9] == 1.0 and lim[6] == lim[8] == lim[10] == 0.0, (act, lim)
    x = c.rand(M, K)
    x[5, 3] = float("nan")
    x[7, 0] = float("inf")
    for act in ACTS:
        y = bq.quant_matmul_act(x, *c.mats[0], act=act, group_size=c.gs, bits=c.bits)
        h = bq.quant_matmul_glu(x, c.mats[0], c.mats[1], act=act, group_size=c.gs, bits=c.bits)
        for o in (y, h):
            assert o[5].isnan().all(), act
            rest = [i for i in range(M) if i not in (5, 7)]
            assert torch.isfinite(o[rest]).all(), act


def test_empty_problems():
    c = Case("q4_0", 32, 64, 4, 1)
    wq, s, _ = c.mats[0]
    assert bq.quant_matmul_act(c.rand(0, 64), wq, s).shape == (0, 32)
    assert bq.quant_matmul_glu(c.rand(0, 64), (wq, s, None), (wq, s, None)).shape == (0, 32)
    nq, ns = wq[:0], s[:0]
    assert bq.quant_matmul_act(c.rand(4, 64), nq, ns).shape == (4, 0)
    dx, dz = bq.quant_matmul_act_backward(c.rand(4, 0), nq, ns, preact=c.rand(4, 0), act="silu")
    assert dx.shape == (4, 64) and not dx.any() and dz.shape == (4, 0)
    db = bq.quant_matmul_act_backward(c.rand(0, 32), wq, s, need_dbias=True)[2]
    assert not db.any()
    kq, ks = wq[:, :0].contiguous(), s[:, :0].contiguous()          # K = 0: z is the bias
    b, r = c.rand(32), c.rand(4, 32)
    y, z = bq.quant_matmul_act(c.rand(4, 0), kq, ks, out_bias=b, act="silu", residual=r, save_preact=True)
    assert torch.equal(z, b.expand(4, 32))
    near(y, f("silu", b.double()) + r.double(), torch.full_like(r.double(), EVAL * 8), "K = 0")
    h = bq.quant_matmul_glu(c.rand(4, 0), (kq, ks, None), (kq, ks, None), b, b)
    near(h, (f("silu", b.double()) * b.double()).expand(4, 32), torch.full_like(r.double(), EVAL * 64), "K = 0")


def test_repeatable_and_independent_of_the_workspace():
    for M in (6, 40, 300):
        c = Case("q4_0", 520, 1024, M, 2)
        x = c.rand(M, c.K)
        a = bq.quant_matmul_glu(x, c.mats[0], c.mats[1])
        dx = bq.quant_matmul_glu_backward(a, a, a, c.mats[0], c.mats[1])[0]
        for _ in range(3):
            junk = torch.full((1 << 24,), 0x7F, dtype=torch.uint8, device="cuda")   # NaN patterns where scratch may land
            del junk
            assert torch.equal(bq.quant_matmul_glu(x, c.mats[0], c.mats[1]), a)
            assert torch.equal(bq.quant_matmul_glu_backward(a, a, a, c.mats[0], c.mats[1])[0], dx)


def feed_forward(c, down, x, h0):
    """A gated feed-forward and its gradient, as a layer runs it."""
    h, g, u = bq.quant_matmul_glu(x, c.mats[0], c.mats[1], save_preact=True, group_size=c.gs, bits=c.bits)
    y = bq.quant_matmul_act(h, *down.mats[0], residual=h0, group_size=c.gs, bits=c.bits)
    dh, _ = bq.quant_matmul_act_backward(y, *down.mats[0], group_size=c.gs, bits=c.bits)
    dx, dg, du = bq.quant_matmul_glu_backward(dh, g, u, c.mats[0], c.mats[1], group_size=c.gs, bits=c.bits)
    return y, dx, dg, du


@pytest.mark.parametrize("M", [3, 37, 600])
def test_feed_forward_on_streams_and_in_graphs(M):
    """The four calls chained: on another stream, captured and replayed with new inputs,
    two graphs and an eager run in any order, the same bits each time."""
    c, down = Case("affine4", 256, 192, M, 2), Case("affine4", 192, 256, M, 1, seed=9)
    x, h0 = c.rand(M, 192), c.rand(M, 192)
    want = [t.clone() for t in feed_forward(c, down, x, h0)]
    z = h0.double() + (f("silu", x.double() @ c.W[0].t()) * (x.double() @ c.W[1].t())) @ down.W[0].t()
    assert float((want[0].double() - z).norm() / z.norm()) < 0.02
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, g, u = bq.quant_matmul_glu(x, c.mats[0], c.mats[1], save_preact=True, group_size=c.gs, bits=c.bits, stream=s)
    y = bq.quant_matmul_act(h, *down.mats[0], residual=h0, group_size=c.gs, bits=c.bits, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want[0])
    x2 = torch.zeros_like(x)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = feed_forward(c, down, x2, h0)
        graphs.append((gr, outs))
    for i in (0, 1, 1, 0):
        x2.copy_(x)
        graphs[i][0].replay()
        graphs[1 - i][0].replay()
        again = feed_forward(c, down, x, h0)
        torch.cuda.synchronize()
        for outs in (graphs[0][1], graphs[1][1], again):
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
    assert bq.bq_device_status() == 0


def test_binding_checks_its_tensors():
    c = Case("affine4", 64, 128, 4, 2)
    wq, s, b = c.mats[0]
    x = c.rand(4, 128)
    kw = dict(group_size=c.gs, bits=c.bits)
    with pytest.raises(ValueError, match="act"):
        bq.quant_matmul_act(x, wq, s, b, act="tanh", **kw)
    with pytest.raises(ValueError, match="w.wq"):
        bq.quant_matmul_act(x[:, :64].contiguous(), wq, s, b, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        bq.quant_matmul_act(c.rand(128, 4).t(), wq, s, b, **kw)
    with pytest.raises(ValueError, match="residual"):
        bq.quant_matmul_act(x, wq, s, b, residual=c.rand(1, 64), **kw)
    with pytest.raises(TypeError, match="residual"):
        bq.quant_matmul_act(x, wq, s, b, residual=torch.zeros(4, 64, device="cuda"), **kw)
    with pytest.raises(ValueError, match="out_bias"):
        bq.quant_matmul_act(x, wq, s, b, out_bias=c.rand(63), **kw)
    with pytest.raises(ValueError, match="both"):
        bq.quant_matmul_glu(x, c.mats[0], (wq, s, None), **kw)
    with pytest.raises(ValueError, match="preact"):
        bq.quant_matmul_act_backward(c.rand(4, 64), wq, s, b, act="silu", **kw)
    with pytest.raises(ValueError, match="up.wq"):
        bq.quant_matmul_glu(x, c.mats[0], tuple(t[:32].contiguous() for t in c.mats[1]), **kw)
    with pytest.raises(ValueError, match="cpu"):
        bq.quant_matmul_act(x, wq, s, b, out_bias=torch.zeros(64, dtype=torch.bfloat16), **kw)
    # a workspace one byte short is refused, one of the reported size is enough
    dy, dx = c.rand(4, 64), torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    need = bq.quant_matmul_epilogue_workspace_size(bq.OP_ACT_BACKWARD, 4, 64, 128, 64, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    def raw(n):
        return bq.lib().quant_matmul_act_backward(dy.data_ptr(), None, wq.data_ptr(), s.data_ptr(), b.data_ptr(), 0,
                                                  dx.data_ptr(), None, None, 4, 64, 128, 64, 4, ws.data_ptr(), n,
                                                  torch.cuda.current_stream().cuda_stream)
    assert raw(need - 1) == 7 and raw(need) == 0
    assert torch.equal(dx, bq.quant_matmul_act_backward(dy, wq, s, b, **kw)[0])
