"""Cases and plain forms of the microscaled formats, their product and gradient, and the norm that feeds it.

Microscaled (MX) rows: blocks of 32 consecutive elements share a power of two 2^e, held in 8 bits (E8M0: e + 127);
an element is the nearest value of its small type to v / 2^e, ties to the even code, beyond the type's largest value
that value.  e = floor(log2(largest |v| of the block)) - top, at least -127 (-127 for a block of zeros).

  mxfp8          elements E4M3 (top = 8, largest 448)
  mxfp4          elements E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (top = 2); two per byte, the first one low

  mxfp8_quantize, mxfp4_quantize, mxfp4_dequantize
  mx_matmul              y = x . W^T for microscaled x (8 or 4 bits) and W (4 bits), rounded once to bf16
  mx_matmul_backward     dx = dy . W for bf16 dy and frozen W
  add_rms_norm           h = bf16(x + r),  s = 1 / sqrt(mean(h^2) + eps),  y = h s w, as bf16 or as MX rows of the unrounded y
  add_rms_norm_backward  dx = dh + s (g - h s^2 mean(g h)) with g = dy w,  dw = sum over tokens of dy h s
"""
import math

import torch

own = False

EPS = 1e-5
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations to 8 bits (Llama-3.2-1B hidden width): latency of a call
        dict(name="quant8_m1", op="quant8", M=1, K=2048, f32=False),
        # a weight matrix to 4 bits and back, as when weights are rounded in place (12288 x 4096 MLP)
        dict(name="round4_weights", op="round4", M=12288, K=4096, f32=True),
        # one token's down projection (Llama-3.2-1B feed-forward), 8-bit activations
        dict(name="mm_a8_m1", op="mm", M=1, N=2048, K=8192, a=8),
        # a 512-token prompt's up projection (Llama-3.2-1B), 8-bit activations
        dict(name="mm_a8_m512", op="mm", M=512, N=8192, K=2048, a=8),
        # a ragged batch through an output projection, 4-bit activations
        dict(name="mm_a4_m1999", op="mm", M=1999, N=4096, K=4096, a=4),
        # a large batch of the wide MLP, 4-bit activations: the largest
        dict(name="mm_a4_m2048", op="mm", M=2048, N=12288, K=4096, a=4),
        # gradient of the down projection over frozen weights, a short ragged batch
        dict(name="mm_bwd_m300", op="mm_bwd", M=300, N=2048, K=8192),
        # gradient of the wide MLP's projection over a training batch
        dict(name="mm_bwd_m2048", op="mm_bwd", M=2048, N=12288, K=4096),
        # one token: the residual stream is advanced, normed and handed on in 8 bits
        dict(name="norm_m1", op="norm", M=1, K=2048, res=True, out="mxfp8"),
        # a batch of 2048 tokens of the wide model, the same
        dict(name="norm_m2048", op="norm", M=2048, K=4096, res=True, out="mxfp8"),
        # norm's gradient over a short ragged batch
        dict(name="norm_bwd_m333", op="norm_bwd", M=333, K=2048, dh=True),
        # norm's gradient over a training batch, wide rows
        dict(name="norm_bwd_m2048", op="norm_bwd", M=2048, K=8192, dh=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["mm", "mm", "mm", "mm_bwd", "norm", "norm", "norm_bwd", "quant8", "round4"])
        K = 32 * max(1, _log(rng, 128, 8192) // 32)
        if op == "mm":
            case = dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 40, 12288), K=K, a=rng.choice([8, 8, 4]))
            if rng.random() < 0.5:  # half of the widths are whole tiles
                case["N"], case["K"] = max(64, case["N"] // 64 * 64), max(128, K // 128 * 128)
        elif op == "mm_bwd":
            case = dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 40, 12288), K=K)
            if rng.random() < 0.5:
                case["N"] = max(64, case["N"] // 64 * 64)
        elif op == "norm":
            out = rng.choice(["bf16", "mxfp8", "mxfp8", "mxfp4"])
            case = dict(op=op, M=_log(rng, 1, 8192), K=K, res=rng.random() < 0.7, out=out)
            if out == "bf16" and rng.random() < 0.4:  # any width
                case["K"] = _log(rng, 33, 12288)
        elif op == "norm_bwd":
            case = dict(op=op, M=_log(rng, 1, 8192), K=K if rng.random() < 0.6 else _log(rng, 33, 12288), dh=rng.random() < 0.6)
        else:
            case = dict(op=op, M=_log(rng, 1, 12288), K=K, f32=rng.random() < 0.5)
        w = work(case)
        if w["flops"] <= 2 * 2048 * 12288 * 4096 and w["bytes"] <= 3e8 and case["M"] * K >= 64:
            return case


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op in ("quant8", "round4"):
        out = M * K + M * K // 32 if op == "quant8" else 2 * M * K
        return {"bytes": M * K * (4 if case["f32"] else 2) + out, "flops": 4 * M * K}
    if op == "norm":
        out = {"bf16": 2 * M * K, "mxfp8": M * K + M * K // 32, "mxfp4": M * K // 2 + M * K // 32}[case["out"]]
        return {"bytes": M * K * (6 if case["res"] else 2) + 2 * K + 4 * M + out, "flops": 6 * M * K}
    if op == "norm_bwd":
        return {"bytes": M * K * (8 if case["dh"] else 6) + 4 * K + 4 * M, "flops": 10 * M * K}
    N = case["N"]
    weights = N * K // 2 + N * K // 32
    if op == "mm":
        return {"bytes": weights + M * K * case["a"] // 8 + M * K // 32 + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": weights + 2 * M * N + 2 * M * K, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    b16 = torch.bfloat16

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def channels(n):
        """Per-channel spread of activations: most near 1, a few channels large."""
        return torch.exp(rand(n, scale=0.7))

    def packed(v, bits):
        """Rows of microscaled codes of v, in a user's layout: (codes, scales)."""
        top, f8 = (2, None) if bits == 4 else (8, torch.float8_e4m3fn)
        blocks = v.float().view(v.shape[0], -1, 32)
        bits_of = blocks.abs().amax(2).view(torch.int32) >> 23
        e = torch.clamp(bits_of - top, min=0)  # the scale's byte
        t = blocks * torch.exp2(127.0 - e.float())[..., None]
        scales = e.to(torch.uint8).view(torch.float8_e8m0fnu)
        if bits == 8:
            return t.clamp(-448, 448).to(f8).view(v.shape), scales
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
        code = torch.bucketize(t.abs(), mid).to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)
        code = code.view(v.shape[0], -1, 2)
        return (code[..., 0] | (code[..., 1] << 4)).contiguous(), scales

    s = {"case": dict(case)}
    if op == "quant8":
        s["x"] = rand(M, K) * channels(K)
    elif op == "round4":
        s["x"] = rand(M, K, scale=0.02)
    elif op == "mm":
        s["w"] = packed(rand(case["N"], K, scale=0.02), 4)
        s["x"] = packed(rand(M, K) * channels(K), case["a"])
    elif op == "mm_bwd":
        s["w"] = packed(rand(case["N"], K, scale=0.02), 4)
        s["dy"] = rand(M, case["N"]).to(b16)
    else:
        s["weight"] = (1 + rand(K, scale=0.2)).to(b16)
        s["x"] = (rand(M, K, scale=2.0) * channels(K)).to(b16)
        if op == "norm":
            s["res"] = (rand(M, K, scale=4.0) * channels(K)).to(b16) if case["res"] else None
        else:
            s["rstd"] = 1 / torch.sqrt(s["x"].double().square().mean(1) + EPS)
            s["rstd"] = s["rstd"].float()
            s["dy"] = rand(M, K).to(b16)
            s["dh"] = rand(M, K).to(b16) if case["dh"] else None
    if op in ("quant8", "round4") and not case["f32"]:
        s["x"] = s["x"].to(b16)
    return s


# ------------------------------------------------------------------ plain forms
def _power(byte):
    """2^(byte - 127)"""
    b = byte.int()
    return torch.where(b > 0, (b << 23).view(torch.float32), 2.0 ** -127)


def _scale_byte(blocks, top):
    return torch.clamp((blocks.abs().amax(2).view(torch.int32) >> 23) - top, min=0)


def _mxfp8(v):
    """fp32 rows to (E4M3 values of the elements, scales)."""
    blocks = v.view(v.shape[0], -1, 32)
    e = _scale_byte(blocks, 8)
    t = (blocks / _power(e)[..., None]).clamp(-448, 448)
    return t.to(torch.float8_e4m3fn).view(v.shape), e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _mxfp4(v):
    """fp32 rows to the bf16 values that their microscaled codes stand for."""
    blocks = v.view(v.shape[0], -1, 32)
    p = _power(_scale_byte(blocks, 2))[..., None]
    t = (blocks / p).clamp(-6, 6)
    step = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0))
    return (torch.round(t / step) * step * p).view(v.shape).to(torch.bfloat16)


def _values(codes, scales):
    """The fp32 values of microscaled rows."""
    p = _power(scales.view(torch.uint8))
    if codes.dtype == torch.uint8:
        grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
        v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], 2)
    else:
        v = codes.float()
    return (v.view(codes.shape[0], -1, 32) * p[..., None]).view(codes.shape[0], -1)


def _plain(s):
    c, b16 = s["case"], torch.bfloat16
    op = c["op"]
    if op == "quant8":
        return list(_mxfp8(s["x"].float()))
    if op == "round4":
        return [_mxfp4(s["x"].float())]
    if op == "mm":
        return [(_values(*s["x"]) @ _values(*s["w"]).t()).to(b16)]
    if op == "mm_bwd":
        return [(s["dy"].float() @ _values(*s["w"])).to(b16)]
    w = s["weight"].float()
    if op == "norm":
        h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(b16)
        hf = h.float()
        rstd = 1 / torch.sqrt((hf * hf).mean(1) + EPS)
        y = hf * rstd[:, None] * w
        out = [y.to(b16)] if c["out"] == "bf16" else list(_mxfp8(y)) if c["out"] == "mxfp8" else [_mxfp4(y)]
        return out + [rstd] + ([h] if c["res"] else [])
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * w
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(b16), (dy * h * rstd).sum(0).to(b16)]


def run(s):
    if not own:
        return _plain(s)
    import bit_quantized_gemm_quant_b200 as bq
    c = s["case"]
    op = c["op"]
    if op == "quant8":
        return list(bq.mxfp8_quantize(s["x"]))
    if op == "round4":
        return [bq.mxfp4_dequantize(*bq.mxfp4_quantize(s["x"]))]
    if op == "mm":
        return [bq.mx_matmul(*s["x"], *s["w"])]
    if op == "mm_bwd":
        return [bq.mx_matmul_backward(s["dy"], *s["w"])]
    if op == "norm":
        y, h, rstd = bq.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS,
                                     quantize=None if c["out"] == "bf16" else c["out"], save_rstd=True)
        out = [y] if c["out"] == "bf16" else list(y) if c["out"] == "mxfp8" else [bq.mxfp4_dequantize(*y)]
        return out + [rstd] + ([h] if c["res"] else [])
    return list(bq.add_rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["dh"]))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, M, K = case["op"], case["M"], case["K"]

    def microscale(v, top, largest, digits, lowest):
        """(elements, scales) of fp64 rows: elements with `digits` bits behind the leading one, none finer than 2^lowest."""
        b = v.reshape(v.shape[0], -1, 32)
        e = (torch.frexp(b.abs().amax(2))[1] - 1 - top).clamp(min=-127)
        e = torch.where(b.abs().amax(2) == 0, torch.full_like(e, -127), e)
        scale = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)
        t = (b / scale[:, :, None]).clamp(-largest, largest)
        unit = torch.ldexp(torch.ones_like(t), (torch.frexp(t)[1] - 1 - digits).clamp(min=lowest))
        return torch.round(t / unit) * unit, scale

    def whole(t, scale):
        return (t * scale[:, :, None]).view(M, K)

    def stands_for(codes, scales):
        e = scales.view(torch.uint8).double() - 127
        if codes.dtype == torch.uint8:
            q = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
            q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
            sign, mag = 1 - 2 * (q >= 8).double(), q % 8
            ex, man = torch.floor(mag / 2), mag % 2
            v = sign * torch.where(ex == 0, man / 2, torch.pow(2.0, ex - 1) * (1 + man / 2))
        else:
            v = codes.double()
        return v * torch.pow(2.0, e).repeat_interleave(32, dim=1)

    if op == "quant8":
        t, scale = microscale(s["x"].double(), 8, 448.0, 3, -9)
        return [t.view(M, K), scale]
    if op == "round4":
        return [whole(*microscale(s["x"].double(), 2, 6.0, 1, -1))]
    if op == "mm":
        return [stands_for(*s["x"]) @ stands_for(*s["w"]).T]
    if op == "mm_bwd":
        return [s["dy"].double() @ stands_for(*s["w"])]
    w, x = s["weight"].double(), s["x"].double()
    if op == "norm":
        h = x if s["res"] is None else (x + s["res"].double()).to(torch.bfloat16).double()
        rstd = torch.rsqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / K + EPS)
        y = torch.einsum("mk,m,k->mk", h, rstd, w)
        if case["out"] == "bf16":
            out = [y]
        elif case["out"] == "mxfp8":
            t, scale = microscale(y, 8, 448.0, 3, -9)
            out = [t.view(M, K), scale]
        else:
            out = [whole(*microscale(y, 2, 6.0, 1, -1))]
        return out + [rstd] + ([h] if case["res"] else [])
    n = x * s["rstd"].double()[:, None]  # the normed rows; y = n w
    dn = s["dy"].double() * w
    dx = (dn - n * torch.linalg.vecdot(dn, n)[:, None] / K) * s["rstd"].double()[:, None]
    return [dx if s["dh"] is None else dx + s["dh"].double(), torch.einsum("mk,mk->k", s["dy"].double(), n)]
