"""Cases and plain forms of the fused-epilogue operators over quantized weights.

  quant_matmul_act            z = x . W^T + b,  y = r + act(z)
  quant_matmul_act_backward   dz = dy act'(z),  dx = dz . W,  db = sum over tokens of dy act'(z)
  quant_matmul_glu            g = x . Wg^T + bg,  u = x . Wu^T + bu,  h = act(g) u
  quant_matmul_glu_backward   dg = dh u act'(g),  du = dh act(g),  dx = dg . Wg + du . Wu,  dbg, dbu sums over tokens

x, r, dy, dh and the saved z, g, u are bf16; W is Q4_0 or affine (2, 3, 4, 6 or 8 bits), and stands for the bf16
matrix that the library's dequantizers give.  Every output is bf16.  The gradient product takes dz (dg, du) as
returned, so that it is the product of what the caller gets.
"""
import math

import torch

own = False

FORMATS = {  # name: (group size, bits); Q4_0 has no biases
    "q4_0": (32, 4), "affine4": (64, 4), "affine8": (64, 8), "affine4_g32": (32, 4), "affine4_g128": (128, 4),
    "affine8_g32": (32, 8), "affine8_g128": (128, 8), "affine2": (64, 2), "affine3": (64, 3), "affine6": (64, 6),
}


def listed():
    return [
        # one small product: latency of a call (the repository's 16 x 256 x 512 problem)
        dict(name="act_small_m16", op="act", fmt="q4_0", M=16, N=256, K=512, act="gelu_tanh", bias=True, res=False, save=False),
        # one token's down projection added to the residual stream (Llama-3.2-1B feed-forward)
        dict(name="act_down_m1", op="act", fmt="q4_0", M=1, N=2048, K=8192, act="none", bias=False, res=True, save=False),
        # a prompt's up projection with bias and activation (12288 x 4096 MLP, 512 tokens)
        dict(name="act_up_m512", op="act", fmt="affine4", M=512, N=12288, K=4096, act="gelu", bias=True, res=False, save=False),
        # training forward of an output projection, odd token count, 8-bit weights, pre-activation kept
        dict(name="act_train_m1999", op="act", fmt="affine8", M=1999, N=4096, K=4096, act="silu", bias=True, res=True, save=True),
        # one token's gated feed-forward (Llama-3.2-1B)
        dict(name="glu_m1", op="glu", fmt="q4_0", M=1, N=8192, K=2048, act="silu", bias=False, save=False),
        # a batch of eight tokens on the wide MLP
        dict(name="glu_m8", op="glu", fmt="affine4", M=8, N=12288, K=4096, act="gelu_tanh", bias=False, save=False),
        # a 512-token prompt's gated feed-forward (Llama-3.2-1B)
        dict(name="glu_m512", op="glu", fmt="q4_0", M=512, N=8192, K=2048, act="silu", bias=False, save=False),
        # training forward of the wide MLP: the largest
        dict(name="glu_train_m2048", op="glu", fmt="affine4", M=2048, N=12288, K=4096, act="silu", bias=False, save=True),
        # gradient of the down projection, a short ragged batch
        dict(name="act_bwd_m300", op="act_bwd", fmt="q4_0", M=300, N=2048, K=8192, act="none", bias=True),
        # gradient through an activation, 8-bit weights
        dict(name="act_bwd_m2048", op="act_bwd", fmt="affine8", M=2048, N=12288, K=4096, act="gelu", bias=True),
        # gradient of the gated feed-forward (Llama-3.2-1B, 512 tokens)
        dict(name="glu_bwd_m512", op="glu_bwd", fmt="q4_0", M=512, N=8192, K=2048, act="silu", bias=False),
        # gradient of the wide gated MLP over a training batch
        dict(name="glu_bwd_m2048", op="glu_bwd", fmt="affine4", M=2048, N=12288, K=4096, act="silu", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["act", "act", "glu", "glu", "act_bwd", "glu_bwd"])
        fmt = rng.choice(["q4_0", "affine4", "affine8", "q4_0", "affine4", "affine8"] + sorted(FORMATS))
        unit = max(FORMATS[fmt][0], 32)
        case = dict(op=op, fmt=fmt, M=_log(rng, 1, 4096), N=_log(rng, 40, 12288), K=unit * max(1, _log(rng, 128, 8192) // unit),
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"] if op.startswith("act") else ["relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5)
        if rng.random() < 0.5:
            case["N"] = max(64, case["N"] // 64 * 64)
        if op == "act":
            case["res"] = rng.random() < 0.5
        if op in ("act", "glu"):
            case["save"] = rng.random() < 0.4
        if work(case)["flops"] <= 4 * 2048 * 12288 * 4096 and case["M"] * case["N"] >= 64:
            return case


def _packed_bytes(case):
    gs, bits = FORMATS[case["fmt"]]
    per = 2 if case["fmt"] == "q4_0" else 4
    return case["N"] * case["K"] * bits // 8 + case["N"] * (case["K"] // gs) * per


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    mats = 2 if op.startswith("glu") else 1
    tok = 2 * M * N  # bytes of one [M][N] bf16 matrix
    n = mats * _packed_bytes(case) + 2 * M * K
    if op == "act":
        n += tok * (1 + bool(case["res"]) + bool(case["save"])) + 2 * N * bool(case["bias"])
    elif op == "glu":
        n += tok * (3 if case["save"] else 1) + 4 * N * bool(case["bias"])
    elif op == "act_bwd":
        n += tok * (1 if case["act"] == "none" else 3) + 2 * N * bool(case["bias"])
    else:
        n += tok * 5 + 4 * N * bool(case["bias"])
    return {"bytes": n, "flops": 2 * mats * M * N * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    def quantize(fmt, w):
        """w fp32 [N][K] -> (codes, scales, biases | None) in the library's layouts."""
        gs, bits = FORMATS[fmt]
        N, K = w.shape
        if fmt == "q4_0":
            b = w.view(N, K // 32, 32)
            top = b.gather(2, b.abs().argmax(2, keepdim=True))
            d = top / -8
            q = torch.where(d == 0, 8.0, torch.clamp(torch.trunc(b / torch.where(d == 0, 1.0, d) + 8.5), 0, 15)).to(torch.uint8)
            return (q[..., :16] | (q[..., 16:] << 4)).reshape(N, K // 2).contiguous(), d.view(N, K // 32).to(torch.float16), None
        b = w.to(torch.bfloat16).float().view(N, K // gs, gs)
        lo, hi = b.amin(2, keepdim=True), b.amax(2, keepdim=True)
        top = (1 << bits) - 1
        s, z = ((hi - lo) / top).to(torch.bfloat16), lo.to(torch.bfloat16)
        q = torch.clamp(torch.round((b - z.float()) / torch.where(s == 0, 1.0, s.float())), 0, top).to(torch.int32)
        q = q.view(N, K // 32, 32)
        words = torch.zeros(N, K // 32, bits, dtype=torch.int32, device=w.device)
        for e in range(32):  # a little-endian bit stream: code e at bits bits*e .. bits*e + bits - 1
            i, sh = bits * e // 32, bits * e % 32
            words[..., i] |= q[..., e] << sh
            if sh + bits > 32:
                words[..., i + 1] |= q[..., e] >> (32 - sh)
        return words.view(N, K * bits // 32), s.view(N, K // gs), z.view(N, K // gs)

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    mats = [quantize(case["fmt"], rand(N, K, scale=0.02)) for _ in range(2 if op.startswith("glu") else 1)]
    s = {"case": dict(case), "mats": mats}
    b16 = torch.bfloat16
    if op in ("act", "glu"):
        s["x"] = rand(M, K).to(b16)
        s["bias"] = [rand(N, scale=0.5).to(b16) for _ in mats] if case["bias"] else [None for _ in mats]
        s["res"] = rand(M, N).to(b16) if case.get("res") else None
    else:
        s["dy"] = rand(M, N).to(b16)
        s["pre"] = [rand(M, N, scale=0.02 * math.sqrt(K)).to(b16) for _ in mats]
    return s


# ------------------------------------------------------------------ plain forms
def _dense(fmt, mat):
    """The bf16 weights of the library's dequantizers, as fp32."""
    gs, bits = FORMATS[fmt]
    wq, s, z = mat
    N = wq.shape[0]
    if z is None:
        b = wq.view(N, -1, 16)
        q = torch.cat([b & 15, b >> 4], 2).float() - 8
        return (q * s.float()[..., None]).view(N, -1).to(torch.bfloat16).float()
    if 32 % bits == 0:
        q = (wq[..., None] >> torch.arange(0, 32, bits, device=wq.device, dtype=torch.int32)) & ((1 << bits) - 1)
    else:
        at = torch.arange(0, wq.shape[1] * 32, bits, device=wq.device)
        lo = wq.long()[:, at // 32] & 0xFFFFFFFF
        hi = wq.long()[:, torch.clamp(at // 32 + 1, max=wq.shape[1] - 1)]
        q = ((lo >> (at % 32)) | torch.where(at % 32 + bits > 32, hi << (32 - at % 32), 0)) & ((1 << bits) - 1)
    q = q.reshape(N, -1, gs).float()
    return (s.float()[..., None] * q + z.float()[..., None]).view(N, -1).to(torch.bfloat16).float()


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _dact(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _b(t):
    return t.to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    fmt, op = c["fmt"], c["op"]
    W = [_dense(fmt, m) for m in s["mats"]]
    if op in ("act", "glu"):
        x = s["x"].float()
        z = [x @ w.t() if b is None else x @ w.t() + b.float() for w, b in zip(W, s["bias"])]
        if op == "act":
            y = _act(c["act"], z[0]) if s["res"] is None else s["res"].float() + _act(c["act"], z[0])
        else:
            y = _act(c["act"], z[0]) * z[1]
        return [_b(y)] + ([_b(v) for v in z] if c["save"] else [])
    dy, pre = s["dy"].float(), [p.float() for p in s["pre"]]
    if op == "act_bwd":
        d = [dy * _dact(c["act"], pre[0])]
    else:
        d = [dy * pre[1] * _dact(c["act"], pre[0]), dy * _act(c["act"], pre[0])]
    db = [_b(v.sum(0)) for v in d] if c["bias"] else []
    d = [_b(v) for v in d]
    dx = d[0].float() @ W[0] if op == "act_bwd" else d[0].float() @ W[0] + d[1].float() @ W[1]
    return [_b(dx)] + d + db


def run(s):
    if not own:
        return _plain(s)
    import bit_quantized_gemm_quant_b200 as bq
    c = s["case"]
    gs, bits = FORMATS[c["fmt"]]
    op, m = c["op"], s["mats"]
    if op == "act":
        r = bq.quant_matmul_act(s["x"], *m[0], out_bias=s["bias"][0], act=c["act"], residual=s["res"], group_size=gs, bits=bits,
                                save_preact=c["save"])
        return list(r) if c["save"] else [r]
    if op == "glu":
        r = bq.quant_matmul_glu(s["x"], m[0], m[1], gate_bias=s["bias"][0], up_bias=s["bias"][1], act=c["act"], group_size=gs,
                                bits=bits, save_preact=c["save"])
        return list(r) if c["save"] else [r]
    if op == "act_bwd":
        r = bq.quant_matmul_act_backward(s["dy"], *m[0], preact=s["pre"][0], act=c["act"], group_size=gs, bits=bits, need_dbias=c["bias"])
    else:
        r = bq.quant_matmul_glu_backward(s["dy"], s["pre"][0], s["pre"][1], m[0], m[1], act=c["act"], group_size=gs, bits=bits,
                                         need_dbias=c["bias"])
    return list(r)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    gs, bits = FORMATS[case["fmt"]]
    N, K, op, act = case["N"], case["K"], case["op"], case["act"]

    def weights(mat):
        codes, scale, zero = mat
        by = codes.view(torch.uint8).view(N, -1)
        if zero is None:
            q = torch.empty(N, K // 32, 32, dtype=torch.float64, device=by.device)
            q[:, :, :16] = (by.view(N, K // 32, 16) % 16).double()
            q[:, :, 16:] = (by.view(N, K // 32, 16) // 16).double()
            w = (q - 8) * scale.double()[:, :, None]
        else:
            k = torch.arange(gs, device=by.device)
            q = torch.zeros(N, K // gs, gs, dtype=torch.float64, device=by.device)
            grouped = by.view(N, K // gs, gs * bits // 8)
            for j in range(bits):  # bit j of each code, from the byte that holds it
                at = k * bits + j
                q += ((grouped[:, :, at // 8] >> (at % 8).to(torch.uint8)) & 1).double() * 2.0 ** j
            w = q * scale.double()[:, :, None] + zero.double()[:, :, None]
        return w.view(N, K).to(torch.bfloat16).double()

    def phi(z):
        return 0.5 * torch.erfc(-z / math.sqrt(2.0))

    def f(z):
        if act == "none":
            return z
        if act == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if act == "silu":
            return z * torch.sigmoid(z)
        if act == "gelu":
            return z * phi(z)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))  # (1 + tanh a) / 2 = sigmoid(2 a)

    def df(z):
        if act == "none":
            return torch.ones_like(z)
        if act == "relu":
            return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
        if act == "silu":
            return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        if act == "gelu":
            return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        a = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(a * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * a * (1 + 0.134145 * z ** 2)

    W = [weights(m) for m in s["mats"]]
    if op in ("act", "glu"):
        z = [s["x"].double() @ w.t() for w in W]
        z = [v if b is None else v + b.double() for v, b in zip(z, s["bias"])]
        y = f(z[0]) if op == "act" else f(z[0]) * z[1]
        if op == "act" and s["res"] is not None:
            y = y + s["res"].double()
        return [y] + (z if case["save"] else [])
    dy, pre = s["dy"].double(), [p.double() for p in s["pre"]]
    d = [dy * df(pre[0])] if op == "act_bwd" else [dy * pre[1] * df(pre[0]), dy * f(pre[0])]
    dx = sum(v.to(torch.bfloat16).double() @ w for v, w in zip(d, W))
    return [dx] + d + ([v.sum(0) for v in d] if case["bias"] else [])
