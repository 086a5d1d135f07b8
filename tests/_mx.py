"""The microscaled formats and the norm by their definitions in 64 bits, for the tests."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
TOP = {8: 8, 4: 2}
LARGEST = {8: 448.0, 4: 6.0}


def scale_bytes(v, bits):
    """E8M0 bytes of fp64 rows [M][K]; 255 where a block holds a NaN or an infinity."""
    b = v.double().reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    e = torch.frexp(torch.where(bad, 1.0, amax))[1] - 1 - TOP[bits] + 127
    e = torch.where(amax == 0, 0, e).clamp(min=0)
    return torch.where(bad, 255, e).to(torch.uint8)


def power(byte):
    p = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64, device=byte.device), byte.int() - 127)
    return torch.where(byte == 255, float("nan"), p)


def rounded(t, bits):
    """fp64 to the nearest value of the element type, ties to even, saturated."""
    t = t.clamp(-LARGEST[bits], LARGEST[bits])
    digits, lowest = (3, -9) if bits == 8 else (1, -1)
    unit = torch.ldexp(torch.ones_like(t), (torch.frexp(t)[1] - 1 - digits).clamp(min=lowest))
    return torch.round(t / unit) * unit


def quantized(v, bits, byte=None):
    """(element values fp64 [M][K], scale bytes) of rows."""
    byte = scale_bytes(v, bits) if byte is None else byte
    b = v.double().reshape(v.shape[0], -1, 32)
    t = torch.where((byte == 255)[..., None], 0.0, b / power(byte)[..., None])
    return rounded(t, bits).reshape(v.shape), byte


def elements(codes):
    """fp64 element values of codes as the library stores them."""
    if codes.dtype == torch.uint8:
        grid = torch.cat([GRID, -GRID]).to(codes.device)
        return torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], 2).reshape(codes.shape[0], -1)
    return codes.float().double()


def values(codes, scales):
    """fp64 values of microscaled rows."""
    e = elements(codes)
    return (e.view(e.shape[0], -1, 32) * power(scales.view(torch.uint8))[..., None]).reshape(e.shape)


def random_codes(rows, K, bits, gen, spread=6, device="cuda"):
    """Random codes (every finite one) and scales 2^-spread .. 2^spread."""
    scales = torch.randint(127 - spread, 128 + spread, (rows, K // 32), generator=gen, device=device, dtype=torch.uint8)
    if bits == 4:
        codes = torch.randint(0, 256, (rows, K // 2), generator=gen, device=device, dtype=torch.uint8)
    else:
        codes = torch.randint(0, 256, (rows, K), generator=gen, device=device, dtype=torch.uint8)
        codes = torch.where((codes & 127) == 127, codes - 1, codes).view(torch.float8_e4m3fn)
    return codes, scales.view(torch.float8_e8m0fnu)
