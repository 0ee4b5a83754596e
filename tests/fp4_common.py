"""Microscaled 4-bit floating point from its definition, in float64, for the tests."""
import torch

MX, NV = torch.float8_e8m0fnu, torch.float8_e4m3fn
BLOCK = {MX: 32, NV: 16}
MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def power_of_two(e):
    """2 ** e in float64 for whole e, from the format's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def binade(v):
    """The e of 2 ** e <= v < 2 ** (e + 1), for v > 0."""
    e = v.log2().round()
    return e - (power_of_two(e) > v).double()


def scale_values(scales):
    """What scales stand for, in float64 (E4M3 without their signs)."""
    b = scales.view(torch.uint8).long()
    if scales.dtype == MX:
        v = power_of_two(b - 127)
        return torch.where(b == 255, torch.full_like(v, float("nan")), v)
    b = b & 127
    e, m = b >> 3, (b & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * power_of_two(e - 7))
    return torch.where(b == 127, torch.full_like(v, float("nan")), v)


def values(q, scales):
    """What packed values and their scales stand for, in float64."""
    codes = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).long()
    a = MAGNITUDES.to(q.device)[codes & 7]
    a = torch.where(codes >= 8, -a, a)
    return a * scale_values(scales).repeat_interleave(BLOCK[scales.dtype], dim=-1)


def quantize(x, fmt, factor=None):
    """(codes [rows, k], scale bytes [rows, k / block]) of x, by the definition."""
    v = x.double()
    if factor is not None:
        v = (v * factor.double()).float().double()
    v = v.view(v.shape[0], -1, BLOCK[fmt])
    bad = ~v.isfinite().all(-1)
    v = torch.where(bad.unsqueeze(-1), torch.zeros_like(v), v)
    top = v.abs().amax(-1)
    if fmt == MX:
        e = torch.where(top > 0, binade(top.clamp(min=2.0 ** -1000)) - 2, torch.full_like(top, -127))
        byte = (e.clamp(-127, 127) + 127).long()
    else:
        want = top / 6
        e = binade(want.clamp(min=2.0 ** -1000)).clamp(min=-6)
        steps = (want / power_of_two(e - 3)).round()       # of the binade, 8 .. 16 (0 .. 8 below)
        byte = torch.where(e == -6, steps, steps + 8 * (e + 6)).clamp(max=126).long()
    scale = scale_values(byte.to(torch.uint8).view(fmt))
    a = torch.where(scale.unsqueeze(-1) > 0, v.abs() / scale.unsqueeze(-1), torch.zeros_like(v))
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = ((a / step).round() * step).clamp(max=6)
    codes = torch.searchsorted(MAGNITUDES.to(a.device), a.contiguous())
    codes = codes + 8 * torch.signbit(v)
    byte = torch.where(bad, torch.full_like(byte, 255 if fmt == MX else 127), byte)
    return codes.flatten(1).to(torch.uint8), byte.to(torch.uint8)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)
