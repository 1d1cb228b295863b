"""Plain 64-bit definitions of the 4-bit rows and their products (the oracle of
their GPU tests), and how far fp32 sums may be off."""
from __future__ import annotations

import torch

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # of codes 0 .. 7; bit 3 is the sign
STEP32 = 2.0 ** -23  # a step of fp32, relative


def e2m1_codes(q: torch.Tensor) -> torch.Tensor:
    """fp64 to the nearest E2M1 code, of two as near the even one (|q| < 7). Borders between neighbours are exact."""
    a = q.abs()
    code = torch.zeros(q.shape, dtype=torch.int64, device=q.device)
    for c in range(1, 8):
        border = (VALUES[c - 1] + VALUES[c]) / 2
        code = torch.where((a > border) | ((a == border) & torch.tensor(c % 2 == 0, device=q.device)),
                           torch.full_like(code, c), code)
    return code | (torch.signbit(q).long() << 3)


def quantize(v: torch.Tensor):
    """(codes [rows][cols/2] uint8, scales [rows][cols/32] uint8) of fp64 values."""
    g = v.double().view(v.shape[0], -1, 32)
    m = g.abs().amax(2)
    bad = ~torch.isfinite(m)  # (amax gives NaN where there is one)
    _, e = torch.frexp(torch.where(bad, torch.zeros_like(m), m))  # m = f * 2^e, f in [0.5, 1)
    e = e.long() - 1
    e = torch.where(m >= 1.75 * torch.exp2(e.double()), e + 1, e)  # two significant bits: 1.75 rounds to 2
    e = torch.where(m == 0, torch.full_like(e, -1000), e)
    byte = (e - 2 + 127).clamp(min=1)
    q = g * torch.exp2(127.0 - byte.double())[:, :, None]
    code = e2m1_codes(torch.where(bad[:, :, None], torch.zeros_like(q), q)).reshape(v.shape)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), byte.to(torch.uint8)


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values of packed codes [.., K/2] and scale bytes [.., K/32] (255: NaN)."""
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return v * s.repeat_interleave(32, -1)


def half_step(q: torch.Tensor) -> torch.Tensor:
    """Half the distance of E2M1's neighbours at q, in its units."""
    a = q.abs()
    return torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)).double()


def product(x, xs, w, ws):
    """(out, magnitude) fp64: the sum and the sum of its terms' sizes."""
    xd, wd = values(x, xs), values(w, ws)
    return xd @ wd.t(), xd.abs() @ wd.abs().t()


def product_bound(out, mag, k: int, dtype) -> torch.Tensor:
    """A group of 32 sums exactly: products are multiples of 1/4 of the scales'
    product up to 36, so its sum is at most 13 bits. Then one fp32 addition per
    group and at most 8 joins of partial sums, each off by at most a step (2^-23)
    of the terms' sizes; below the normal numbers a step is 2^-149. bf16: half a
    step (2^-8) of a result off by that, at least 2^-134."""
    n = (k + 31) // 32 + 8
    err = n * (mag * STEP32 + 2.0 ** -149)
    if dtype == torch.float32:
        return err
    return err * (1 + 2.0 ** -8) + out.abs() * 2.0 ** -8 + 2.0 ** -134


def random_codes(shape, g):
    return torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8)


def random_scales(shape, g, lo=117, hi=133):
    return torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int32).to(torch.uint8)
