"""Plain 64-bit definitions of the 8-bit rows, their products and the balance
loss, on the host (the oracle of their GPU tests), and how far fp32 may be off."""
from __future__ import annotations

import math

import torch

U24 = 2.0 ** -24  # half a step of fp32, relative
TINY = 2.0 ** -90


def blocks(n: int) -> int:
    return (n + 127) // 128


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """fp64 to the nearest E4M3 value, ties to even (|v| <= 464)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def groups(v: torch.Tensor) -> torch.Tensor:
    rows, cols = v.shape
    return torch.nn.functional.pad(v, (0, blocks(cols) * 128 - cols)).view(rows, -1, 128)


def quantize_f32(v: torch.Tensor):
    """The stated fp32 arithmetic, operation by operation: (codes uint8 with
    every NaN as 0x7F, scales). v fp32 on the host."""
    g = groups(v)
    fine = torch.isfinite(g)
    amax = torch.where(fine, g.abs(), torch.zeros(())).amax(2).clamp_min(TINY)
    top = torch.full_like(amax, 448.0)
    q = torch.where(fine, g * (top / amax)[:, :, None], torch.full((), float("nan")))
    codes = q.reshape(v.shape[0], -1)[:, :v.shape[1]].contiguous().to(torch.float8_e4m3fn).view(torch.uint8)
    return canonical(codes), amax / top


def canonical(codes: torch.Tensor) -> torch.Tensor:
    codes = codes.view(torch.uint8)
    return torch.where(codes & 0x7F == 0x7F, torch.full_like(codes, 0x7F), codes)


def expand(xs: torch.Tensor, k: int) -> torch.Tensor:
    return xs.double().repeat_interleave(128, -1)[..., :k]


def eights(v: torch.Tensor) -> torch.Tensor:
    """The largest size of each eight neighbouring values (the last eight filled with zeros)."""
    k = v.shape[1]
    return torch.nn.functional.pad(v, (0, -k % 8)).view(v.shape[0], -1, 8).abs().amax(2)


def product(x, xs, w, ws):
    """(out, magnitude, largest) fp64: the sum, the sum of its terms' sizes, the
    sum over each eight neighbouring terms of a bound on their largest."""
    k, n = x.shape[1], w.shape[0]
    xd = x.float().double() * expand(xs, k)
    wd = w.float().double() * expand(ws, k).repeat_interleave(128, 0)[:n]
    top = eights(xd) @ eights(wd).t()
    return xd @ wd.t(), xd.abs() @ wd.abs().t(), top


def product_bound(out, mag, top, k: int, dtype) -> torch.Tensor:
    """A block: 128 exact products added in fp32, each addition off by at
    most one step (2^-23) of the terms' sizes so far; then per block one
    rounding of the scales' product, one of the multiply-add, and at most 8
    joins of partial sums and one more addition each: (nkb + 12) half steps.
    bf16: half a step of the result on top, of a value off by the former;
    and the E4M3 matrix instruction, which bf16 outputs of many rows take,
    drops from each of eight neighbouring products what lies below 2^-14 of
    the largest of them (its leading bit; read off the instruction with one
    large product and one power of two): 7 * 2^-14 of it per eight."""
    err = mag * (128 * 2 * U24 + (blocks(k) + 12) * U24)
    if dtype == torch.float32:
        return err + 1e-37
    return (err + top * 7 * 2.0 ** -14) * (1 + 2.0 ** -8) + out.abs() * 2.0 ** -8 + 1e-37


def assert_product(got, x, xs, w, ws, what=""):
    ref, mag, top = product(x, xs, w, ws)
    err = (got.double() - ref).abs()
    bad = ~(err <= product_bound(ref, mag, top, x.shape[1], got.dtype))
    assert not bad.any(), (what, int(bad.sum()), float(err.max()), bad.nonzero()[:4].tolist())


def random_codes(shape, gen, spread=140.0):
    return (torch.randn(shape, generator=gen) * spread).clamp(-448, 448).to(torch.float8_e4m3fn)


def random_scales(shape, gen):
    return torch.exp(torch.randn(shape, generator=gen)) * 0.01


def cancelling(rows, n, k, gen, experts=None):
    """Operands (codes, power-of-two scales) of whole numbers whose sums fp32
    holds in any order, and sums of fewer bits do not: every block has one
    product of 2^16 and one of -2^16, in different eights, beside products of
    at most 4. A block's partial sums stay below 2^18, its sum below 2^9, all of
    them quarters at least after the scales."""
    lead = () if experts is None else (experts,)
    x = torch.randint(-2, 3, (rows, k), generator=gen).float()
    w = torch.randint(-2, 3, (*lead, n, k), generator=gen).float()
    for b in range(0, k, 128):
        two = torch.randperm(min(128, k - b) // 8, generator=gen)[:2] * 8 + b
        at = two + torch.randint(0, 8, (2,), generator=gen)
        x[:, at] = 256.0
        sign = torch.randint(0, 2, (*lead, n), generator=gen) * 2 - 1
        w[..., at[0]], w[..., at[1]] = 256.0 * sign, -256.0 * sign
    scales = lambda *shape: torch.exp2(torch.randint(-1, 2, shape, generator=gen).float())
    f8 = torch.float8_e4m3fn
    return x.to(f8), scales(rows, blocks(k)), w.to(f8), scales(*lead, blocks(n), blocks(k))


def balance(logits, ids, mask=None, grad_losses=None, w=None, grad_w=None, counts=None):
    """(losses [2], counts [E+1], grad) in fp64; counts given: the gradient takes those."""
    lg = logits.double()
    t, e = lg.shape
    k = ids.shape[1]
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    live = live & (lg != float("-inf")).any(1)
    c = torch.zeros(e + 1, dtype=torch.int64)
    for i in ids[live].reshape(-1).tolist():
        if 0 <= i < e:
            c[i] += 1
    c[e] = int(live.sum())
    n = max(int(c[e]), 1)
    safe = torch.where(live[:, None], lg, torch.zeros((), dtype=torch.float64))
    lse = torch.logsumexp(safe, 1)
    # (not exp(logit - lse): beside logits of 3e38 the logarithm of the sum is lost in lse even in 64 bits)
    p = torch.softmax(safe, 1) * live[:, None]
    lse = lse * live
    f = c[:e].double() * e / (k * n)
    losses = torch.stack([(f * p.sum(0) / n).sum(), (lse * lse).sum() / n])
    if grad_losses is None:
        return losses, c, None, None
    if counts is not None:
        n = max(int(counts[e]), 1)
        f = counts[:e].double() * e / (k * n)
    gb, gz = grad_losses.double()
    grad = gb / n * p * (f - (p @ f)[:, None]) + gz / n * 2 * lse[:, None] * p
    # (lse is the largest logit plus the logarithm of a sum in [1, E]: in fp32 its
    # error goes by the sizes of the two, also where they cancel)
    parts = lse.abs() + torch.where(live, safe.amax(1).abs(), torch.zeros((), dtype=torch.float64)) + math.log(e)
    size = gb.abs() / n * p * (f + (p @ f)[:, None]) + gz.abs() / n * 2 * parts[:, None] * p
    if w is not None:
        wd, dwd = w.double(), grad_w.double()
        gate = wd * (dwd - (wd * dwd).sum(1, keepdim=True)) * live[:, None]
        gs = wd * (dwd.abs() + (wd * dwd).abs().sum(1, keepdim=True)) * live[:, None]
        for j in range(k):
            ok = (ids[:, j] >= 0) & (ids[:, j] < e)
            at = ids[:, j].long().clamp(0, e - 1)[:, None]
            grad.scatter_add_(1, at, (gate[:, j] * ok)[:, None])
            size.scatter_add_(1, at, (gs[:, j] * ok)[:, None])
    return losses, c, grad, size
