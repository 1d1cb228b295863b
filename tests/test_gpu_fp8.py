"""The 8-bit rows and their products on the GPU against 64-bit definitions
(tests/fp8_ref.py): group edges, ragged widths, few and many rows, empty
experts, strides, gathers, NaN and infinities, streams, graphs."""
from __future__ import annotations

import pytest
import torch

from tests import fp8_ref as R

pytestmark = pytest.mark.gpu
B = pytest.importorskip("latent_mixture_experts_amd.binding")
F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activations(rows, cols, g, dtype):
    x = torch.randn((rows, cols), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))
    return x.to(dtype)


# ---- quantisation ----------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 8192), (3, 112), (5, 128), (17, 144), (64, 272), (33, 4096),
                                       (1000, 2064), (2500, 640)])
def test_quantize_is_the_stated_arithmetic(rows, cols, dtype):
    x = activations(rows, cols, gen(rows + cols), dtype)
    codes, scales = B.fp8_quantize(x.cuda())
    ref, ref_s = R.quantize_f32(x.float())
    assert torch.equal(scales.cpu(), ref_s)
    assert torch.equal(R.canonical(codes.cpu().view(torch.uint8)), ref)
    # and against 64 bits: half a step of E4M3 at the value, and the two fp32 quotients' roundings
    v, s = x.double(), R.expand(scales.cpu(), cols)
    q = (v / s).abs().clamp_min(2.0 ** -6)
    half = torch.exp2(torch.floor(torch.log2(q)) - 4)
    back = codes.cpu().double() * s
    assert bool(((back - v).abs() <= s * (half * (1 + 8 * R.U24) + q * 8 * R.U24)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_special_values(dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.zeros((9, 256))
    x[0, 3] = 1.0                       # one value, the rest zero
    x[1, :] = torch.linspace(-1, 1, 256)
    x[1, 5], x[1, 200] = inf, nan       # non-finite values among finite ones, one per group
    x[2, :] = nan
    x[3, :128], x[3, 128:] = -inf, inf
    x[4, :] = 2.0 ** -126               # below the smallest scale
    x[4, 128] = 2.0 ** -89
    x[5, :] = torch.finfo(dtype).max
    x[6, :] = torch.where(torch.arange(256) % 2 == 0, 448.0, 27.0)  # exact codes and ties
    x[7, :] = -0.0
    x[8, :] = torch.finfo(torch.bfloat16).tiny / 8                 # a denormal
    x = x.to(dtype)
    codes, scales = B.fp8_quantize(x.cuda())
    ref, ref_s = R.quantize_f32(x.float())
    assert torch.equal(scales.cpu(), ref_s)
    assert torch.isfinite(scales).all()
    assert torch.equal(R.canonical(codes.cpu().view(torch.uint8)), ref)


def test_quantize_strided_rows_and_given_outputs():
    g = gen(5)
    wide = activations(40, 1024, g, torch.bfloat16).cuda()
    x = wide[:, 256:512]
    codes = torch.empty((40, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((40, 2), device="cuda")
    B.fp8_quantize(x, codes, scales)
    ref, ref_s = R.quantize_f32(x.float().cpu())
    assert torch.equal(R.canonical(codes.cpu()), ref) and torch.equal(scales.cpu(), ref_s)
    bits = B.fp8_quantize(x.contiguous().view(torch.int16))  # bf16 as bit patterns
    assert torch.equal(bits[0].view(torch.uint8), codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,inter", [(1, 16), (7, 144), (300, 512), (1100, 4096)])
def test_swiglu(rows, inter, dtype):
    g = gen(rows)
    gu = torch.randn((rows, 2 * inter), generator=g) * 3
    gu[0, :8] = torch.tensor([-100.0, -90.0, -50.0, -20.0, 20.0, 90.0, 300.0, -300.0])
    gu = gu.to(dtype)
    codes, scales = B.fp8_swiglu(gu.cuda())
    d = gu.double()
    h = d[:, :inter] * torch.sigmoid(d[:, :inter]) * d[:, inter:]
    amax = R.groups(h).abs().amax(2).clamp_min(R.TINY)
    # exponential and reciprocal 1 ulp each, the low part's 1, five roundings: under 16 half steps
    rel = 16 * R.U24
    assert bool(((scales.cpu().double() - amax / 448).abs() <= (rel + 2 * R.U24) * amax / 448).all())
    s = R.expand(scales.cpu(), inter)
    q = (h / s).abs().clamp_min(2.0 ** -6)
    half = torch.exp2(torch.floor(torch.log2(q * (1 + 2 * rel))) - 4)
    back = codes.cpu().double() * s
    # (2^-126 / 448: what a flushed denormal product may lose)
    assert bool(((back - h).abs() <= s * (half + q * (2 * rel)) + 2.0 ** -126).all())


@pytest.mark.parametrize("dtype,than", [(torch.float32, 1.0), (torch.bfloat16, 1.1)])
def test_swiglu_is_as_near_as_elementary_operations(dtype, than):
    """The scales' error against 64 bits, root mean square over 65536 groups:
    no larger than that of the same formula in elementary fp32 operations (bf16
    rows, whose instructions are fewer: a tenth at most)."""
    g = torch.Generator("cuda").manual_seed(21)
    gu = (torch.randn((2048, 8192), generator=g, device="cuda") * 2).to(dtype)
    scales = B.fp8_swiglu(gu)[1]
    gate, up = gu.float().chunk(2, 1)
    plain = (gate / (1 + torch.exp(-gate)) * up).view(2048, 32, 128).abs().amax(2) / torch.full((), 448.0, device="cuda")
    d, u = gu.double().chunk(2, 1)
    ref = (d * torch.sigmoid(d) * u).view(2048, 32, 128).abs().amax(2) / 448
    off = lambda s: float(((s.double() - ref) / ref).square().mean().sqrt() / R.U24)
    assert off(scales) <= than * off(plain), (off(scales), off(plain))


def test_swiglu_of_far_gates():
    """Every gate down to the exponential's overflow and far beyond it is finite, and zero there."""
    gate = torch.cat([torch.linspace(-210, -80, 4000), torch.tensor([-1e4, -1e30, -3e38]), torch.zeros(93)])
    up = torch.full_like(gate, -2.0)
    codes, scales = B.fp8_swiglu(torch.cat([gate, up])[None].cuda())
    back = codes.cpu().float() * R.expand(scales.cpu(), gate.numel()).float()
    assert torch.isfinite(back).all() and torch.isfinite(scales).all()
    assert float(back.abs().max()) < 2.0 ** -90


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_of_gates_up_to_the_exponentials_overflow(dtype):
    """exp(-gate) between 2^126 and fp32's largest value: silu is a normal
    number there, and a large up value makes it count."""
    gate = torch.cat([torch.linspace(-88.7228, -86.0, 500), torch.linspace(-88.5, -40.0, 98),
                      torch.tensor([-88.5, -88.0])]).to(dtype)
    gate = gate[gate > -88.7229]  # (as the type rounds it)
    gu = torch.cat([gate[:, None].expand(-1, 128), torch.full((gate.numel(), 128), 2.0 ** 100)], 1).to(dtype)
    codes, scales = B.fp8_swiglu(gu.cuda())
    d = gu[:, 0].double()
    h = d * torch.sigmoid(d) * 2.0 ** 100
    # exponential and reciprocal two half steps each, five roundings, one of a denormal above 2^-128: 4; under
    # 16 half steps; the scale's quotient one more. Every value of a group is its largest: code -448.
    assert bool(((scales[:, 0].cpu().double() * 448 / -h - 1).abs() <= 18 * R.U24).all())
    assert bool((codes.float() == -448).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_of_large_and_tiny_gates(dtype):
    """silu from 2^-80 to the type's largest value, and zeros of both signs."""
    gate = torch.tensor([2.0 ** -80, -2.0 ** -80, 1e-20, -1e-7, 0.5, -1.25, 15.0, 20.0, 90.0, 199.0, 201.0, 1e10, 2e30, 3e38,
                         0.0, -0.0], dtype=dtype)
    gu = torch.cat([gate[:, None].expand(-1, 128), torch.full((gate.numel(), 128), -1.0, dtype=dtype)], 1)
    codes, scales = B.fp8_swiglu(gu.cuda())
    d = gate.double()
    h = d * torch.sigmoid(d)
    amax = h.abs().clamp_min(R.TINY)
    # (h: under 16 half steps, the scale's quotient one more)
    assert bool(((scales[:, 0].cpu().double() * 448 / amax - 1).abs() <= 18 * R.U24).all())
    want = torch.where(h == 0, 0.0, torch.where(h > 0, -448.0, 448.0))
    assert bool((codes.cpu().double() == want[:, None]).all())


def test_swiglu_non_finite():
    gu = torch.ones((4, 256))
    gu[0, 3] = float("nan")
    gu[1, 4] = float("inf")
    gu[2, 5] = -float("inf")
    gu[3, 128 + 6] = float("nan")
    codes, scales = B.fp8_swiglu(gu.cuda())
    c = codes.cpu().float()
    for r, j in ((0, 3), (1, 4), (2, 5), (3, 6)):
        assert torch.isnan(c[r, j]) and int(torch.isnan(c[r]).sum()) == 1
    assert torch.isfinite(scales).all()


def test_zero_rows():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    codes, scales = B.fp8_quantize(x)
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    w, ws = torch.zeros((64, 256), dtype=F8, device="cuda"), torch.ones((1, 2), device="cuda")
    assert B.fp8_linear(codes, scales, w, ws).shape == (0, 64)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = B.fp8_grouped(codes, scales, off, w.repeat(2, 1).view(2, 64, 256), ws.repeat(2, 1).view(2, 1, 2))
    assert out.shape == (0, 64)


# ---- products --------------------------------------------------------------

def operands(rows, n, k, g, experts=None):
    x, xs = R.random_codes((rows, k), g), R.random_scales((rows, R.blocks(k)), g)
    lead = () if experts is None else (experts,)
    w, ws = R.random_codes((*lead, n, k), g), R.random_scales((*lead, R.blocks(n), R.blocks(k)), g)
    return x, xs, w, ws


def dev(*ts):
    return [t.cuda() for t in ts]


SHAPES = [(1, 1, 16), (1, 256, 128), (1, 4096, 1024), (2, 130, 144), (15, 16, 8192), (16, 127, 112), (17, 129, 256),
          (31, 64, 4112), (33, 272, 640), (64, 128, 128), (65, 128, 1024), (100, 1, 32), (127, 7, 528),
          (128, 256, 512), (129, 257, 640), (257, 384, 1040), (500, 1000, 272), (700, 255, 2048)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_linear(rows, n, k, dtype):
    x, xs, w, ws = operands(rows, n, k, gen(rows * 7 + n + k))
    got = B.fp8_linear(*dev(x, xs, w, ws), dtype)
    assert got.dtype == dtype and got.shape == (rows, n)
    R.assert_product(got.cpu(), x, xs, w, ws)


# (rows, n, k) that fill the chip with each tile size, with ragged rows, weight rows and blocks of K
WIDE = [(30, 9000, 400), (33, 8000, 528), (48, 6001, 1040), (60, 8000, 400), (70, 8200, 1040), (200, 4000, 1040), (200, 4100, 400), (5, 20000, 528), (9, 65536, 144), (300, 5000, 272), (500, 4200, 1168), (520, 8200, 144),
        (1030, 8200, 144), (2100, 4200, 528), (2300, 8200, 256), (511, 20001, 144)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,k", WIDE)
def test_linear_wide(rows, n, k, dtype):
    ops = dev(*operands(rows, n, k, gen(rows * 3 + n + k)))
    R.assert_product(B.fp8_linear(*ops, dtype), *ops)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("experts,mean,n,k", [(90, 1, 2100, 272), (256, 20, 300, 144), (30, 40, 2100, 400),
                                              (60, 40, 3000, 144), (30, 60, 4200, 144), (30, 130, 2100, 272),
                                              (4, 600, 4200, 144), (3, 1700, 2100, 528), (8, 375, 700, 1040)])
def test_grouped_wide(experts, mean, n, k, dtype):
    """Uneven groups, some empty, for each tile size."""
    g = gen(experts + mean + n)
    part = torch.rand(experts, generator=g)
    part[part < 0.15] = 0.0
    part[0] += 1.0
    sizes = (part / part.sum() * mean * experts).round().int().tolist()
    bounds = [0] + torch.tensor(sizes).cumsum(0).tolist()
    x, xs, w, ws = dev(*operands(bounds[-1], n, k, g, experts))
    got = B.fp8_grouped(x, xs, torch.tensor(bounds, dtype=torch.int32).cuda(), w, ws, dtype)
    check_grouped(got, x, xs, w, ws, bounds)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(9000, 400), (4100, 1040), (2080, 272), (300, 2064)])
def test_grouped_few_rows_wide(n, k, dtype):
    """A token's routes: one or two rows on a few of the experts, K split between fewer and more wavefronts."""
    g = gen(n)
    sizes = [0] * 40
    for e in (0, 3, 4, 9, 20, 31, 38, 39):
        sizes[e] = 1 + (e == 9)
    bounds = [0] + torch.tensor(sizes).cumsum(0).tolist()
    x, xs, w, ws = dev(*operands(bounds[-1], n, k, g, 40))
    got = B.fp8_grouped(x, xs, torch.tensor(bounds, dtype=torch.int32).cuda(), w, ws, dtype)
    check_grouped(got, x, xs, w, ws, bounds)


@pytest.mark.parametrize("rows,n,k", SHAPES + WIDE)
def test_sums_in_fp32_lose_nothing(rows, n, k):
    """Sums that cancel to less than 2^-14 of their terms: exact with an fp32
    out, and rounded once from the exact one in bf16 with f32_sums; the bf16
    default within what it may drop."""
    x, xs, w, ws = ops = dev(*R.cancelling(rows, n, k, gen(rows + n + k)))
    want = R.product(*ops)[0]
    assert torch.equal(B.fp8_linear(*ops, torch.float32).double(), want)
    assert torch.equal(B.fp8_linear(*ops, f32_sums=True), want.float().bfloat16())
    out = torch.empty((rows, n + 3), device="cuda")[:, 3:]
    B.fp8_linear(*ops, out=out, f32_sums=True)
    assert torch.equal(out.double(), want)
    R.assert_product(B.fp8_linear(*ops), *ops)


# (rows, n, k) on both sides of where few rows go from the streaming kernel to the tiles
FEW = [(1, 4112, 4096), (1, 4112, 4112), (1, 4097, 8208), (3, 5000, 1360), (3, 5000, 1376), (5, 8200, 1040), (16, 4200, 256),
       (16, 4200, 272), (11, 4090, 8192), (13, 4090, 8192), (16, 500, 6144), (16, 500, 6160), (2, 20000, 2064), (16, 20000, 272),
       (4, 8190, 4096), (5, 8190, 4096), (2, 7168, 8192), (3, 7168, 8192), (2, 7000, 8192)]


@pytest.mark.parametrize("dtype,f32_sums", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
@pytest.mark.parametrize("rows,n,k", FEW)
def test_linear_few_rows(rows, n, k, dtype, f32_sums):
    ops = dev(*operands(rows, n, k, gen(rows * 5 + n + k)))
    R.assert_product(B.fp8_linear(*ops, dtype, f32_sums=f32_sums), *ops)
    ops = dev(*R.cancelling(rows, n, k, gen(rows + n + k)))
    got, want = B.fp8_linear(*ops, dtype, f32_sums=f32_sums), R.product(*ops)[0]
    assert torch.equal(got, want.float().to(dtype))  # (a bf16 out of so few rows sums in fp32 anyway)


GROUPS = [(90, 1, 2100, 272), (256, 20, 300, 144), (30, 40, 2100, 400), (60, 40, 3000, 144), (30, 60, 4200, 144),
          (30, 130, 2100, 272), (4, 600, 4200, 144), (8, 375, 700, 1040), (5, 2, 272, 640)]


@pytest.mark.parametrize("experts,mean,n,k", GROUPS)
def test_grouped_sums_in_fp32_lose_nothing(experts, mean, n, k):
    g = gen(experts + mean + n)
    sizes = torch.randint(0, 2 * mean + 1, (experts,), generator=g).tolist()
    bounds = [0] + torch.tensor(sizes).cumsum(0).tolist()
    x, xs, w, ws = dev(*R.cancelling(bounds[-1], n, k, g, experts))
    off = torch.tensor(bounds, dtype=torch.int32).cuda()
    wide = B.fp8_grouped(x, xs, off, w, ws, torch.float32)
    half = B.fp8_grouped(x, xs, off, w, ws, f32_sums=True)
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            want = R.product(x[a:b], xs[a:b], w[e], ws[e])[0]
            assert torch.equal(wide[a:b].double(), want) and torch.equal(half[a:b], want.float().bfloat16()), e
    check_grouped(B.fp8_grouped(x, xs, off, w, ws), x, xs, w, ws, bounds)


@pytest.mark.parametrize("rows", [1, 20, 40, 150])
def test_every_position_counts_once(rows):
    """One nonzero code per row of x and every code value in w: out is that code times the scales."""
    k, n = 512, 300
    g = gen(rows)
    at = torch.randint(0, k, (rows,), generator=g)
    x = torch.zeros((rows, k), dtype=torch.uint8)
    x[torch.arange(rows), at] = 0x38  # 1.0
    w = torch.randint(0, 256, (n, k), generator=g, dtype=torch.uint8)
    w[w & 0x7F == 0x7F] = 0
    xs = torch.exp2(torch.randint(-3, 4, (rows, 4), generator=g).float())
    ws = torch.exp2(torch.randint(-3, 4, (3, 4), generator=g).float())
    got = B.fp8_linear(*dev(x, xs, w, ws), torch.float32).cpu()
    wd = w.view(F8).float() * R.expand(ws, k).float().repeat_interleave(128, 0)[:n]
    assert torch.equal(got, (wd[:, at] * xs[torch.arange(rows), at // 128]).t())


@pytest.mark.parametrize("rows", [3, 24, 50, 200])
def test_nan_codes_stay_in_their_row_and_column(rows):
    x, xs, w, ws = operands(rows, 200, 384, gen(rows))
    xb, wb = x.view(torch.uint8), w.view(torch.uint8)
    xb[1, 380] = 0x7F
    wb[150, 3] = 0xFF
    got = B.fp8_linear(*dev(x, xs, w, ws), torch.float32).cpu()
    want = torch.zeros((rows, 200), dtype=torch.bool)
    want[1, :], want[:, 150] = True, True
    assert torch.equal(torch.isnan(got), want)


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_linear_strides(rows):
    """Rows of x in a wider buffer, out a slice of a wider one whose other columns stay."""
    g = gen(rows)
    n, k = 200, 400
    wide = R.random_codes((rows, 1024), g)
    _, xs, w, ws = operands(rows, n, k, g)
    x = wide.cuda()[:, 512:512 + k]
    for dtype in (torch.bfloat16, torch.float32):
        for lo, total in ((0, 200), (3, 331), (8, 256)):
            buf = torch.full((rows, total), 7.0, dtype=dtype, device="cuda")
            B.fp8_linear(x, *dev(xs, w, ws), out=buf[:, lo:lo + n])
            R.assert_product(buf[:, lo:lo + n].cpu(), wide[:, 512:512 + k], xs, w, ws, (dtype, lo))
            rest = torch.cat([buf[:, :lo], buf[:, lo + n:]], 1)
            assert bool((rest == 7.0).all())


def sizes_case(name, experts, g):
    if name == "uniform":
        return [5] * experts
    if name == "one expert":
        return [0] * (experts - 1) + [90]
    if name == "edges":
        return ([0, 1, 15, 16, 17, 0, 63, 64, 65, 127, 128, 129, 0, 250] * experts)[:experts]
    if name == "many":
        return torch.randint(90, 180, (experts,), generator=g).tolist()
    if name == "first only":
        return [3] + [0] * (experts - 1)
    return torch.randint(0, 4, (experts,), generator=g).tolist()


def check_grouped(got, x, xs, w, ws, bounds, rows_of=None):
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            at = torch.arange(a, b, device=x.device) if rows_of is None else rows_of[a:b]
            R.assert_product(got[a:b], x[at], xs[at], w[e], ws[e], e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name,experts,n,k", [
    ("uniform", 6, 128, 256), ("one expert", 9, 144, 400), ("edges", 14, 272, 384), ("edges", 28, 33, 144),
    ("many", 5, 300, 640), ("first only", 256, 64, 128), ("few", 256, 48, 272), ("few", 255, 130, 128),
    ("edges", 3, 512, 2048), ("many", 1, 257, 1040)])
def test_grouped(name, experts, n, k, dtype):
    g = gen(experts + n)
    sizes = sizes_case(name, experts, g)
    bounds = [0] + torch.tensor(sizes).cumsum(0).tolist()
    rows = bounds[-1]
    x, xs, w, ws = operands(rows, n, k, g, experts)
    off = torch.tensor(bounds, dtype=torch.int32)
    got = B.fp8_grouped(*dev(x, xs, off, w, ws), dtype)
    check_grouped(got.cpu(), x, xs, w, ws, bounds)


@pytest.mark.parametrize("rows_per", [2, 30, 60, 200])
def test_grouped_gather_and_rows_outside(rows_per):
    """Rows read through an index with a divisor, out of range ones clamped;
    output rows before the first and behind the last expert's stay as they were."""
    g = gen(rows_per)
    experts, n, k, top = 4, 272, 400, 3
    sizes = [rows_per, 0, rows_per + 5, 1]
    bounds = [4] + (4 + torch.tensor(sizes).cumsum(0)).tolist()
    rows, x_rows = bounds[-1] + 9, 37
    x, xs, w, ws = operands(x_rows, n, k, g, experts)
    index = torch.randint(0, x_rows * top, (rows,), generator=g, dtype=torch.int32)
    index[5], index[6] = x_rows * top + 100, -50
    out = torch.full((rows, n), 3.0, device="cuda")
    B.fp8_grouped(*dev(x, xs, torch.tensor(bounds, dtype=torch.int32), w, ws), row_index=index.cuda(), index_div=top,
                  out=out)
    got = out.cpu()
    assert bool((got[:4] == 3.0).all()) and bool((got[bounds[-1]:] == 3.0).all())
    src = torch.div(index, top, rounding_mode="trunc").clamp(0, x_rows - 1).long()
    check_grouped(got, x, xs, w, ws, bounds, src)


def test_grouped_repeated_index_and_strides():
    g = gen(11)
    x, xs, w, ws = operands(6, 96, 128, g, 2)
    wide = torch.zeros((6, 256), dtype=torch.uint8)
    wide[:, 64:192] = x.view(torch.uint8)
    index = torch.tensor([2, 2, 2, 5, 0, 2], dtype=torch.int32)
    bounds = [0, 4, 6]
    buf = torch.zeros((6, 131), device="cuda")
    B.fp8_grouped(wide.cuda()[:, 64:192], xs.cuda(), torch.tensor(bounds, dtype=torch.int32).cuda(), *dev(w, ws),
                  row_index=index.cuda(), out=buf[:, 5:101])
    check_grouped(buf[:, 5:101].cpu(), x, xs, w, ws, bounds, index.long())
    assert float(buf[:, :5].abs().sum() + buf[:, 101:].abs().sum()) == 0.0


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_bad_offsets_stay_inside(rows):
    """Offsets that decrease or leave the rows: nothing outside out is written, no error."""
    x, xs, w, ws = operands(rows, 144, 128, gen(rows), 3)
    guard = torch.full((rows + 64, 144), 5.0, device="cuda")
    for off in ([0, rows + 40, 2 * rows, 3 * rows], [rows, 0, rows, 0], [-7, rows, -100, rows],
                [2 ** 31 - 1, -2 ** 31, 0, 2 ** 31 - 1]):
        B.fp8_grouped(*dev(x, xs, torch.tensor(off, dtype=torch.int32), w, ws), out=guard[32:32 + rows])
        assert bool((guard[:32] == 5.0).all()) and bool((guard[32 + rows:] == 5.0).all())


@pytest.mark.parametrize("rows", [1, 30, 60, 400])
def test_same_bits_every_time(rows):
    x, xs, w, ws = dev(*operands(rows, 500, 1040, gen(rows)))
    a = B.fp8_linear(x, xs, w, ws, torch.float32)
    for _ in range(3):
        assert torch.equal(B.fp8_linear(x, xs, w, ws, torch.float32), a)
    # a row does not depend on the rows beside it within the same kernel form
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    b = B.fp8_grouped(x, xs, off, w[None].contiguous(), ws[None].contiguous(), torch.float32)
    assert torch.equal(a, b)


def test_a_side_stream():
    x, xs, w, ws = dev(*operands(200, 256, 512, gen(1)))
    want = B.fp8_linear(x, xs, w, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.fp8_linear(x, xs, w, ws)
    out = torch.zeros_like(want)
    B.fp8_linear(x, xs, w, ws, out=out, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want)


def test_inputs_dropped_after_a_call_on_a_given_stream():
    """The call still waits on its stream when the caller drops its inputs: the
    current stream does not get their memory."""
    g = gen(4)
    x, xs, w, ws = dev(*operands(512, 256, 4096, g))
    want = B.fp8_linear(x, xs, w, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dropped = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = B.fp8_linear(dropped, xs, w, ws, stream=s)
    at = dropped.data_ptr()
    del dropped
    fresh = [torch.zeros_like(x) for _ in range(4)]
    if not s.query():  # (the call has not run yet)
        assert all(t.data_ptr() != at for t in fresh)
    s.synchronize()
    assert torch.equal(got, want)


def test_captured_on_a_given_stream():
    """A call on a stream forked from the captured one and joined again, its
    input made and dropped inside the capture."""
    g = gen(6)
    _, _, w, ws = dev(*operands(1, 256, 512, g))
    x = torch.empty((70, 512), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()

    def run():
        c, cs = B.fp8_quantize(x * 2)
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        out = B.fp8_linear(c, cs, w, ws, stream=s)
        del c, cs
        other = x * 3
        here.wait_stream(s)
        return out, other

    x.copy_(activations(70, 512, g, torch.bfloat16))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(4):
        x.copy_(activations(70, 512, gen(seed), torch.bfloat16))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run())), seed


@pytest.mark.parametrize("tokens", [2, 40, 500])
def test_captured_run_replays_as_eager(tokens):
    """quantize -> grouped -> swiglu -> grouped in one graph, replayed with new
    inputs and new groups, eager work between."""
    g = gen(tokens)
    experts, k, inter = 8, 256, 128
    x = torch.empty((tokens, k), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    w13, s13 = dev(R.random_codes((experts, 2 * inter, k), g), R.random_scales((experts, 2, 2), g))
    w2, s2 = dev(R.random_codes((experts, k, inter), g), R.random_scales((experts, 2, 1), g))

    def run():
        c, s = B.fp8_quantize(x)
        gu = B.fp8_grouped(c, s, off, w13, s13)
        h, hs = B.fp8_swiglu(gu)
        return B.fp8_grouped(h, hs, off, w2, s2, torch.float32)

    def fill(seed):
        q = gen(seed)
        x.copy_(activations(tokens, k, q, torch.bfloat16))
        cut = torch.randint(0, tokens + 1, (experts - 1,), generator=q).sort().values.tolist()
        off.copy_(torch.tensor([0] + cut + [tokens], dtype=torch.int32))

    fill(0)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(1, 6):
        fill(seed)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, run()), seed


def test_refusals():
    x, xs, w, ws = dev(*operands(4, 128, 256, gen(2)))
    for bad in (lambda: B.fp8_linear(x, xs[:, :1].contiguous(), w, ws), lambda: B.fp8_linear(x, xs, w[:, :128], ws),
                lambda: B.fp8_linear(x, xs.cpu(), w, ws), lambda: B.fp8_linear(x.float(), xs, w, ws),
                lambda: B.fp8_linear(x.t(), xs, w, ws), lambda: B.fp8_linear(x, xs, w, ws, torch.float16),
                lambda: B.fp8_linear(x, xs, w, ws, out=torch.empty((4, 127), device="cuda")),
                lambda: B.fp8_quantize(x), lambda: B.fp8_quantize(xs[0]),
                lambda: B.fp8_swiglu(torch.zeros((2, 33), device="cuda")),
                lambda: B.fp8_grouped(x, xs, torch.zeros(2, device="cuda"), w[None], ws[None]),
                lambda: B.fp8_grouped(x, xs, torch.zeros(3, dtype=torch.int32, device="cuda"), w[None], ws[None])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.MoeError) as e:
        B.fp8_quantize(torch.zeros((2, 24), device="cuda"))
    assert e.value.status == B.MOE_EUNSUPPORTED
    with pytest.raises(B.MoeError) as e:
        B.fp8_quantize(torch.zeros((2, 40), device="cuda")[:, 1:17])
    assert e.value.status == B.MOE_EALIGN


# ---- a run of them together --------------------------------------------------

@pytest.mark.parametrize("tokens", [1, 6, 70, 600])
def test_layer_in_eight_bits(tokens):
    """moe_route's routing, then the pooler, the experts and the unpooler in
    8 bits as a user chains them; each product against 64 bits on the GPU's
    own inputs, the whole against the layer in 64 bits."""
    dims = dict(hidden=512, latent=256, inter=128, n_experts=16, top_k=4)
    H, L, I, E, K = (dims[k] for k in ("hidden", "latent", "inter", "n_experts", "top_k"))
    g = gen(tokens)
    x = torch.randn((tokens, H), generator=g).bfloat16().cuda()
    router = (torch.randn((E, H), generator=g) * 0.05).cuda()

    def weight(*shape):
        w = torch.randn(shape, generator=g) / shape[-1] ** 0.5
        b = torch.nn.functional.pad(w, (0, 0, 0, 0)).view(*shape[:-2], shape[-2] // 128, 128, shape[-1] // 128, 128)
        s = b.abs().amax(dim=(-3, -1)) / 448
        c = (b / s[..., :, None, :, None]).view(shape).to(F8)
        return c.cuda(), s.contiguous().cuda()

    pool, w13, w2, unpool = weight(L, H), weight(E, 2 * I, L), weight(E, L, I), weight(H, L)
    d = B.make_dims(dims)
    r = B.route(d, x.view(torch.int16), router, B.alloc_workspace(d, tokens))
    xq = B.fp8_quantize(x)
    lat = B.fp8_linear(*xq, *pool)
    lq = B.fp8_quantize(lat)
    gu = B.fp8_grouped(*lq, r["offsets"], *w13, row_index=r["sorted"], index_div=K)
    hq = B.fp8_swiglu(gu)
    rows = B.fp8_grouped(*hq, r["offsets"], *w2, out_dtype=torch.float32)
    order = r["sorted"].long()
    normed = rows / (rows.square().mean(1, keepdim=True) + 1e-6).sqrt() * r["w"].reshape(-1)[order][:, None]
    y = torch.zeros((tokens, L), device="cuda").index_add_(0, order // K, normed).bfloat16()
    yq = B.fp8_quantize(y)
    out = B.fp8_linear(*yq, *unpool)

    cpu = lambda ts: [t.cpu() for t in ts]
    bounds = r["offsets"].tolist()
    assert bounds[-1] == tokens * K
    R.assert_product(lat.cpu(), *cpu(xq), *cpu(pool), "pooler")
    check_grouped(gu.cpu(), *cpu(lq), *cpu(w13), bounds, order.cpu() // K)
    check_grouped(rows.cpu(), *cpu(hq), *cpu(w2), bounds)
    R.assert_product(out.cpu(), *cpu(yq), *cpu(unpool), "unpooler")
    # the layer in 64 bits without any 8-bit activation: four quantisations of
    # at most 2^-4 per value, their errors independent (rms 2^-4 / sqrt(3) at
    # the most), through unit-gain random projections; swiglu and the norm at most double it
    wd = lambda c, s: c.double() * s.double().repeat_interleave(128, -1).repeat_interleave(128, -2)
    ld = x.double() @ wd(*pool).t()
    ref = torch.zeros((tokens, L), dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if a < b:
            t = order[a:b] // K
            z = ld[t] @ wd(w13[0][e], w13[1][e]).t()
            h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
            o = h @ wd(w2[0][e], w2[1][e]).t()
            o = o / (o.square().mean(1, keepdim=True) + 1e-6).sqrt() * r["w"].reshape(-1)[order[a:b]].double()[:, None]
            ref.index_add_(0, t, o)
    ref = ref @ wd(*unpool).t()
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel < 4 * 2 * 2.0 ** -4 / 3 ** 0.5, rel


# ---- offsets past 32 bits --------------------------------------------------

MANY = (1 << 24) + 37  # rows: more than one launch of the quantisation takes


def far_rows():
    """Where offsets and launches turn over, and the ends."""
    at = [0, MANY - 64, (1 << 24) - 32, (1 << 31) // 144 - 32, (1 << 32) // 288 - 32, (1 << 31) // 272 - 32]
    return torch.cat([torch.arange(a, a + 64) for a in at])


def test_quantize_of_many_rows():
    x = torch.empty((MANY, 144), dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(MANY, device="cuda")[:, None] % 1009 - 504)
    x[:, 5:20] += torch.arange(15, device="cuda", dtype=torch.bfloat16)
    codes, scales = B.fp8_quantize(x)
    at = far_rows()
    ref, ref_s = R.quantize_f32(x[at.cuda()].float().cpu())
    assert torch.equal(scales[at.cuda()].cpu(), ref_s)
    assert torch.equal(R.canonical(codes.view(torch.uint8)[at.cuda()].cpu()), ref)
    # every row against the first of the same values
    codes = codes.view(torch.uint8)
    for r in range(0, MANY, 1009 << 10):
        n = min(1009 << 10, MANY - r)
        assert torch.equal(codes[r:r + n], codes[:n]) and torch.equal(scales[r:r + n], scales[:n]), r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_of_many_rows(dtype):
    g = gen(3)
    few, few_s, w, ws = operands(1009, 144, 144, g)
    times = MANY // 1009 + 1
    x = few.view(torch.uint8).cuda().repeat(times, 1)[:MANY].view(F8)
    xs = few_s.cuda().repeat(times, 1)[:MANY].contiguous()
    got = B.fp8_linear(x, xs, *dev(w, ws), dtype)
    at = far_rows()
    R.assert_product(got[at.cuda()].cpu(), x.view(torch.uint8)[at.cuda()].cpu().view(F8), xs[at.cuda()].cpu(), w, ws)
    for r in range(0, MANY, 1009 << 10):  # (a row's sum does not depend on its place)
        n = min(1009 << 10, MANY - r)
        assert torch.equal(got[r:r + n], got[:n]), r


def test_sizes_past_32_bits_are_refused():
    x = torch.empty((1 << 31, 16), dtype=torch.uint8, device="cuda")
    xs = torch.empty((1 << 31, 1), device="cuda")
    w, ws = torch.zeros((16, 16), dtype=torch.uint8, device="cuda"), torch.ones((1, 1), device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        B.fp8_linear(x, xs, w, ws)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    index = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        B.fp8_grouped(x[:4], xs[:4], off, w[None], ws[None], row_index=index, index_div=(1 << 32) + 1)
