"""The 4-bit rows, their products and the way into expert order without a GPU:
the argument checks, and the oracle against definitions of its own."""
from __future__ import annotations

import types

import pytest
import torch

from latent_mixture_experts_amd import binding as B
from tests import fp4_ref as R

P = 0x10000  # a fake, 16-byte aligned "device" address: never dereferenced


def _quant(fn="moe_fp4_quantize", rows=4, cols=256, x=P, ldx=None, t=B.TYPE_BF16, codes=P, scales=P):
    wide = cols * (2 if "swiglu" in fn else 1)
    return getattr(B.lib(), fn + "_validate")(rows, cols, x, wide if ldx is None else ldx, t, codes, scales)


def _dequant(rows=4, cols=256, codes=P, scales=P, out=P, ldo=None, t=B.TYPE_BF16):
    return B.lib().moe_fp4_dequantize_validate(rows, cols, codes, scales, out, cols if ldo is None else ldo, t)


@pytest.mark.parametrize("fn", ["moe_fp4_quantize", "moe_fp4_swiglu"])
def test_quantize_arguments(fn):
    wide = 512 if "swiglu" in fn else 256
    assert _quant(fn) == B.MOE_OK
    assert _quant(fn, t=B.TYPE_F32) == B.MOE_OK
    assert _quant(fn, scales=P + 1, cols=32) == B.MOE_OK
    assert _quant(fn, ldx=wide + 8) == B.MOE_OK
    assert _quant(fn, rows=0, x=None, codes=None, scales=None) == B.MOE_OK
    for k in ("x", "codes", "scales"):
        assert _quant(fn, **{k: None}) == B.MOE_EINVAL
    assert _quant(fn, x=P + 2) == B.MOE_EALIGN
    assert _quant(fn, codes=P + 8) == B.MOE_EALIGN
    assert _quant(fn, ldx=wide + 4) == B.MOE_EALIGN
    assert _quant(fn, ldx=wide + 4, t=B.TYPE_F32) == B.MOE_OK
    assert _quant(fn, ldx=wide - 8) == B.MOE_EINVAL
    assert _quant(fn, rows=-1) == B.MOE_EINVAL
    assert _quant(fn, cols=0) == B.MOE_EINVAL
    for t in (2, -1, B.TYPE_BF16 | B.SUM_F32):
        assert _quant(fn, t=t) == B.MOE_EINVAL
    for cols in (16, 250, 65568):
        assert _quant(fn, cols=cols) == B.MOE_EUNSUPPORTED
    assert _quant(fn, cols=2 ** 31 - 32, ldx=2 ** 40) == B.MOE_EUNSUPPORTED
    assert _quant(fn, ldx=(1 << 22) + 8) == B.MOE_EUNSUPPORTED
    assert _quant(fn, rows=1 << 28) == B.MOE_EUNSUPPORTED


def test_dequantize_arguments():
    assert _dequant() == B.MOE_OK
    assert _dequant(scales=P + 3, out=P + 2, ldo=257) == B.MOE_OK
    assert _dequant(t=B.TYPE_F32, out=P + 2) == B.MOE_EALIGN
    assert _dequant(rows=0, codes=None, scales=None, out=None) == B.MOE_OK
    for k in ("codes", "scales", "out"):
        assert _dequant(**{k: None}) == B.MOE_EINVAL
    assert _dequant(codes=P + 8) == B.MOE_EALIGN
    assert _dequant(ldo=255) == B.MOE_EINVAL
    assert _dequant(rows=-1) == B.MOE_EINVAL
    assert _dequant(t=3) == B.MOE_EINVAL
    for bad in (dict(cols=48), dict(cols=65568), dict(ldo=(1 << 22) + 1), dict(rows=1 << 28)):
        assert _dequant(**bad) == B.MOE_EUNSUPPORTED, bad


def _linear(T=4, N=256, K=512, x=P, ldx=None, xs=P, w=P, ws=P, out=P, ldo=None, t=B.TYPE_BF16):
    return B.lib().moe_fp4_linear_validate(T, N, K, x, K // 2 if ldx is None else ldx, xs, w, ws, out,
                                           N if ldo is None else ldo, t)


def _grouped(rows=4, E=8, N=256, K=512, off=P, idx=None, div=1, x_rows=None, x=P, ldx=None, xs=P, w=P,
             ws=P, out=P, ldo=None, t=B.TYPE_BF16):
    return B.lib().moe_fp4_grouped_validate(rows, E, N, K, off, idx, div, rows if x_rows is None else x_rows,
                                            x, K // 2 if ldx is None else ldx, xs, w, ws, out,
                                            N if ldo is None else ldo, t)


@pytest.mark.parametrize("fn", [_linear, _grouped])
def test_product_arguments(fn):
    rows = "T" if fn is _linear else "rows"
    assert fn() == B.MOE_OK
    assert fn(t=B.TYPE_F32, N=7, K=32) == B.MOE_OK
    assert fn(xs=P + 1, ws=P + 3, out=P + 2) == B.MOE_OK
    assert fn(out=P + 2, t=B.TYPE_F32) == B.MOE_EALIGN
    assert fn(**{rows: 0}, x=None, xs=None, w=None, ws=None, out=None) == B.MOE_OK
    for k in ("x", "xs", "w", "ws", "out"):
        assert fn(**{k: None}) == B.MOE_EINVAL
    assert fn(x=P + 8) == B.MOE_EALIGN
    assert fn(w=P + 4) == B.MOE_EALIGN
    assert fn(ldx=264) == B.MOE_EALIGN
    assert fn(ldx=240) == B.MOE_EINVAL
    assert fn(ldo=255) == B.MOE_EINVAL
    assert fn(ldo=257) == B.MOE_OK
    for t in (-1, 2, B.TYPE_BF16 | B.SUM_F32):  # (the sums are fp32 in any case: no flag)
        assert fn(t=t) == B.MOE_EINVAL
    for bad in (dict(N=0), dict(K=0), {rows: -1}):
        assert fn(**bad) == B.MOE_EINVAL
    for big in (dict(K=528), dict(K=65568), dict(N=65537), {rows: 1 << 28}, dict(ldx=(1 << 22) + 16),
                dict(ldo=(1 << 22) + 1)):
        assert fn(**big) == B.MOE_EUNSUPPORTED, big


def test_grouped_arguments():
    assert _grouped(E=0) == B.MOE_EINVAL
    assert _grouped(E=257) == B.MOE_EUNSUPPORTED
    assert _grouped(off=None) == B.MOE_EINVAL
    assert _grouped(off=P + 2) == B.MOE_EALIGN
    assert _grouped(x_rows=3) == B.MOE_EINVAL
    assert _grouped(x_rows=1, idx=P, div=8) == B.MOE_OK
    assert _grouped(x_rows=0, idx=P) == B.MOE_EINVAL
    assert _grouped(idx=P + 2) == B.MOE_EALIGN
    assert _grouped(idx=P, div=0) == B.MOE_EINVAL
    assert _grouped(div=2) == B.MOE_EINVAL
    assert _grouped(x_rows=-1) == B.MOE_EINVAL
    assert _grouped(idx=P, x_rows=(1 << 31) // 256) == B.MOE_EUNSUPPORTED
    assert _grouped(idx=P, x_rows=(1 << 31) // 256 - 1) == B.MOE_OK


def _sort(T=100, E=16, K=4, ids=P, first=0, off=P, order=P, pos=P, ws=P, nbytes=1 << 30):
    return B.lib().moe_sort_routes_validate(T, E, K, ids, first, off, order, pos, ws, nbytes)


def test_sort_arguments():
    assert _sort() == B.MOE_OK
    assert _sort(first=-2 ** 31) == B.MOE_OK and _sort(first=2 ** 31 - 1) == B.MOE_OK
    assert _sort(T=0, ids=None, order=None, pos=None, ws=None, nbytes=0) == B.MOE_OK
    for k in ("ids", "off", "order", "pos"):
        assert _sort(**{k: None}) == B.MOE_EINVAL
        assert _sort(**{k: P + 2}) == B.MOE_EALIGN
    for bad in (dict(T=-1), dict(E=0), dict(K=0)):
        assert _sort(**bad) == B.MOE_EINVAL
    for big in (dict(E=257), dict(K=9), dict(T=1 << 26, K=4), dict(T=2 ** 31 - 1, K=8)):
        assert _sort(**big) == B.MOE_EUNSUPPORTED
    many = B.sort_workspace_bytes(1 << 20, 256, 8)
    if many:  # (few routes need none)
        assert _sort(T=1 << 20, E=256, K=8, nbytes=many) == B.MOE_OK
        assert _sort(T=1 << 20, E=256, K=8, nbytes=many - 1) == B.MOE_EWORKSPACE
        assert _sort(T=1 << 20, E=256, K=8, ws=None) == B.MOE_EINVAL
        assert _sort(T=1 << 20, E=256, K=8, ws=P + 8) == B.MOE_EALIGN
    assert B.sort_workspace_bytes(8, 256, 8) == 0
    assert _sort(T=8, E=256, K=8, ws=None, nbytes=0) == B.MOE_OK


def _gather(T=10, K=4, rows=40, cols=64, x=P, ldx=None, t=B.TYPE_BF16, pos=P, taken=None, out=P, ldo=None):
    return B.lib().moe_gather_rows_validate(T, K, rows, cols, x, cols if ldx is None else ldx, t, pos, taken, out,
                                            cols if ldo is None else ldo)


def _combine(T=10, K=4, rows=40, cols=64, x=P, ldx=None, t=B.TYPE_BF16, pos=P, w=P, out=P, ldo=None, ot=B.TYPE_BF16):
    return B.lib().moe_combine_rows_validate(T, K, rows, cols, x, cols if ldx is None else ldx, t, pos, w, out,
                                             cols if ldo is None else ldo, ot)


def _back(T=10, K=4, rows=40, cols=64, g=P, ldg=None, gt=B.TYPE_BF16, x=P, ldx=None, t=B.TYPE_BF16, pos=P, w=P,
          taken=None, gr=P, ldr=None, gw=P):
    return B.lib().moe_combine_rows_backward_validate(
        T, K, rows, cols, g, cols if ldg is None else ldg, gt, x, cols if ldx is None else ldx, t, pos, w, taken, gr,
        cols if ldr is None else ldr, gw)


@pytest.mark.parametrize("fn", [_gather, _combine, _back])
def test_rows_arguments(fn):
    assert fn() == B.MOE_OK
    assert fn(cols=1) == B.MOE_OK and fn(cols=65536) == B.MOE_OK
    assert fn(x=P + 2, ldx=65) == B.MOE_OK
    assert fn(x=P + 1) == B.MOE_EALIGN
    assert fn(x=P + 2, t=B.TYPE_F32) == B.MOE_EALIGN
    assert fn(pos=P + 2) == B.MOE_EALIGN
    assert fn(pos=None) == B.MOE_EINVAL and fn(x=None) == B.MOE_EINVAL
    assert fn(ldx=63) == B.MOE_EINVAL
    assert fn(t=2) == B.MOE_EINVAL
    for bad in (dict(T=-1), dict(K=0), dict(rows=-1), dict(cols=0)):
        assert fn(**bad) == B.MOE_EINVAL
    for big in (dict(K=9), dict(T=1 << 26), dict(rows=1 << 28), dict(cols=65537), dict(ldx=(1 << 22) + 1)):
        assert fn(**big) == B.MOE_EUNSUPPORTED


def test_rows_outputs_arguments():
    for fn in (_gather, _combine):
        assert fn(out=None) == B.MOE_EINVAL
        assert fn(ldo=63) == B.MOE_EINVAL
        assert fn(ldo=(1 << 22) + 1) == B.MOE_EUNSUPPORTED
        assert fn(out=P + 1) == B.MOE_EALIGN
    assert _gather(T=0, x=None, pos=None) == B.MOE_OK
    assert _gather(rows=0, out=None) == B.MOE_OK
    assert _gather(taken=P + 4) == B.MOE_OK and _gather(taken=P + 2) == B.MOE_EALIGN
    assert _combine(w=None) == B.MOE_OK and _combine(w=P + 2) == B.MOE_EALIGN
    assert _combine(ot=B.TYPE_F32, out=P + 2) == B.MOE_EALIGN
    assert _combine(ot=7) == B.MOE_EINVAL
    assert _combine(T=0, pos=None, w=None, out=None) == B.MOE_OK
    assert _combine(rows=0, x=None) == B.MOE_OK      # (tokens without any row: zeros)
    assert _back(gr=None, gw=None) == B.MOE_EINVAL
    assert _back(gr=None) == B.MOE_OK and _back(gw=None, x=None) == B.MOE_OK and _back(w=None) == B.MOE_OK
    assert _back(gw=P + 2) == B.MOE_EALIGN and _back(g=None) == B.MOE_EINVAL
    assert _back(g=P + 2, gt=B.TYPE_F32) == B.MOE_EALIGN and _back(gt=5) == B.MOE_EINVAL
    assert _back(ldg=63) == B.MOE_EINVAL and _back(ldr=63) == B.MOE_EINVAL
    assert _back(taken=P + 2) == B.MOE_EALIGN and _back(taken=P) == B.MOE_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 64))
    codes, scales = torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 2), dtype=torch.uint8)
    routes = dict(offsets=torch.zeros(3, dtype=torch.int32), positions=torch.zeros((2, 2), dtype=torch.int32))
    for call in (lambda: B.fp4_quantize(x), lambda: B.fp4_swiglu(torch.zeros((2, 128))),
                 lambda: B.fp4_dequantize(codes, scales), lambda: B.fp4_linear(codes, scales, codes, scales),
                 lambda: B.fp4_grouped(codes, scales, routes["offsets"], codes[None], scales[None]),
                 lambda: B.sort_routes(routes["positions"], 2), lambda: B.gather_rows(x, routes),
                 lambda: B.combine_rows(x, routes), lambda: B.combine_rows_backward(x, x, routes),
                 lambda: B.gather_rows(x.requires_grad_(), routes)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_given_stream_holds_every_tensor_of_the_call(monkeypatch):
    """What a call on a stream of its own reads or writes is recorded on that stream before anything is
    enqueued; a stream of another device is refused before that."""
    held, enqueued = set(), []
    monkeypatch.setattr(B, "_device", lambda t: t.device)
    monkeypatch.setattr(B, "_empty", lambda shape, dtype, dev, stream: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(B, "_run", lambda *a: enqueued.append(set(held)))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.add((t.data_ptr(), id(s))))
    mine = types.SimpleNamespace(device=torch.device("cpu"), cuda_stream=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)

    def run(fn, reads, *args, **named):
        held.clear()
        with pytest.raises(ValueError, match="stream"):
            fn(*args, **named, stream=other)
        assert not held, fn.__name__
        for stream in (mine, None):
            held.clear()
            fn(*args, **named, stream=stream)
            want = {(t.data_ptr(), id(stream)) for t in reads} if stream else set()
            assert want <= enqueued[-1] and (stream or not enqueued[-1]), (fn.__name__, stream)

    u8, i32 = torch.uint8, torch.int32
    x = torch.zeros((4, 256))
    c, s = torch.zeros((4, 128), dtype=u8), torch.zeros((4, 8), dtype=u8)
    run(B.fp4_quantize, (x, c, s), x, c, s)
    run(B.fp4_quantize, (x,), x)
    run(B.fp4_swiglu, (x,), x)
    run(B.fp4_dequantize, (c, s, x), c, s, out=x)
    run(B.fp4_dequantize, (c, s), c, s)
    w, ws, off = torch.zeros((2, 16, 128), dtype=u8), torch.zeros((2, 16, 8), dtype=u8), torch.zeros(3, dtype=i32)
    out, idx = torch.zeros((6, 16)), torch.zeros(6, dtype=i32)
    run(B.fp4_linear, (c, s, w[0], ws[0], out), c, s, w[0], ws[0], out=out[:4])
    run(B.fp4_grouped, (c, s, off, w, ws, idx, out), c, s, off, w, ws, row_index=idx, out=out)
    ids, sw = torch.zeros((900, 4), dtype=i32), torch.zeros(1 << 16, dtype=u8)
    run(B.sort_routes, (ids, sw), ids, 8, ws=sw)
    routes = dict(offsets=off, sorted=torch.zeros(8, dtype=i32), positions=torch.zeros((4, 2), dtype=i32))
    rows, wt = torch.zeros((8, 256)), torch.zeros((4, 2))
    run(B.gather_rows, (x, off, routes["positions"], rows), x, routes, out=rows, zero_rest=True)
    run(B.gather_rows_backward, (rows, routes["positions"], x), rows, routes, out=x)
    run(B.combine_rows, (rows, routes["positions"], wt, x), rows, routes, wt, out=x)
    run(B.combine_rows_backward, (x, rows, routes["positions"], off, wt), x, rows, routes, wt, zero_rest=True)
    run(B.combine_rows_backward, (x, rows, routes["positions"], wt, rows), x, rows, routes, wt, grad_rows=torch.zeros((8, 256)))


def test_sizes_past_32_bits_are_refused():
    for call in (lambda: B.sort_workspace_bytes(2 ** 32 + 4096, 16, 4), lambda: B.sort_workspace_bytes(4, 2 ** 40, 4)):
        with pytest.raises(ValueError, match="32-bit"):
            call()


# ---- the oracle --------------------------------------------------------------

def test_oracle_codes_are_the_nearest():
    table = torch.tensor(R.VALUES, dtype=torch.float64)
    q = torch.cat([torch.linspace(0, 6.999, 20001, dtype=torch.float64), (table[1:] + table[:-1]) / 2])
    code = R.e2m1_codes(q)
    off = (q - table[code]).abs()
    assert bool((off <= (q[:, None] - table[None, :]).abs().amin(1)).all())
    ties = (table[1:] + table[:-1]) / 2
    assert bool((R.e2m1_codes(ties) % 2 == 0).all())
    assert torch.equal(R.e2m1_codes(-q) & 8, torch.full_like(code, 8))


def test_oracle_scales_never_saturate():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((200, 64), generator=g) * torch.exp(20 * torch.randn((200, 1), generator=g))
    x[0] = 1.75
    x[1] = torch.nextafter(torch.tensor(1.75), torch.tensor(0.0))
    x[2] = 7.0
    x[3] = 2.0 ** -149
    x[4] = torch.finfo(torch.float32).max
    codes, scales = R.quantize(x.double())
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    q = x.double() / s
    assert bool((q.abs() < 7).all())
    assert bool(((R.values(codes, scales) - x.double()).abs() <= R.half_step(q) * s).all())
    # the smallest scale that does it, but for the bound at 2^-126
    tight = (q.abs().view(200, 2, 32).amax(2) >= 3.5) | (scales == 1)
    assert bool(tight.all())
    assert scales[0, 0] == scales[1, 0] + 1


def test_oracle_matches_the_layers_weights():
    """The bytes mean what the layer's oracle takes them for."""
    import oracle

    g = torch.Generator().manual_seed(4)
    codes, scales = R.random_codes((5, 48), g), R.random_scales((5, 3), g)
    v = R.values(codes, scales)
    for n in range(5):
        for k in (0, 1, 31, 32, 63, 64, 95):
            assert oracle.mxfp4_value(codes.numpy(), scales.numpy(), 96, n, k) == float(v[n, k])


def test_oracle_product_bound_notices_a_lost_group():
    g = torch.Generator().manual_seed(5)
    x, xs, w, ws = (R.random_codes((9, 128), g), R.random_scales((9, 8), g), R.random_codes((33, 128), g),
                    R.random_scales((33, 8), g))
    out, mag = R.product(x, xs, w, ws)
    for dtype in (torch.float32, torch.bfloat16):
        good = out.to(torch.float32).to(dtype).double()
        assert bool(((good - out).abs() <= R.product_bound(out, mag, 256, dtype)).all())
    xs2 = xs.clone()
    xs2[:, 3] += 1
    worse, _ = R.product(x, xs2, w, ws)
    assert float(((worse - out).abs() > R.product_bound(out, mag, 256, torch.bfloat16)).double().mean()) > 0.3
