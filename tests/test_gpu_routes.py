"""Routes sorted by expert, the rows' way into that order and back, and the
gradients, against plain 64-bit definitions: empty and foreign experts, tokens
without routes, odd widths, strides, both types, streams, graphs, autograd."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
B = pytest.importorskip("latent_mixture_experts_amd.binding")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative
TYPES = [torch.bfloat16, torch.float32]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def sort_ref(ids, E, first=0):
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    positions = torch.empty_like(order)
    positions[order] = torch.arange(order.numel())
    order = torch.where(torch.arange(order.numel()) < offsets[-1], order, torch.full_like(order, -1))
    positions = torch.where(key < E, positions, torch.full_like(positions, -1))
    return {k: v.to(torch.int32) for k, v in dict(offsets=offsets, sorted=order, positions=positions.view(ids.shape)).items()}


def same(got, want):
    return all(torch.equal(got[k].cpu(), want[k]) for k in ("offsets", "sorted", "positions"))


def random_ids(T, K, E, g, spread=None):
    """Experts of each token, some twice, some none of ours."""
    return torch.randint(-1, E + 1 if spread is None else spread, (T, K), generator=g).to(torch.int32)


# ---- sort --------------------------------------------------------------------

@pytest.mark.parametrize("T,K,E", [(0, 4, 8), (1, 1, 1), (1, 8, 256), (7, 3, 5), (16, 4, 2), (61, 4, 16), (64, 8, 256), (100, 8, 256),
                                   (768, 8, 256), (769, 8, 256), (1000, 5, 100), (4096, 8, 256), (5000, 7, 33), (32767, 8, 256),
                                   (60000, 8, 256), (300000, 3, 7), (700001, 8, 256)])
def test_sort(T, K, E):
    ids = random_ids(T, K, E, gen(T + K))
    assert same(B.sort_routes(ids.cuda(), E), sort_ref(ids, E))


@pytest.mark.parametrize("T", [9, 2000, 40000])
def test_sort_edges(T):
    g = gen(T)
    K = 4
    for ids, E, first in (
            (torch.full((T, K), 3), 8, 0),                        # all to one expert
            (torch.full((T, K), -1), 8, 0),                       # none
            (torch.randint(0, 256, (T, K), generator=g), 32, 96),  # the experts of one of eight processes
            (torch.randint(0, 256, (T, K), generator=g), 256, -255),
            (torch.randint(0, 256, (T, K), generator=g), 1, 255),
            (torch.randint(-(1 << 31), (1 << 31) - 1, (T, K), generator=g), 200, 0),
            (torch.where(torch.rand((T, K), generator=g) < 0.5, (1 << 31) - 1, -(1 << 31)), 256, -(1 << 31)),
            (torch.where(torch.rand((T, K), generator=g) < 0.5, (1 << 31) - 1, -(1 << 31)), 256, (1 << 31) - 1)):
        ids = ids.to(torch.int32)
        assert same(B.sort_routes(ids.cuda(), E, first), sort_ref(ids, E, first)), (E, first)


def test_sort_is_moe_routes_grouping():
    from latent_mixture_experts_amd import synth

    dims = dict(hidden=256, latent=128, inter=128, n_experts=48, top_k=6)
    lay = synth.make_layer(dims, 90, seed=2)
    d = B.make_dims(dims)
    r = B.route(d, torch.from_numpy(lay.x).view(torch.int16).cuda(), torch.from_numpy(lay.router).cuda(), B.alloc_workspace(d, 90))
    s = B.sort_routes(r["ids"], 48)
    assert torch.equal(s["offsets"], r["offsets"]) and torch.equal(s["sorted"], r["sorted"])


def test_sort_refusals():
    ids = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    for bad in (lambda: B.sort_routes(ids.long(), 4), lambda: B.sort_routes(ids[0], 4), lambda: B.sort_routes(ids.t(), 4),
                lambda: B.sort_routes(ids, -1), lambda: B.sort_routes(ids, 1 << 40), lambda: B.sort_routes(ids, 4, 1 << 31)):
        with pytest.raises(ValueError):
            bad()
    for status, bad in ((B.MOE_EINVAL, lambda: B.sort_routes(ids, 0)), (B.MOE_EUNSUPPORTED, lambda: B.sort_routes(ids, 257)),
                        (B.MOE_EUNSUPPORTED, lambda: B.sort_routes(torch.zeros((4, 9), dtype=torch.int32, device="cuda"), 4))):
        with pytest.raises(B.MoeError) as e:
            bad()
        assert e.value.status == status


# ---- rows --------------------------------------------------------------------

SHAPES = [(1, 1, 1, 1), (1, 8, 16, 4096), (3, 2, 4, 7), (5, 8, 8, 8), (9, 3, 4, 100), (17, 4, 8, 384), (33, 8, 64, 130),
          (61, 4, 16, 1000), (200, 6, 32, 513), (257, 8, 256, 2048), (1030, 5, 7, 264), (4099, 2, 16, 33), (2, 8, 8, 65536)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,E,C", SHAPES)
def test_gather_and_its_gradient(T, K, E, C, dtype):
    g = gen(T + C)
    ids = random_ids(T, K, E, g)
    routes = B.sort_routes(ids.cuda(), E)
    order, taken = routes["sorted"].cpu().long(), int(routes["offsets"][-1])
    x = torch.randn((T, C), generator=g).to(dtype)
    want = x[order[:taken] // K]
    out = torch.full((T * K, C), -5.0, dtype=dtype, device="cuda")
    assert B.gather_rows(x.cuda(), routes, out=out) is out
    assert torch.equal(out[:taken].cpu(), want) and (out[taken:] == -5).all()
    out = B.gather_rows(x.cuda(), routes, zero_rest=True)
    assert torch.equal(out[:taken].cpu(), want) and (out[taken:] == 0).all()

    drows = torch.randn((T * K, C), generator=g).to(dtype)
    drows[taken:] = float("nan")  # (read by nobody)
    dx = B.gather_rows_backward(drows.cuda(), routes)
    terms = torch.zeros((T, K, C), dtype=torch.float64)
    at = routes["positions"].cpu().long()
    terms[at >= 0] = drows[at[at >= 0]].double()
    want, mag = terms.sum(1), terms.abs().sum(1)
    # K sums of half a step of fp32, one rounding to the type
    assert dx.dtype == dtype
    assert bool(((dx.cpu().double() - want).abs() <= mag * K * HALF[torch.float32] + want.abs() * HALF[dtype] * 1.01).all())


@pytest.mark.parametrize("C", [64, 61])
def test_gather_moves_every_bit_pattern(C):
    """Subnormal values, infinities and NaN of any payload as they are, in both types."""
    T = (65536 + C - 1) // C
    routes = B.sort_routes(torch.arange(T, dtype=torch.int32).remainder(7)[:, None].cuda(), 7)
    order = routes["sorted"].long()
    x = torch.arange(T * C, dtype=torch.int32).to(torch.int16).view(T, C).cuda()
    assert torch.equal(B.gather_rows(x, routes), x[order])
    y = torch.randint(-(1 << 31), (1 << 31) - 1, (T, C), generator=gen(C)).to(torch.int32)
    y[0, :4] = torch.tensor([1, 0x7F800001, -1, 0x00400000])
    y = y.cuda().view(torch.float32)
    assert torch.equal(B.gather_rows(y, routes).view(torch.int32), y.view(torch.int32)[order])


@pytest.mark.parametrize("out_dtype", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,E,C", SHAPES)
def test_combine_and_its_gradient(T, K, E, C, dtype, out_dtype):
    g = gen(T * 3 + C)
    ids = random_ids(T, K, E, g)
    routes = B.sort_routes(ids.cuda(), E)
    at, taken = routes["positions"].cpu().long(), int(routes["offsets"][-1])
    rows = torch.randn((T * K, C), generator=g).to(dtype)
    rows[taken:] = float("nan")
    w = torch.randn((T, K), generator=g)
    w[at < 0] = float("nan")  # (weights of routes that are not here are read by nobody)
    mine = torch.zeros((T, K, C), dtype=torch.float64)
    mine[at >= 0] = rows[at[at >= 0]].double()
    wd = torch.where(at >= 0, w, torch.zeros(())).double()
    out = B.combine_rows(rows.cuda(), routes, w.cuda(), out_dtype)
    terms = wd[:, :, None] * mine
    want, mag = terms.sum(1), terms.abs().sum(1)
    assert out.dtype == out_dtype
    # K multiply-adds of half a step each, one rounding
    assert bool(((out.cpu().double() - want).abs() <= mag * K * HALF[torch.float32] + want.abs() * HALF[out_dtype] * 1.01).all())

    dout = torch.randn((T, C), generator=g).to(out_dtype)
    drows, dw = B.combine_rows_backward(dout.cuda(), rows.cuda(), routes, w.cuda(), zero_rest=True)
    want = torch.zeros((T * K, C), dtype=torch.float64)
    want[at[at >= 0]] = (wd[:, :, None] * dout.double()[:, None, :])[at >= 0]
    assert drows.dtype == dtype
    assert bool(((drows.cpu().double() - want).abs() <= want.abs() * (HALF[torch.float32] + HALF[dtype]) * 1.01).all())
    terms = mine * dout.double()[:, None, :]
    # a sum of C products: each multiply-add, and each join, half a step of the sizes so far
    assert bool(((dw.cpu().double() - terms.sum(2)).abs() <= terms.abs().sum(2) * (C + 16) * HALF[torch.float32]).all())
    # one gradient alone, and rows behind the last left as they were
    given = torch.full((T * K, C), -5.0, dtype=dtype, device="cuda")
    only, none = B.combine_rows_backward(dout.cuda(), rows.cuda(), routes, w.cuda(), want_w=False, grad_rows=given)
    assert none is None and only is given and torch.equal(given[:taken], drows[:taken]) and (given[taken:] == -5).all()
    none, only = B.combine_rows_backward(dout.cuda(), rows.cuda(), routes, w.cuda(), want_rows=False)
    assert none is None and torch.equal(only, dw)


def test_combine_gradient_against_differences():
    """dw and drows against differences of the GPU's own sums, in fp32 on values where the differences are exact:
    small integers over powers of two."""
    g = gen(4)
    T, K, E, C = 6, 3, 5, 40
    ids = random_ids(T, K, E, g)
    routes = B.sort_routes(ids.cuda(), E)
    rows = torch.randint(-8, 9, (T * K, C), generator=g).float().cuda()
    w = torch.randint(-8, 9, (T, K), generator=g).float().cuda() / 8
    dout = torch.randint(-4, 5, (T, C), generator=g).float().cuda()
    f = lambda a, b: (B.combine_rows(a, routes, b).double() * dout.double()).sum()
    drows, dw = B.combine_rows_backward(dout, rows, routes, w, zero_rest=True)
    base = f(rows, w)
    for t in range(T):
        for k in range(K):
            b = w.clone()
            b[t, k] += 1
            assert float(f(rows, b) - base) == float(dw[t, k])
    for i in range(T * K):
        for c in (0, 17, C - 1):
            a = rows.clone()
            a[i, c] += 1
            assert float(f(a, w) - base) == float(drows[i, c])


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan_travel_by_their_routes(dtype):
    ids = torch.tensor([[0, 1], [1, 0], [-1, 0]], dtype=torch.int32).cuda()
    routes = B.sort_routes(ids, 2)
    at = routes["positions"].cpu()
    rows = torch.ones((6, 16), dtype=dtype)
    rows[at[0, 0], 3] = float("inf")
    rows[at[1, 1], 5] = float("nan")
    w = torch.tensor([[1.0, 2.0], [1.0, 1.0], [float("nan"), -1.0]])
    out = B.combine_rows(rows.cuda(), routes, w.cuda(), torch.float32).cpu()
    assert torch.isinf(out[0, 3]) and torch.isnan(out[1, 5])
    assert int((~torch.isfinite(out)).sum()) == 2 and (out[2] == -1).all()
    zero = B.combine_rows(rows.cuda(), routes, torch.zeros((3, 2)).cuda(), torch.float32).cpu()
    assert torch.isnan(zero[0, 3]) and zero[0, 2] == 0  # 0 * inf, as the formula has it


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [64, 61])
def test_strides(C, dtype):
    """Rows at any pitch, on either side, off 16 bytes."""
    g = gen(C)
    T, K, E = 23, 3, 6
    ids = random_ids(T, K, E, g)
    routes = B.sort_routes(ids.cuda(), E)
    for shift, pitch in ((8, 80), (3, 71)):
        wide = torch.randn((T, pitch + 16), generator=g).to(dtype).cuda()
        x = wide[:, shift:shift + C]
        hold = torch.full((T * K, pitch + 16), -5.0, dtype=dtype, device="cuda")
        B.gather_rows(x, routes, out=hold[:, shift:shift + C], zero_rest=True)
        want = B.gather_rows(x.contiguous(), routes, zero_rest=True)
        assert torch.equal(hold[:, shift:shift + C], want)
        assert (hold[:, :shift] == -5).all() and (hold[:, shift + C:] == -5).all()
        w = torch.randn((T, K), generator=g).cuda()
        out = torch.full((T, pitch + 16), -5.0, device="cuda")
        B.combine_rows(hold[:, shift:shift + C], routes, w, out=out[:, shift:shift + C])
        assert torch.equal(out[:, shift:shift + C], B.combine_rows(want, routes, w, torch.float32))
        assert (out[:, :shift] == -5).all() and (out[:, shift + C:] == -5).all()
        drows = torch.full((T * K, pitch + 16), -5.0, dtype=dtype, device="cuda")
        a = B.combine_rows_backward(out[:, shift:shift + C], hold[:, shift:shift + C], routes, w, zero_rest=True,
                                    grad_rows=drows[:, shift:shift + C])
        b = B.combine_rows_backward(out[:, shift:shift + C].contiguous(), want, routes, w, zero_rest=True)
        # (dots in another order: each within C + 16 roundings of its terms' sizes)
        at = routes["positions"].long()
        mine = torch.where((at >= 0)[:, :, None], want.double()[at.clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda"))
        mag = (mine.abs() * out[:, shift:shift + C].double().abs()[:, None, :]).sum(2)
        assert torch.equal(a[0], b[0])
        assert bool(((a[1].double() - b[1].double()).abs() <= 2 * (C + 16) * HALF[torch.float32] * mag).all())
        assert (drows[:, :shift] == -5).all() and (drows[:, shift + C:] == -5).all()


def test_fewer_rows_than_routes_and_bad_positions():
    """Positions outside the rows are none: no access outside the buffers."""
    T, K, C = 40, 4, 32
    g = gen(1)
    hold = torch.full((30 + 64, C), -5.0, device="cuda")
    out = hold[32:62]
    positions = torch.randperm(T * K, generator=g).view(T, K).to(torch.int32)
    positions[0] = torch.tensor([-1, 30, 1 << 30, -(1 << 31)])
    routes = dict(offsets=torch.tensor([0, 1 << 30], dtype=torch.int32).cuda(), positions=positions.cuda())
    x = torch.randn((T, C), generator=g)
    B.gather_rows(x.cuda(), routes, out=out, zero_rest=True)
    assert (hold[:32] == -5).all() and (hold[62:] == -5).all()
    back = B.combine_rows(out, routes).cpu()
    inside = ((positions >= 0) & (positions < 30)).sum(1)
    assert torch.allclose(back, x * inside[:, None], rtol=1e-6)
    routes["offsets"] = torch.tensor([-77], dtype=torch.int32).cuda()
    drows = torch.full((30 + 64, C), -5.0, device="cuda")
    B.combine_rows_backward(x.cuda(), out, dict(routes, positions=torch.full((T, K), -1, dtype=torch.int32).cuda()),
                            zero_rest=True, grad_rows=drows[32:62])
    assert (drows[:32] == -5).all() and (drows[62:] == -5).all() and (drows[32:62] == 0).all()
    empty = B.combine_rows(torch.empty((0, C), device="cuda"), routes)
    assert empty.shape == (T, C) and (empty == 0).all()
    none = dict(offsets=torch.zeros(1, dtype=torch.int32).cuda(), positions=torch.empty((0, 4), dtype=torch.int32).cuda())
    assert B.combine_rows(out, none).shape == (0, C)
    grad, dw = B.combine_rows_backward(torch.empty((0, C), device="cuda"), out, none, zero_rest=True)
    assert (grad == 0).all() and dw.shape == (0, 4)


def test_offsets_past_32_bits():
    T, K, C = 80000, 4, 8192  # rows of 5 GiB in bf16, 2.6e9 values
    x = torch.randn((T, C), device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(2))
    ids = torch.randint(0, 8, (T, K), device="cuda", dtype=torch.int32)
    routes = B.sort_routes(ids, 8)
    rows = B.gather_rows(x, routes)
    assert rows.numel() > 1 << 31
    at = torch.cat([torch.arange(50), torch.arange(T * K - 50, T * K)]).cuda()
    assert torch.equal(rows[at], x[routes["sorted"][at].long() // K])
    back = B.combine_rows(rows, routes)
    assert torch.equal(back[-50:], (x[-50:].float() * 4).bfloat16()) and torch.equal(back[:50], (x[:50].float() * 4).bfloat16())
    grad, _ = B.combine_rows_backward(x, rows, routes, want_w=False)
    assert torch.equal(grad[at], rows[at])


def test_rows_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    routes = B.sort_routes(ids, 3)
    x, rows = torch.zeros((4, 16), device="cuda"), torch.zeros((8, 16), device="cuda")
    for bad in (lambda: B.gather_rows(x[:3], routes), lambda: B.gather_rows(x.half(), routes),
                lambda: B.gather_rows(x, routes, out=rows.bfloat16()), lambda: B.gather_rows(x, routes, out=rows[:, :8]),
                lambda: B.gather_rows(x[:, ::2], routes), lambda: B.gather_rows(x, dict(routes, positions=ids.long())),
                lambda: B.combine_rows(rows, routes, torch.zeros((4, 3), device="cuda")),
                lambda: B.combine_rows(rows, routes, torch.zeros((4, 2), device="cuda").bfloat16()),
                lambda: B.combine_rows(rows, routes, out_dtype=torch.float16),
                lambda: B.combine_rows(rows[0], routes), lambda: B.combine_rows(rows, routes, torch.zeros((4, 2))),
                lambda: B.combine_rows_backward(x[:, :8], rows, routes),
                lambda: B.combine_rows_backward(x, rows, routes, want_rows=False, grad_rows=rows),
                lambda: B.combine_rows(rows.requires_grad_(), routes, out=x),
                lambda: B.gather_rows(x.clone().requires_grad_(), routes, out=rows.detach())):
        with pytest.raises(ValueError):
            bad()


# ---- autograd, streams, graphs -------------------------------------------------

def test_training_step_with_autograd():
    """gather -> expert products -> combine -> loss, with the balance loss, in fp32 against autograd on plain indexing."""
    g = gen(11)
    T, K, E, C, F = 50, 4, 8, 32, 24
    logits = torch.randn((T, E), generator=g).cuda().requires_grad_()
    x = torch.randn((T, C), generator=g).cuda().requires_grad_()
    weights = (torch.randn((E, F, C), generator=g) / 6).cuda().requires_grad_()
    target = torch.randn((T, F), generator=g).cuda()

    def step(own):
        best = logits.topk(K, 1)
        ids, w = best.indices.to(torch.int32), torch.softmax(best.values, 1)
        if own:
            routes = B.sort_routes(ids, E)
            rows = B.gather_rows(x, routes)
            off = routes["offsets"].tolist()
            y = torch.cat([rows[a:b] @ weights[e].t() for e, (a, b) in enumerate(zip(off, off[1:]))])
            out = B.combine_rows(y, routes, w)
        else:
            y = torch.stack([x @ weights[e].t() for e in range(E)], 1)  # [T][E][F]
            out = (w[:, :, None] * torch.gather(y, 1, ids.long()[:, :, None].expand(-1, -1, F))).sum(1)
        loss = ((out - target) ** 2).mean()
        grads = torch.autograd.grad(loss, (x, weights, logits))
        return loss, grads

    la, ga = step(True)
    lb, gb = step(False)
    assert torch.allclose(la, lb, rtol=1e-5)
    for a, b in zip(ga, gb):  # (the same sums in other orders: dozens of fp32 roundings of the terms' sizes)
        assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max())


@pytest.mark.parametrize("dtype", TYPES)
def test_autograd_is_the_backward_call(dtype):
    g = gen(12)
    T, K, E, C = 30, 3, 5, 48
    ids = random_ids(T, K, E, g)
    routes = B.sort_routes(ids.cuda(), E)
    x = torch.randn((T, C), generator=g).to(dtype).cuda().requires_grad_()
    rows = B.gather_rows(x, routes)
    taken = int(routes["offsets"][-1])
    assert (rows[taken:] == 0).all()
    w = torch.randn((T, K), generator=g).cuda().requires_grad_()
    leaf = rows.detach().requires_grad_()
    out = B.combine_rows(leaf, routes, w, torch.float32)
    out.sum().backward()  # (an expanded gradient)
    a, b = B.combine_rows_backward(torch.ones_like(out), leaf.detach(), routes, w.detach(), zero_rest=True)
    assert torch.equal(leaf.grad, a) and torch.equal(w.grad, b)
    rows.backward(a)
    assert torch.equal(x.grad, B.gather_rows_backward(a, routes))
    # weights alone, rows alone, neither
    w2 = w.detach().requires_grad_()
    B.combine_rows(leaf.detach(), routes, w2).sum().backward()
    assert w2.grad is not None
    r2 = leaf.detach().requires_grad_()
    B.combine_rows(r2, routes).sum().backward()
    assert torch.equal(r2.grad, B.gather_rows(torch.ones((T, C), dtype=dtype, device="cuda"), routes, zero_rest=True))
    with torch.no_grad():
        assert not B.combine_rows(r2, routes, w2).requires_grad
    y = B.gather_rows(x, routes).sum()
    with pytest.raises(RuntimeError, match="twice"):
        torch.autograd.grad(y, x, create_graph=True)


def test_gradients_are_refused_in_a_capture():
    g = gen(13)
    routes = B.sort_routes(random_ids(8, 2, 4, g).cuda(), 4)
    x = torch.randn((8, 16), generator=g).cuda().requires_grad_()
    w = torch.rand((8, 2), generator=g).cuda().requires_grad_()
    rows = torch.randn((16, 16), generator=g).cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="capture"):
            B.gather_rows(x, routes)
        with pytest.raises(ValueError, match="capture"):
            B.combine_rows(rows, routes, w)
        a = B.gather_rows(x.detach(), routes, zero_rest=True)
        out = B.combine_rows(a, routes, w.detach())
        drows, dw = B.combine_rows_backward(out, a, routes, w.detach(), zero_rest=True)
        dx = B.gather_rows_backward(drows, routes)
    with torch.no_grad():
        for i in range(3):
            x.normal_(generator=torch.Generator("cuda").manual_seed(i))
            graph.replay()
            torch.cuda.synchronize()
            a2 = B.gather_rows(x, routes, zero_rest=True)
            o2 = B.combine_rows(a2, routes, w)
            d2, w2 = B.combine_rows_backward(o2, a2, routes, w, zero_rest=True)
            assert torch.equal(a, a2) and torch.equal(out, o2) and torch.equal(drows, d2) and torch.equal(dw, w2)
            assert torch.equal(dx, B.gather_rows_backward(d2, routes))


def test_the_same_bits_every_time_and_on_two_streams():
    g = gen(16)
    T, K, E, C = 900, 8, 64, 1030
    ids, x, w = random_ids(T, K, E, g).cuda(), torch.randn((T, C), generator=g).cuda(), torch.rand((T, K), generator=g).cuda()

    def step(stream=None):
        routes = B.sort_routes(ids, E, stream=stream)
        rows = B.gather_rows(x, routes, zero_rest=True, stream=stream)
        out = B.combine_rows(rows, routes, w, stream=stream)
        return (*routes.values(), rows, out, *B.combine_rows_backward(out, rows, routes, w, zero_rest=True, stream=stream))

    want = step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [step(s) for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_sort_captured_and_replayed():
    g = gen(14)
    for T in (5, 3000, 20000):
        ids = random_ids(T, 4, 32, g).cuda()
        B.sort_routes(ids, 32)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            routes = B.sort_routes(ids, 32)
        for _ in range(3):
            ids.copy_(random_ids(T, 4, 32, g))
            graph.replay()
            torch.cuda.synchronize()
            assert same(routes, sort_ref(ids.cpu(), 32))


def test_other_stream_and_dropped_tensors():
    g = gen(15)
    ids = random_ids(3000, 4, 16, g)
    x = torch.randn((3000, 64), generator=g)
    side = torch.cuda.Stream()
    xd, idd = x.cuda(), ids.cuda()
    torch.cuda.synchronize()
    routes = B.sort_routes(idd, 16, stream=side)
    rows = B.gather_rows(xd, routes, zero_rest=True, stream=side)
    out = B.combine_rows(rows, routes, stream=side)
    grads = B.combine_rows_backward(out, rows, routes, zero_rest=True, stream=side)
    del xd, idd
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(4)]
    side.synchronize()
    assert same(routes, sort_ref(ids, 16))
    n = (routes["positions"] >= 0).sum(1).cpu()
    assert torch.allclose(out.cpu(), x * n[:, None], rtol=1e-6)
    assert grads[0].shape == (12000, 64)
    del junk


def test_rows_refilled_before_the_backward_pass_are_refused():
    """Frozen 4-bit experts, a trained router, one buffer of rows for every micro-batch."""
    g = gen(17)
    T, K, E, C = 20, 2, 4, 64
    routes = B.sort_routes(torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32).cuda(), E)
    w = B.fp4_quantize(torch.randn((E * C, C), generator=g).cuda())
    w = w[0].view(E, C, C // 2), w[1].view(E, C, C // 32)
    xs = [B.fp4_quantize(torch.randn((T * K, C), generator=g).cuda()) for _ in range(2)]
    buf = torch.empty((T * K, C), device="cuda")
    weights = torch.rand((T, K), generator=g).cuda().requires_grad_()
    B.fp4_grouped(*xs[0], routes["offsets"], *w, out=buf)
    y = B.combine_rows(buf, routes, weights)
    y.sum().backward(retain_graph=True)
    _, dw = B.combine_rows_backward(torch.ones_like(y), buf, routes, weights.detach())
    assert torch.equal(weights.grad, dw)
    B.fp4_grouped(*xs[1], routes["offsets"], *w, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    assert torch.equal(weights.grad, dw)
