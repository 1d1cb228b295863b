"""The balance loss, the routes per expert and the gradient of the router
logits on the GPU against 64 bits (tests/fp8_ref.py)."""
from __future__ import annotations

import pytest
import torch

from tests import fp8_ref as R

pytestmark = pytest.mark.gpu
B = pytest.importorskip("latent_mixture_experts_amd.binding")
INF = float("inf")


def case(T, E, K, masked, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed + T + E)
    logits = torch.randn((T, E), generator=g) * spread + torch.randn((1, E), generator=g)
    best = logits.topk(K, 1)
    ids, w = best.indices.to(torch.int32), torch.softmax(best.values, 1)
    dw = torch.randn((T, K), generator=g)
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if masked else None
    return logits, ids, w, dw, mask


def cuda(t):
    return None if t is None else t.cuda()


def check_loss(losses, counts, ref, ref_c):
    assert counts.cpu().tolist() == ref_c.tolist()
    # probabilities: exponential and quotient under 8 half steps; sums of positive terms: at most
    # 64 tokens of a row, 16 rows, 128 + 4 joins; f, the products and the sum over the experts 16 more
    rel = (8 + 64 + 16 + 132 + 16) * R.U24
    got = losses.cpu().double()
    assert abs(float(got[0] - ref[0])) <= rel * float(ref[0]) + 1e-30
    # lse^2: the logarithm's own error is absolute, a few steps of the sizes of maximum and logarithm
    assert abs(float(got[1] - ref[1])) <= 2 * rel * float(ref[1]) + 1e-12


def check_grad(got, ref, size):
    # per entry: expf, logf, the quotients and the two 256-term sums (16 in a lane, four joins): under 64 half steps
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= 64 * R.U24 * size + 1e-30).all()), float((err / (size + 1e-30)).max() / R.U24)


SHAPES = [(1, 1, 1), (1, 256, 8), (3, 5, 2), (16, 16, 4), (61, 16, 4), (64, 255, 8), (65, 64, 1), (100, 3, 3),
          (333, 130, 7), (1000, 256, 8), (9001, 256, 8), (20000, 12, 2), (40000, 66, 6)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_loss_and_gradient(T, E, K, masked):
    logits, ids, w, dw, mask = case(T, E, K, masked)
    gl = torch.tensor([0.7, 0.02])
    ref, ref_c, grad, size = R.balance(logits, ids, mask, gl, w, dw)
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda(), cuda(mask))
    check_loss(losses, counts, ref, ref_c)
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, gl.cuda(), cuda(mask), w.cuda(), dw.cuda())
    check_grad(got, grad, size)
    grad, size = R.balance(logits, ids, mask, gl)[2:]
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, gl.cuda(), cuda(mask))
    check_grad(got, grad, size)


@pytest.mark.parametrize("T", [50, 300])
def test_tokens_that_do_not_count(T):
    """Masked tokens may hold anything; tokens whose logits are all -inf do
    not count; -inf for some experts is a probability of zero."""
    logits, ids, w, dw, mask = case(T, 20, 4, True)
    logits[mask == 0] = float("nan")
    logits[3, :], mask[3] = -INF, 1
    logits[7, 5:], mask[7] = -INF, 1
    logits[9, :], mask[9] = torch.finfo(torch.float32).min, 1
    logits[11, :], mask[11] = 3e38, 1  # (lse^2 overflows: left to the balance loss alone)
    gl = torch.tensor([1.0, 0.0])
    ref, ref_c, grad, size = R.balance(logits, ids, mask, gl, w, dw)
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda(), mask.cuda())
    assert counts.cpu().tolist() == ref_c.tolist()
    assert abs(float(losses[0].cpu().double() - ref[0])) <= 300 * R.U24 * float(ref[0])
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, gl.cuda(), mask.cuda(), w.cuda(), dw.cuda())
    assert bool((got.cpu()[mask == 0] == 0).all()) and bool((got.cpu()[3] == 0).all())
    check_grad(got, grad, size)


@pytest.mark.parametrize("T", [0, 5, 200])
def test_nothing_counts(T):
    logits, ids, w, dw, _ = case(max(T, 1), 12, 3, False)
    logits, ids, w, dw = logits[:T], ids[:T], w[:T], dw[:T]
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda(), mask)
    assert losses.tolist() == [0.0, 0.0] and counts.tolist() == [0] * 13
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, torch.ones(2, device="cuda"), mask, w.cuda(),
                                  dw.cuda())
    assert got.shape == (T, 12) and bool((got == 0).all())


def test_nan_and_inf_logits_show():
    logits, ids, w, dw, _ = case(70, 8, 2, False)
    logits[4, 2] = float("nan")
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda())
    assert torch.isnan(losses).all() and int(counts[8]) == 70
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, torch.ones(2, device="cuda"))
    assert torch.isnan(got[4]).all() and torch.isfinite(torch.cat([got[:4], got[5:]])).all()


def test_repeated_and_foreign_ids():
    """An expert listed twice counts and adds twice; ids outside the experts neither count nor add."""
    logits, ids, w, dw, _ = case(90, 10, 4, False)
    ids[5] = torch.tensor([2, 2, 7, 2], dtype=torch.int32)
    ids[6] = torch.tensor([-1, 10, 3, 2 ** 31 - 1], dtype=torch.int32)
    gl = torch.tensor([0.5, 0.1])
    ref, ref_c, grad, size = R.balance(logits, ids, None, gl, w, dw)
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda())
    check_loss(losses, counts, ref, ref_c)
    got = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, gl.cuda(), None, w.cuda(), dw.cuda())
    check_grad(got, grad, size)


def test_even_routing_gives_one():
    T, E, K = 96, 12, 3
    logits = torch.zeros((T, E), device="cuda")
    ids = ((torch.arange(T)[:, None] * K + torch.arange(K)) % E).to(torch.int32).cuda()
    losses, counts = B.balance_loss(logits, ids)
    assert counts.tolist() == [T * K // E] * E + [T]
    assert abs(float(losses[0]) - 1.0) < 300 * R.U24


def test_counts_of_the_whole_batch():
    """Two halves with summed counts give the whole batch's gradient (per half: N is the batch's)."""
    logits, ids, w, dw, mask = case(500, 40, 4, True)
    gl = torch.tensor([0.3, 0.1])
    _, _, grad, size = R.balance(logits, ids, mask, gl, w, dw)
    parts = [(logits[:200], ids[:200], w[:200], dw[:200], mask[:200]), (logits[200:], ids[200:], w[200:], dw[200:], mask[200:])]
    counts = sum(B.balance_loss(l.cuda(), i.cuda(), m.cuda())[1] for l, i, _, _, m in parts)
    got = torch.cat([B.balance_loss_backward(l.cuda(), i.cuda(), counts, gl.cuda(), m.cuda(), a.cuda(), b.cuda())
                     for l, i, a, b, m in parts])
    check_grad(got, grad, size)


def test_gradient_against_differences():
    """Central differences of the GPU's own losses. Step h = 2^-4 of a logit:
    the third derivatives of both losses in one logit are at most 8 f_max / N
    and 16 (1 + lse) / N, so h^2 / 6 of those; and 64 half steps of the loss over 2h."""
    T, E, K = 6, 5, 2
    logits, ids, _, _, _ = case(T, E, K, False, spread=1.0)
    h = 2.0 ** -4
    losses, counts = B.balance_loss(logits.cuda(), ids.cuda())
    f_max = float((counts[:E].double() * E / (K * T)).max())
    lse = float(torch.logsumexp(logits.double(), 1).abs().max())
    for which, third in ((0, 8 * f_max / T), (1, 16 * (1 + lse) / T)):
        gl = torch.zeros(2)
        gl[which] = 1.0
        grad = B.balance_loss_backward(logits.cuda(), ids.cuda(), counts, gl.cuda()).cpu().double()
        bound = h * h / 6 * third + 64 * R.U24 * float(losses[which]) / h
        for t in range(T):
            for e in range(E):
                d = torch.zeros_like(logits)
                d[t, e] = h
                up = B.balance_loss((logits + d).cuda(), ids.cuda())[0]
                dn = B.balance_loss((logits - d).cuda(), ids.cuda())[0]
                diff = float(up[which].double() - dn[which].double()) / (2 * h)
                assert abs(diff - float(grad[t, e])) <= bound, (which, t, e, diff, float(grad[t, e]), bound)


@pytest.mark.parametrize("T", [40, 5000])
def test_captured_and_deterministic(T):
    logits, ids, w, dw, mask = (cuda(t) for t in case(T, 256, 8, True))
    gl = torch.tensor([0.3, 0.1], device="cuda")
    ws = torch.empty(max(B.balance_workspace_bytes(T, 256), 16), dtype=torch.uint8, device="cuda")

    def run():
        losses, counts = B.balance_loss(logits, ids, mask, ws)
        return losses, counts, B.balance_loss_backward(logits, ids, counts, gl, mask, w, dw)

    first = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(4):
        if seed:
            logits.add_(torch.randn(logits.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        ws.fill_(255)  # (what the workspace held does not matter)
        graph.replay()
        got = [t.clone() for t in out]
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
        if seed == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_loss_from_the_router():
    """moe_route's logits, ids and offsets: the counts are the offsets' steps."""
    dims = dict(hidden=256, latent=128, inter=128, n_experts=24, top_k=3)
    g = torch.Generator().manual_seed(8)
    x = torch.randn((150, 256), generator=g).bfloat16().cuda()
    router = (torch.randn((24, 256), generator=g) * 0.1).cuda()
    d = B.make_dims(dims)
    r = B.route(d, x.view(torch.int16), router, B.alloc_workspace(d, 150))
    losses, counts = B.balance_loss(r["logits"], r["ids"])
    assert torch.equal(counts[:24], r["offsets"][1:] - r["offsets"][:-1]) and int(counts[24]) == 150
    gl, dw = torch.tensor([0.1, 0.01]), torch.randn((150, 3), generator=g)
    ref, ref_c, grad, size = R.balance(r["logits"].cpu(), r["ids"].cpu(), None, gl, r["w"].cpu(), dw)
    check_loss(losses, counts, ref, ref_c)
    got = B.balance_loss_backward(r["logits"], r["ids"], counts, gl.cuda(), None, r["w"], dw.cuda())
    check_grad(got, grad, size)


def test_a_given_stream():
    """A call on a stream of its own, its workspace and results allocated
    there, while the current stream frees and takes memory."""
    logits, ids, w, dw, mask = (cuda(t) for t in case(20000, 256, 8, True))
    gl = torch.tensor([0.3, 0.1], device="cuda")
    want = B.balance_loss(logits, ids, mask)
    want_g = B.balance_loss_backward(logits, ids, want[1], gl, mask, w, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        losses, counts = B.balance_loss(logits, ids, mask, stream=s)
        got.append((losses, counts, B.balance_loss_backward(logits, ids, counts, gl, mask, w, dw, stream=s)))
        torch.full((1 << 18,), 7.0, device="cuda")
    s.synchronize()
    for losses, counts, g in got:
        assert torch.equal(losses, want[0]) and torch.equal(counts, want[1]) and torch.equal(g, want_g)


@pytest.mark.parametrize("given_stream", [False, True])
@pytest.mark.parametrize("T", [40, 700])
def test_losses_carry_their_gradient(T, given_stream):
    """Logits that require a gradient get it from the losses, as one term of a
    larger loss too; where they do not, or no gradient is wanted, nothing is recorded."""
    logits, ids, w, dw, mask = case(T, 20, 4, True)
    gl = torch.tensor([0.7, 0.02])
    grad, size = R.balance(logits, ids, mask, gl)[2:]
    leaf = logits.cuda().requires_grad_()
    plain, plain_c = B.balance_loss(leaf.detach(), ids.cuda(), mask.cuda())
    assert not plain.requires_grad
    with torch.no_grad():
        assert not B.balance_loss(leaf, ids.cuda(), mask.cuda())[0].requires_grad
    s = torch.cuda.Stream() if given_stream else None
    if s:
        s.wait_stream(torch.cuda.current_stream())
    losses, counts = B.balance_loss(leaf, ids.cuda(), mask.cuda(), stream=s)
    if s:
        torch.cuda.current_stream().wait_stream(s)
    assert losses.requires_grad and not counts.requires_grad
    assert torch.equal(losses.detach(), plain) and torch.equal(counts, plain_c)
    other = (leaf.square() * 0.25).sum()
    ((losses * gl.cuda()).sum() + other).backward()
    got = leaf.grad.cpu().double() - 0.5 * logits.double()
    # (the sum of both parts in fp32: half a step of each and of the whole)
    assert bool(((got - grad).abs() <= 64 * R.U24 * size + 2 * R.U24 * logits.double().abs() + 1e-30).all())
    # through a router, one loss alone: its gradient is an expanded one
    x, wr = torch.randn((T, 16), device="cuda"), torch.randn((20, 16), device="cuda", requires_grad=True)
    lg = x @ wr.t()
    B.balance_loss(lg, ids.cuda(), mask.cuda())[0].sum().backward()
    one = torch.ones(2, device="cuda")
    want = B.balance_loss_backward(lg.detach(), ids.cuda(), plain_c, one, mask.cuda()).t() @ x
    assert torch.equal(wr.grad, want) or float((wr.grad - want).norm() / want.norm()) < 1e-6
    B.balance_loss(leaf, ids.cuda(), mask.cuda())[0].sum()
    again, _ = B.balance_loss(leaf, ids.cuda(), mask.cuda())
    with pytest.raises(RuntimeError, match="differentiate twice|once_differentiable"):
        (g,) = torch.autograd.grad(again.sum(), leaf, create_graph=True)
        g.sum().backward()


def test_no_gradient_is_recorded_in_a_capture():
    """A captured call with logits that require a gradient is refused (an
    eager pass over the same leaves may live); detached it runs, its gradient by its own call."""
    logits, ids, _, _, mask = (cuda(t) for t in case(90, 20, 4, True))
    leaf = logits.clone().requires_grad_()
    living, counts = B.balance_loss(leaf, ids, mask)
    one = torch.ones(2, device="cuda")
    want = B.balance_loss_backward(logits, ids, counts, one, mask)
    ws = torch.empty(B.balance_workspace_bytes(90, 20), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="capture"):
            B.balance_loss(leaf, ids, mask, ws)
        losses, c = B.balance_loss(leaf.detach(), ids, mask, ws)
        g = B.balance_loss_backward(leaf, ids, c, one, mask)
    for _ in range(3):
        g.zero_()
        graph.replay()
        assert torch.equal(g, want) and torch.equal(losses, living.detach())
        torch.cuda.synchronize()
    living.sum().backward()
    assert torch.equal(leaf.grad, want)


def test_refusals():
    logits, ids, w, dw, mask = (cuda(t) for t in case(70, 8, 2, True))
    counts = torch.zeros(9, dtype=torch.int32, device="cuda")
    gl = torch.ones(2, device="cuda")
    for bad in (lambda: B.balance_loss(logits.double(), ids), lambda: B.balance_loss(logits, ids.long()),
                lambda: B.balance_loss(logits, ids[:60]), lambda: B.balance_loss(logits.t(), ids),
                lambda: B.balance_loss(logits, ids, mask[:60]), lambda: B.balance_loss(logits, ids, mask.float()),
                lambda: B.balance_loss_backward(logits, ids, counts[:8], gl),
                lambda: B.balance_loss_backward(logits, ids, counts, gl, w=w),
                lambda: B.balance_loss_backward(logits, ids, counts, gl.cpu()),
                lambda: B.balance_loss_backward(logits, ids, counts, gl, w=w, grad_w=dw[:, :1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.MoeError) as e:
        B.balance_loss(logits, ids, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.MOE_EWORKSPACE


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,row", [(1 << 26, [0.3, 1.1, -0.7, 0.05]), ((1 << 22) + 77, [0.3, 1.1, -0.7]),
                                   ((1 << 19) + 1, [0.3, 1.1])])
def test_sums_over_many_tokens(T, row, masked):
    """Equal tokens: their mean is the token's own value, and additions of one
    sign do not drift."""
    row = torch.tensor([row])
    logits, ids = row.cuda().repeat(T, 1), torch.ones((T, 1), dtype=torch.int32, device="cuda")
    mask = (torch.arange(T, device="cuda") % 3 > 0) if masked else None
    n = T if mask is None else int(mask.sum())
    losses, counts = B.balance_loss(logits, ids, mask)
    assert counts.tolist() == ([0, n, 0, 0][:row.shape[1]] + [n])
    p, lse = torch.softmax(row.double(), 1)[0], float(torch.logsumexp(row.double(), 1)[0])
    # exponential and quotient 8 half steps, 32 tokens in fp32, joins of 2 + 16 + 40, f and the sum over the experts 16;
    # lse^2: twice the logarithm's
    rel = (8 + 32 + 2 + 16 + 40 + 16) * R.U24
    assert abs(float(losses[0]) / (row.shape[1] * float(p[1])) - 1) <= rel
    assert abs(float(losses[1]) / lse ** 2 - 1) <= rel + 16 * R.U24


def test_offsets_past_32_bits():
    """Rows of logits and gradients beyond 2^32 bytes: the same values as near
    the start."""
    few, E, K = 1024, 144, 4
    logits, ids, w, dw, _ = case(few, E, K, False)
    times = (1 << 32) // (4 * E * few) + 2
    T = few * times
    big = [t.cuda().repeat(times, 1) for t in (logits, ids, w, dw)]
    losses, counts = B.balance_loss(big[0], big[1])
    one, one_c = B.balance_loss(logits.cuda(), ids.cuda())
    assert torch.equal(counts, one_c * times) and T * E * 4 > 1 << 32
    # the same mean: sums of up to T / (64 * 256) + 16 + 256 positive terms, each addition half a step
    tol = (T / (64 * 256) + 16 + 256) * R.U24
    assert bool(((losses - one).abs() <= 2 * tol * one).all()), (losses, one)
    gl = torch.tensor([0.7, 0.02], device="cuda") * T
    got = B.balance_loss_backward(big[0], big[1], counts, gl, None, big[2], big[3]).view(times, few, E)
    assert bool((got == got[0]).all())
    ref, size = R.balance(logits, ids, None, gl.cpu() / times, w, dw)[2:]
    check_grad(got[-1], ref, size)
