"""What autograd is told of calls that write tensors of the caller, without a
GPU: the library call is replaced, the binding around it runs."""
from __future__ import annotations

import types

import pytest
import torch

from latent_mixture_experts_amd import binding as B

U8, I32, F8 = torch.uint8, torch.int32, torch.float8_e4m3fn


@pytest.fixture
def host(monkeypatch):
    """The binding on host tensors: every library call succeeds and does nothing."""
    monkeypatch.setattr(B, "_device", lambda t: t.device)
    monkeypatch.setattr(B, "_run", lambda *a: None)
    monkeypatch.setattr(B, "_no_capture", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(device=torch.device("cpu"), cuda_stream=0))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    fine = lambda *a: B.MOE_OK
    names = ["route", "latent_forward", "latent_forward_timed", "latent_forward_routed", "latent_forward_persistent",
             "latent_forward_noalloc", "block_forward"]
    monkeypatch.setattr(B, "_lib", types.SimpleNamespace(moe_balance_workspace_bytes=lambda *a: 0,
                                                         **{"moe_" + n: fine for n in names}))


def _routes(T=4, K=2, E=2):
    return dict(offsets=torch.zeros(E + 1, dtype=I32), sorted=torch.zeros(T * K, dtype=I32),
                positions=torch.zeros((T, K), dtype=I32))


def _calls():
    """(name, call of what it writes, the tensors it writes)"""
    x, c8, s8 = torch.zeros((4, 256)), torch.zeros((4, 256), dtype=F8), torch.zeros((4, 2))
    c4, s4 = torch.zeros((4, 128), dtype=U8), torch.zeros((4, 8), dtype=U8)
    w8, ws8 = torch.zeros((2, 16, 256), dtype=F8), torch.zeros((2, 1, 2))
    w4, ws4 = torch.zeros((2, 16, 128), dtype=U8), torch.zeros((2, 16, 8), dtype=U8)
    off, routes, wt = torch.zeros(3, dtype=I32), _routes(), torch.zeros((4, 2))
    rows = torch.zeros((8, 256))
    lg, ids, counts = torch.zeros((70, 8)), torch.zeros((70, 2), dtype=I32), torch.zeros(9, dtype=I32)
    new = torch.zeros
    yield "fp8_quantize", lambda c, s: B.fp8_quantize(x, c, s), (new((4, 256), dtype=F8), new((4, 2)))
    yield "fp8_swiglu", lambda c, s: B.fp8_swiglu(x, c, s), (new((4, 128), dtype=F8), new((4, 1)))
    yield "fp8_linear", lambda o: B.fp8_linear(c8, s8, w8[0], ws8[0], out=o), (new((4, 16)),)
    yield "fp8_grouped", lambda o: B.fp8_grouped(c8, s8, off, w8, ws8, out=o), (new((4, 16)),)
    yield "fp4_quantize", lambda c, s: B.fp4_quantize(x, c, s), (new((4, 128), dtype=U8), new((4, 8), dtype=U8))
    yield "fp4_swiglu", lambda c, s: B.fp4_swiglu(x, c, s), (new((4, 64), dtype=U8), new((4, 4), dtype=U8))
    yield "fp4_dequantize", lambda o: B.fp4_dequantize(c4, s4, out=o), (new((4, 256)),)
    yield "fp4_linear", lambda o: B.fp4_linear(c4, s4, w4[0], ws4[0], out=o), (new((4, 16)),)
    yield "fp4_grouped", lambda o: B.fp4_grouped(c4, s4, off, w4, ws4, out=o), (new((4, 16)),)
    yield "gather_rows", lambda o: B.gather_rows(x, routes, out=o), (new((8, 256)),)
    yield "gather_rows_backward", lambda o: B.gather_rows_backward(rows, routes, out=o), (new((4, 256)),)
    yield "combine_rows", lambda o: B.combine_rows(rows, routes, wt, out=o), (new((4, 256)),)
    yield "combine_rows_backward", lambda o: B.combine_rows_backward(x, rows, routes, wt, grad_rows=o), (new((8, 256)),)
    yield "balance_loss_backward", lambda o: B.balance_loss_backward(lg, ids, counts, new(2), out=o), (new((70, 8)),)
    d = B.make_dims(dict(hidden=256, latent=128, inter=64, n_experts=8, top_k=2))
    st, w = types.SimpleNamespace(cuda_stream=0), B.MoeWeights()
    yield "route", lambda ws: B.route(d, x, x, ws, stream=st), (new(512, dtype=U8),)
    for name, args in (("latent_forward", (x, w)), ("latent_forward_routed", (x, ids, wt, w)),
                       ("latent_forward_persistent", (x, w)), ("block_forward", (x, wt, wt, 1e-6, w))):
        yield (name, lambda o, ws, name=name, args=args: getattr(B, name)(d, *args, o, ws, stream=st),
               (new((4, 256)), new(512, dtype=U8)))
    yield "latent_forward timed", lambda o, ws: B.latent_forward(d, x, w, o, ws, stream=st, events=[None] * 16), (
        new((4, 256)), new(512, dtype=U8))
    yield "latent_forward_noalloc", lambda o: B.latent_forward_noalloc(d, x, w, o, stream=st), (new((4, 256)),)


NAMES = [c[0] for c in _calls()]


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_writes_counts_as_written(host, name):
    """Outputs (and the layer's workspace, whose views show its intermediates) of the caller count a write, as after
    torch's own calls, so that autograd refuses what it saved of them before."""
    call, written = next((c, w) for n, c, w in _calls() if n == name)
    before = [t._version for t in written]
    call(*written)
    assert all(t._version > b for t, b in zip(written, before))
    with torch.inference_mode():  # (tensors of inference mode count nothing)
        fixed = [torch.zeros_like(t) for t in written]
    call(*fixed)


def test_rows_overwritten_before_the_backward_pass_are_refused(host):
    """Frozen experts with a trained router: the second micro-batch's rows in the first one's buffer."""
    c, s = torch.zeros((8, 128), dtype=U8), torch.zeros((8, 8), dtype=U8)
    w, ws, off = torch.zeros((2, 16, 128), dtype=U8), torch.zeros((2, 16, 8), dtype=U8), torch.zeros(3, dtype=I32)
    buf, weights = torch.zeros((8, 16)), torch.zeros((4, 2), requires_grad=True)
    B.fp4_grouped(c, s, off, w, ws, out=buf)
    y = B.combine_rows(buf, _routes(), weights)
    y.sum().backward(retain_graph=True)  # (as it should be)
    B.fp4_grouped(c, s, off, w, ws, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", [n for n in NAMES if n != "route"])
def test_outputs_that_require_a_gradient_are_refused(host, name):
    """A call that writes a tensor has no gradient for it: refused before anything is enqueued, as torch refuses
    out= (with gradients off it is written)."""
    call, written = next((c, w) for n, c, w in _calls() if n == name)
    marked = [t for t in written if t.dtype == torch.float32]
    for t in marked:
        t.requires_grad_()
        before = t._version
        with pytest.raises(ValueError, match="requires a gradient"):
            call(*written)
        assert t._version == before and t.requires_grad
        with torch.no_grad():
            call(*written)
        call(*(w.detach() for w in written))
        t.requires_grad_(False)
    assert marked or name.startswith("fp4_quantize") or name == "fp4_swiglu"


def _carrying():
    """(name, call of a tensor that carries a tangent, its shape) for every differentiable argument of the calls that
    are recorded for autograd"""
    routes, x, rows, wt = _routes(), torch.zeros((4, 256)), torch.zeros((8, 256)), torch.zeros((4, 2))
    ids = torch.zeros((70, 2), dtype=I32)
    yield "gather_rows x", lambda t: B.gather_rows(t, routes), (4, 256)
    yield "combine_rows rows", lambda t: B.combine_rows(t, routes, wt), (8, 256)
    yield "combine_rows w", lambda t: B.combine_rows(rows, routes, t), (4, 2)
    yield "balance_loss logits", lambda t: B.balance_loss(t, ids), (70, 8)
    yield "gather_rows out", lambda t: B.gather_rows(x, routes, out=t), (8, 256)
    yield "combine_rows out", lambda t: B.combine_rows(rows, routes, wt, out=t), (4, 256)


@pytest.mark.parametrize("name", [c[0] for c in _carrying()])
def test_tangents_are_refused(host, name):
    """No call has a derivative in forward mode; none drops a tangent, or leaves one beside other values, in silence."""
    call, shape = next((c, s) for n, c, s in _carrying() if n == name)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(torch.zeros(shape), torch.ones(shape))
        for grad in (True, False):  # (forward mode goes on where gradients are off)
            with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="tangent"):
                call(dual)
        call(torch.zeros(shape))  # (inside a level, without a tangent)
    call(torch.zeros(shape))


def test_a_result_that_cannot_carry_a_gradient_is_refused(host):
    """Rows of bf16 bits held as int16: torch takes such a result for a constant, and the weights would get no gradient."""
    routes, w = _routes(), torch.zeros((4, 2), requires_grad=True)
    bits = torch.zeros((8, 256), dtype=torch.int16)
    for rows, dtype in ((bits, None), (bits, torch.int16), (torch.zeros((8, 256)), torch.int16)):
        with pytest.raises(ValueError, match="gradient"):
            B.combine_rows(rows, routes, w, dtype)
        with torch.no_grad():
            assert B.combine_rows(rows, routes, w, dtype).dtype == torch.int16
    for dtype in (torch.float32, torch.bfloat16):
        y = B.combine_rows(bits, routes, w, dtype)
        assert y.requires_grad
        y.sum().backward()
        assert w.grad.shape == w.shape
    assert not B.combine_rows(bits, routes, w.detach()).requires_grad
