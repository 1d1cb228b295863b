"""ctypes binding of libmoe.so (include/moe.h), for torch tensors.

Argument marshalling only: device pointers, sizes and the current HIP
stream go to the C ABI, which runs every step on the GPU. There is no other
implementation behind these functions; a missing library raises.
"""
from __future__ import annotations

import ctypes
import os

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EALIGN, MOE_EWORKSPACE, MOE_EHIP = 0, -1, -2, -3, -4, -5
N_STAGES = 8
STAGES = ("router", "topk", "permute", "pool", "gateup", "down", "combine", "unpool")
VIEWS = dict(logits=0, ids=1, weights=2, offsets=3, sorted=4, latent=5, h=6, rows=7, y=8,
             norm_f32=9, norm_bf16=10, layer_out=11, sync=12, rows_bf16=13)

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t


FMT_MXFP4, FMT_NVFP4 = 0, 1  # expert weight formats (MOE_FMT_*)


class MoeDims(ctypes.Structure):
    _fields_ = [("hidden", _i32), ("latent", _i32), ("inter", _i32), ("n_experts", _i32),
                ("top_k", _i32), ("norm_eps", ctypes.c_float), ("gain_per_expert", _i32),
                ("expert_format", _i32), ("expert_split_rows", _i32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("router", _vp), ("pooler", _vp), ("w13_codes", _vp), ("w13_scales", _vp),
                ("w2_codes", _vp), ("w2_scales", _vp), ("norm_gain", _vp), ("unpooler", _vp),
                ("w13_global", _vp), ("w2_global", _vp)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().moe_status_string(status).decode()
        if status == MOE_EHIP:
            msg += f" (hip error {lib().moe_last_hip_error()})"
        super().__init__(f"{what}: {msg} [{status}]")


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m latent_mixture_experts_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_workspace_bytes.restype = _sz
        L.moe_workspace_bytes.argtypes = [ctypes.POINTER(MoeDims), _i32]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _sz, _vp]
        L.moe_route_validate.restype = ctypes.c_int
        L.moe_route_validate.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _vp, _sz]
        L.moe_latent_forward.restype = ctypes.c_int
        L.moe_latent_forward.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp,
                                         ctypes.POINTER(MoeWeights), _vp, _vp, _sz, _vp]
        L.moe_latent_forward_timed.restype = ctypes.c_int
        L.moe_latent_forward_timed.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp,
                                               ctypes.POINTER(MoeWeights), _vp, _vp, _sz, _vp,
                                               ctypes.POINTER(_vp)]
        L.moe_latent_forward_persistent.restype = ctypes.c_int
        L.moe_latent_forward_persistent.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp,
                                                    ctypes.POINTER(MoeWeights), _vp, _vp, _sz, _vp]
        L.moe_latent_forward_noalloc.restype = ctypes.c_int
        L.moe_latent_forward_noalloc.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp,
                                                 ctypes.POINTER(MoeWeights), _vp, _vp]
        L.moe_latent_forward_routed.restype = ctypes.c_int
        L.moe_latent_forward_routed.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp, _vp,
                                                ctypes.POINTER(MoeWeights), _vp, _vp, _sz, _vp]
        L.moe_latent_forward_routed_validate.restype = ctypes.c_int
        L.moe_latent_forward_routed_validate.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp,
                                                         _vp, ctypes.POINTER(MoeWeights), _vp,
                                                         _vp, _sz]
        L.moe_block_workspace_bytes.restype = _sz
        L.moe_block_workspace_bytes.argtypes = [ctypes.POINTER(MoeDims), _i32]
        L.moe_block_forward.restype = ctypes.c_int
        L.moe_block_forward.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp, _vp,
                                        ctypes.c_float, ctypes.POINTER(MoeWeights), _vp, _vp, _sz,
                                        _vp]
        L.moe_block_forward_validate.restype = ctypes.c_int
        L.moe_block_forward_validate.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp, _vp, _vp,
                                                 ctypes.c_float, ctypes.POINTER(MoeWeights), _vp,
                                                 _vp, _sz]
        L.moe_latent_forward_validate.restype = ctypes.c_int
        L.moe_latent_forward_validate.argtypes = [ctypes.POINTER(MoeDims), _i32, _vp,
                                                  ctypes.POINTER(MoeWeights), _vp, _vp, _sz]
        L.moe_workspace_view.restype = ctypes.c_int
        L.moe_workspace_view.argtypes = [ctypes.POINTER(MoeDims), _i32, _i32,
                                         ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
        i64 = ctypes.c_int64
        for name, args in {
            "moe_fp8_quantize": [_i32, _i32, _vp, i64, _i32, _vp, _vp],
            "moe_fp8_swiglu": [_i32, _i32, _vp, i64, _i32, _vp, _vp],
            "moe_fp8_linear": [_i32, _i32, _i32, _vp, i64, _vp, _vp, _vp, _vp, i64, _i32],
            "moe_fp8_grouped": [_i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _vp, i64, _vp, _vp,
                                _vp, _vp, i64, _i32],
            "moe_fp4_quantize": [_i32, _i32, _vp, i64, _i32, _vp, _vp],
            "moe_fp4_swiglu": [_i32, _i32, _vp, i64, _i32, _vp, _vp],
            "moe_fp4_dequantize": [_i32, _i32, _vp, _vp, _vp, i64, _i32],
            "moe_fp4_linear": [_i32, _i32, _i32, _vp, i64, _vp, _vp, _vp, _vp, i64, _i32],
            "moe_fp4_grouped": [_i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _vp, i64, _vp, _vp,
                                _vp, _vp, i64, _i32],
            "moe_sort_routes": [_i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _sz],
            "moe_gather_rows": [_i32, _i32, _i32, _i32, _vp, i64, _i32, _vp, _vp, _vp, i64],
            "moe_combine_rows": [_i32, _i32, _i32, _i32, _vp, i64, _i32, _vp, _vp, _vp, i64, _i32],
            "moe_combine_rows_backward": [_i32, _i32, _i32, _i32, _vp, i64, _i32, _vp, i64, _i32, _vp, _vp,
                                          _vp, _vp, i64, _vp],
            "moe_balance_loss": [_i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz],
            "moe_balance_loss_backward": [_i32, _i32, _i32] + [_vp] * 8,
        }.items():
            for fn, more in ((getattr(L, name), [_vp]), (getattr(L, name + "_validate"), [])):
                fn.restype, fn.argtypes = ctypes.c_int, args + more
        L.moe_balance_workspace_bytes.restype = _sz
        L.moe_balance_workspace_bytes.argtypes = [_i32, _i32]
        L.moe_sort_workspace_bytes.restype = _sz
        L.moe_sort_workspace_bytes.argtypes = [_i32, _i32, _i32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_last_hip_error.restype = ctypes.c_int
        L.moe_last_hip_error.argtypes = []
        _lib = L
    return _lib


def make_dims(dims: dict, eps: float = 1e-6, gain_per_expert: int = 0,
              expert_format: int = FMT_MXFP4, expert_split_rows: int = 0) -> MoeDims:
    return MoeDims(dims["hidden"], dims["latent"], dims["inter"], dims["n_experts"],
                   dims["top_k"], eps, int(gain_per_expert), int(expert_format),
                   int(expert_split_rows))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _no_tangent(**tensors) -> None:
    """The calls have no derivative in forward mode. (Its level first, -1 outside: asking a tensor costs 0.6 us.)"""
    if forward_ad._current_level >= 0:
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{name}: carries a tangent (no derivative in forward mode)")


def _writable(name: str, t) -> None:
    """The calls have no gradient for what they write."""
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: is written and requires a gradient (pass {name}.detach())")
    if forward_ad._current_level >= 0:
        _no_tangent(**{name: t})


_increment_version = torch.autograd.graph.increment_version


def _written(*given) -> None:
    """Counts a write of the caller's tensors (None: not given), as torch's own calls
    do: a backward pass that saved them before this call refuses to run on what they hold now."""
    for t in given:
        if isinstance(t, torch.Tensor):
            _increment_version(t)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def workspace_bytes(d: MoeDims, max_tokens: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(d), max_tokens))


def alloc_workspace(d: MoeDims, max_tokens: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(d, max_tokens)
    if n == 0 and max_tokens > 0:
        raise MoeError(MOE_EUNSUPPORTED, "moe_workspace_bytes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def block_workspace_bytes(d: MoeDims, max_tokens: int) -> int:
    return int(lib().moe_block_workspace_bytes(ctypes.byref(d), max_tokens))


def alloc_block_workspace(d: MoeDims, max_tokens: int, device="cuda") -> torch.Tensor:
    n = block_workspace_bytes(d, max_tokens)
    if n == 0 and max_tokens > 0:
        raise MoeError(MOE_EUNSUPPORTED, "moe_block_workspace_bytes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def make_weights(w: dict) -> MoeWeights:
    """Pointers of the weight tensors (w13_global / w2_global: NVFP4 only)."""
    return MoeWeights(*(_ptr(w.get(k)) for k in ("router", "pooler", "w13_codes", "w13_scales",
                                                  "w2_codes", "w2_scales", "norm_gain", "unpooler",
                                                  "w13_global", "w2_global")))


def route(d: MoeDims, x: torch.Tensor, router: torch.Tensor, ws: torch.Tensor,
          want_logits: bool = True, stream=None) -> dict:
    """moe_route on T = x.shape[0] tokens; returns the output tensors."""
    T = x.shape[0]
    E, K = d.n_experts, d.top_k
    dev = x.device
    out = dict(ids=torch.empty((T, K), dtype=torch.int32, device=dev),
               w=torch.empty((T, K), dtype=torch.float32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               sorted=torch.empty(T * K, dtype=torch.int32, device=dev))
    out["logits"] = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    rc = lib().moe_route(ctypes.byref(d), T, _ptr(x), _ptr(router), _ptr(out["ids"]),
                         _ptr(out["w"]), _ptr(out["offsets"]), _ptr(out["sorted"]),
                         _ptr(out["logits"]), _ptr(ws), ws.numel(), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_route")
    _written(ws)
    return out


def latent_forward(d: MoeDims, x: torch.Tensor, weights: MoeWeights, out: torch.Tensor,
                   ws: torch.Tensor, stream=None, events=None) -> torch.Tensor:
    """moe_latent_forward, or moe_latent_forward_timed when ``events`` holds
    2 * MOE_N_STAGES hipEvent_t handles (start, stop of each step; None
    entries are skipped)."""
    _writable("out", out)
    T = x.shape[0]
    if events is None:
        rc = lib().moe_latent_forward(ctypes.byref(d), T, _ptr(x), ctypes.byref(weights),
                                      _ptr(out), _ptr(ws), ws.numel(), _stream(stream))
    else:
        arr = (_vp * len(events))(*[e if e else None for e in events])
        rc = lib().moe_latent_forward_timed(ctypes.byref(d), T, _ptr(x), ctypes.byref(weights),
                                            _ptr(out), _ptr(ws), ws.numel(), _stream(stream), arr)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_latent_forward")
    _written(out, ws)
    return out


def latent_forward_routed(d: MoeDims, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor,
                          weights: MoeWeights, out: torch.Tensor, ws: torch.Tensor,
                          stream=None) -> torch.Tensor:
    """moe_latent_forward_routed: the layer with the routing given (ids
    [T][K] int32, w [T][K] fp32, on the device)."""
    _writable("out", out)
    T = x.shape[0]
    rc = lib().moe_latent_forward_routed(ctypes.byref(d), T, _ptr(x), _ptr(ids), _ptr(w),
                                         ctypes.byref(weights), _ptr(out), _ptr(ws), ws.numel(),
                                         _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_latent_forward_routed")
    _written(out, ws)
    return out


def latent_forward_persistent(d: MoeDims, x: torch.Tensor, weights: MoeWeights, out: torch.Tensor,
                              ws: torch.Tensor, stream=None) -> torch.Tensor:
    """moe_latent_forward_persistent: the layer for one or two tokens in one launch."""
    _writable("out", out)
    T = x.shape[0]
    rc = lib().moe_latent_forward_persistent(ctypes.byref(d), T, _ptr(x), ctypes.byref(weights),
                                             _ptr(out), _ptr(ws), ws.numel(), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_latent_forward_persistent")
    _written(out, ws)
    return out


def latent_forward_noalloc(d: MoeDims, x: torch.Tensor, weights: MoeWeights, out: torch.Tensor,
                           stream=None) -> torch.Tensor:
    """moe_latent_forward_noalloc: the layer with the library's own per-GPU
    scratch array as its workspace (no workspace argument)."""
    _writable("out", out)
    T = x.shape[0]
    rc = lib().moe_latent_forward_noalloc(ctypes.byref(d), T, _ptr(x), ctypes.byref(weights),
                                          _ptr(out), _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_latent_forward_noalloc")
    _written(out)
    return out


def block_forward(d: MoeDims, resid: torch.Tensor, pre_gain: torch.Tensor, post_gain: torch.Tensor,
                  block_eps: float, weights: MoeWeights, out: torch.Tensor, ws: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """moe_block_forward: out = resid + post_norm(layer(pre_norm(resid)))."""
    _writable("out", out)
    T = resid.shape[0]
    rc = lib().moe_block_forward(ctypes.byref(d), T, _ptr(resid), _ptr(pre_gain), _ptr(post_gain),
                                 block_eps, ctypes.byref(weights), _ptr(out), _ptr(ws), ws.numel(),
                                 _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_block_forward")
    _written(out, ws)
    return out


def workspace_view_range(d: MoeDims, T: int, which: str) -> tuple[int, int]:
    """(byte offset, bytes) of an intermediate in the workspace."""
    off, nb = _sz(), _sz()
    rc = lib().moe_workspace_view(ctypes.byref(d), T, VIEWS[which], ctypes.byref(off), ctypes.byref(nb))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_workspace_view")
    return off.value, nb.value


def workspace_view(d: MoeDims, T: int, ws: torch.Tensor, which: str, dtype, shape):
    """An intermediate of the last moe_latent_forward, viewed in the workspace."""
    off, nb = workspace_view_range(d, T, which)
    return ws[off:off + nb].view(dtype).view(shape)


# ---- 8-bit and 4-bit rows, their products, expert order, the balance loss ---
# These take their sizes from the tensors, so they check them: a wrong shape,
# type, layout or device raises ValueError before anything is enqueued. They
# run on the tensors' device, on its current stream unless one is given (a
# torch.cuda.Stream). What they allocate then belongs to that stream, and what
# they were given may be dropped once they return; order between the streams
# (inputs written before, results read after, there or elsewhere) is the caller's.
# Outputs that are given (out, codes, scales, grad_rows) count as written; one that
# requires a gradient is refused.
# Only balance_loss, gather_rows and combine_rows are recorded for autograd, for
# its reverse mode (they refuse a tangent of forward mode); the 8-bit and 4-bit
# calls have no gradient, and what they return requires none.
TYPE_BF16, TYPE_F32 = 0, 1  # MOE_TYPE_*
SUM_F32 = 0x100  # MOE_SUM_F32
_FLOATS = {torch.bfloat16: TYPE_BF16, torch.int16: TYPE_BF16, torch.float32: TYPE_F32}  # int16: bf16 bits
_CODES = (torch.float8_e4m3fn, torch.uint8)
_ANY_FLOAT = tuple(_FLOATS)
_F32, _I32, _MASK = (torch.float32,), (torch.int32,), (torch.uint8, torch.bool)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _int32(*sizes: int) -> None:
    """ctypes would cut a larger one off without a word. (Sizes that are never
    negative may come joined by |, which costs a call less.)"""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"sizes are 32-bit, got {n}")


def _check(name: str, t: torch.Tensor, dev: torch.device, types, shape, pitched: bool = False) -> None:
    """t is on dev, of one of the types, of that shape, and dense (pitched: its rows are, at any pitch)."""
    if (t.shape != shape or t.dtype not in types or t.device != dev or
            not (t.is_contiguous() or (pitched and (t.shape[1] == 1 or t.stride(1) == 1)
                                       and t.stride(0) >= t.shape[1]))):
        raise ValueError(f"{name}: needs {'rows' if pitched else 'a dense tensor'} {list(shape)} of "
                         f"{' or '.join(str(x) for x in types)} on {dev}, got {list(t.shape)} {t.dtype} "
                         f"on {t.device}, strides {t.stride()}")


def _pitch(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _same_device(dev: torch.device, stream) -> None:
    if stream.device != dev:
        raise ValueError(f"the tensors are on {dev}, the stream on {stream.device}")


def _run(what: str, dev: torch.device, stream, *args) -> None:
    fn = getattr(_lib or lib(), what)
    if stream is not None:
        _same_device(dev, stream)
    # (the current stream's handle alone: building a torch.cuda.Stream costs as much as the launch)
    st = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if dev.index == torch._C._cuda_getDevice():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _empty(shape, dtype, dev: torch.device, stream) -> torch.Tensor:
    """A tensor of the stream that the call runs on: memory of another stream's
    pool could still be in use there, or be handed out again before the call is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """_empty on the device of like (new_empty: a sixth less of a call's host time than the device by name)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    return _empty(shape, dtype, like.device, stream)


def _hold(stream, *tensors) -> None:
    """Memory of the call's tensors is not handed out again before the given
    stream has done the call, also when the caller drops them right after it."""
    if stream is not None:
        _same_device(tensors[0].device, stream)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _device(t: torch.Tensor) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, got {dev}")
    return dev


def _quantize(what: str, x: torch.Tensor, cols: int, codes, scales, stream):
    dev = _device(x)
    rows = x.shape[0]
    _int32(rows | cols)
    _check("x", x, dev, _ANY_FLOAT, (rows, x.shape[1]), pitched=True)
    given = codes, scales
    if codes is None:
        codes = _empty((rows, cols), torch.float8_e4m3fn, dev, stream)
    else:
        _writable("codes", codes)
        _check("codes", codes, dev, _CODES, (rows, cols))
    if scales is None:
        scales = _empty((rows, _blocks(cols)), torch.float32, dev, stream)
    else:
        _writable("scales", scales)
        _check("scales", scales, dev, _F32, (rows, _blocks(cols)))
    _hold(stream, x, codes, scales)
    _run(what, dev, stream, rows, cols, x.data_ptr(), _pitch(x), _FLOATS[x.dtype], codes.data_ptr(),
         scales.data_ptr())
    if given[0] is not None or given[1] is not None:
        _written(*given)
    return codes, scales


def fp8_quantize(x: torch.Tensor, codes=None, scales=None, stream=None):
    """moe_fp8_quantize of x [rows][cols] (bf16 or fp32, every row at a multiple
    of 16 bytes): (codes [rows][cols] e4m3, scales [rows][ceil(cols/128)] fp32)."""
    _need(x.dim() == 2, "x: needs two dimensions")
    return _quantize("moe_fp8_quantize", x, x.shape[1], codes, scales, stream)


def fp8_swiglu(gate_up: torch.Tensor, codes=None, scales=None, stream=None):
    """moe_fp8_swiglu of gate_up [rows][2 * inter] (gate values, then up
    values): silu(gate) * up as fp8_quantize gives it."""
    _need(gate_up.dim() == 2 and gate_up.shape[1] % 2 == 0, "gate_up: needs two dimensions, the second even")
    return _quantize("moe_fp8_swiglu", gate_up, gate_up.shape[1] // 2, codes, scales, stream)


def _out(out, rows: int, n: int, dtype, dev: torch.device, stream) -> torch.Tensor:
    if out is None:
        if dtype not in _FLOATS:
            raise ValueError(f"out_dtype: bfloat16 or float32, got {dtype}")
        return _empty((rows, n), dtype, dev, stream)
    _writable("out", out)
    _check("out", out, dev, _ANY_FLOAT, (rows, n), pitched=True)
    return out


def fp8_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               out_dtype=torch.bfloat16, out=None, stream=None, f32_sums: bool = False) -> torch.Tensor:
    """moe_fp8_linear: x [T][K] e4m3 with x_scales [T][ceil(K/128)], times w
    [N][K] e4m3 with w_scales [ceil(N/128)][ceil(K/128)] -> [T][N] of
    out_dtype, or into out. Rows of x at multiples of 16 bytes, rows of out at
    any pitch. f32_sums: a bf16 out, too, sums in fp32 throughout (MOE_SUM_F32)."""
    _need(x.dim() == 2 and w.dim() == 2, "x, w: need two dimensions")
    dev = _device(x)
    (T, K), N = x.shape, w.shape[0]
    _int32(T | K | N)
    _check("x", x, dev, _CODES, (T, K), pitched=True)
    _check("x_scales", x_scales, dev, _F32, (T, _blocks(K)))
    _check("w", w, dev, _CODES, (N, K))
    _check("w_scales", w_scales, dev, _F32, (_blocks(N), _blocks(K)))
    given = out
    out = _out(out, T, N, out_dtype, dev, stream)
    _hold(stream, x, x_scales, w, w_scales, out)
    _run("moe_fp8_linear", dev, stream, T, N, K, x.data_ptr(), _pitch(x), x_scales.data_ptr(),
         w.data_ptr(), w_scales.data_ptr(), out.data_ptr(), _pitch(out),
         _FLOATS[out.dtype] | SUM_F32 if f32_sums else _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


def fp8_grouped(x: torch.Tensor, x_scales: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                w_scales: torch.Tensor, out_dtype=torch.bfloat16, row_index=None, index_div: int = 1,
                out=None, stream=None, f32_sums: bool = False) -> torch.Tensor:
    """moe_fp8_grouped: rows offsets[e] .. offsets[e+1]-1 times expert e's
    weights, w [E][N][K] with w_scales [E][ceil(N/128)][ceil(K/128)], offsets
    [E+1] int32. The rows are those of x, or with row_index [rows] int32 row
    row_index[i] // index_div of x for output row i. Rows of out that no expert
    takes are left as they are (as allocated, without out). f32_sums as for
    fp8_linear."""
    _need(x.dim() == 2 and w.dim() == 3, "x: needs two dimensions, w three")
    dev = _device(x)
    (x_rows, K), (E, N, _) = x.shape, w.shape
    rows = x_rows if row_index is None else row_index.numel()
    _int32(rows | x_rows | K | E | N, index_div)
    _check("x", x, dev, _CODES, (x_rows, K), pitched=True)
    _check("x_scales", x_scales, dev, _F32, (x_rows, _blocks(K)))
    _check("offsets", offsets, dev, _I32, (E + 1,))
    _check("w", w, dev, _CODES, (E, N, K))
    _check("w_scales", w_scales, dev, _F32, (E, _blocks(N), _blocks(K)))
    if row_index is not None:
        _check("row_index", row_index, dev, _I32, (rows,))
    given = out
    out = _out(out, rows, N, out_dtype, dev, stream)
    _hold(stream, x, x_scales, offsets, w, w_scales, row_index, out)
    _run("moe_fp8_grouped", dev, stream, rows, E, N, K, offsets.data_ptr(), _ptr(row_index), index_div,
         x_rows, x.data_ptr(), _pitch(x), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
         out.data_ptr(), _pitch(out), _FLOATS[out.dtype] | SUM_F32 if f32_sums else _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


_NIBBLES, _E8M0 = (torch.uint8,), (torch.uint8, torch.float8_e8m0fnu)


def _result(like: torch.Tensor, out, rows: int, n: int, dtype, dev: torch.device, stream) -> torch.Tensor:
    """_out, by _new."""
    if out is None and stream is None and dtype in _FLOATS:
        return like.new_empty((rows, n), dtype=dtype)
    return _out(out, rows, n, dtype, dev, stream)


def _fp4_quantize(what: str, x: torch.Tensor, cols: int, codes, scales, stream):
    dev = _device(x)
    rows = x.shape[0]
    _int32(rows | cols)
    _check("x", x, dev, _ANY_FLOAT, (rows, x.shape[1]), pitched=True)
    if cols % 32:
        raise ValueError(f"x: needs a width in groups of 32, got {cols}")
    given = codes, scales
    if codes is None:
        codes = _new(x, (rows, cols // 2), torch.uint8, stream)
    else:
        _writable("codes", codes)
        _check("codes", codes, dev, _NIBBLES, (rows, cols // 2))
    if scales is None:
        scales = _new(x, (rows, cols // 32), torch.uint8, stream)
    else:
        _writable("scales", scales)
        _check("scales", scales, dev, _E8M0, (rows, cols // 32))
    _hold(stream, x, codes, scales)
    _run(what, dev, stream, rows, cols, x.data_ptr(), _pitch(x), _FLOATS[x.dtype], codes.data_ptr(),
         scales.data_ptr())
    if given[0] is not None or given[1] is not None:
        _written(*given)
    return codes, scales


def fp4_quantize(x: torch.Tensor, codes=None, scales=None, stream=None):
    """moe_fp4_quantize of x [rows][cols] (bf16 or fp32, every row at a multiple
    of 16 bytes): (codes [rows][cols/2] uint8, two E2M1 values a byte; scales
    [rows][cols/32] uint8, E8M0): the layer's MXFP4, also for its weights."""
    _need(x.dim() == 2, "x: needs two dimensions")
    return _fp4_quantize("moe_fp4_quantize", x, x.shape[1], codes, scales, stream)


def fp4_swiglu(gate_up: torch.Tensor, codes=None, scales=None, stream=None):
    """moe_fp4_swiglu of gate_up [rows][2 * inter] (gate values, then up
    values): silu(gate) * up as fp4_quantize gives it."""
    _need(gate_up.dim() == 2 and gate_up.shape[1] % 2 == 0, "gate_up: needs two dimensions, the second even")
    return _fp4_quantize("moe_fp4_swiglu", gate_up, gate_up.shape[1] // 2, codes, scales, stream)


def fp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.bfloat16, out=None,
                   stream=None) -> torch.Tensor:
    """moe_fp4_dequantize: the values [rows][cols] of codes [rows][cols/2] and
    scales [rows][cols/32], of out_dtype or into out (rows at any pitch)."""
    _need(codes.dim() == 2, "codes: needs two dimensions")
    dev = _device(codes)
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    _int32(rows | cols)
    _check("codes", codes, dev, _NIBBLES, (rows, cols // 2))
    _check("scales", scales, dev, _E8M0, (rows, cols // 32))
    given = out
    out = _result(codes, out, rows, cols, out_dtype, dev, stream)
    _hold(stream, codes, scales, out)
    _run("moe_fp4_dequantize", dev, stream, rows, cols, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
         _pitch(out), _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


def fp4_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """moe_fp4_linear: x [T][K/2] with x_scales [T][K/32] times w [N][K/2] with
    w_scales [N][K/32], as fp4_quantize gives them -> [T][N] of out_dtype, or
    into out. Rows of x at multiples of 16 bytes, rows of out at any pitch."""
    _need(x.dim() == 2 and w.dim() == 2, "x, w: need two dimensions")
    dev = _device(x)
    (T, half), N = x.shape, w.shape[0]
    K = 2 * half
    _int32(T | K | N)
    _check("x", x, dev, _NIBBLES, (T, half), pitched=True)
    _check("x_scales", x_scales, dev, _E8M0, (T, K // 32))
    _check("w", w, dev, _NIBBLES, (N, half))
    _check("w_scales", w_scales, dev, _E8M0, (N, K // 32))
    given = out
    out = _result(x, out, T, N, out_dtype, dev, stream)
    _hold(stream, x, x_scales, w, w_scales, out)
    _run("moe_fp4_linear", dev, stream, T, N, K, x.data_ptr(), _pitch(x), x_scales.data_ptr(), w.data_ptr(),
         w_scales.data_ptr(), out.data_ptr(), _pitch(out), _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


def fp4_grouped(x: torch.Tensor, x_scales: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                w_scales: torch.Tensor, out_dtype=torch.bfloat16, row_index=None, index_div: int = 1,
                out=None, stream=None) -> torch.Tensor:
    """moe_fp4_grouped: rows offsets[e] .. offsets[e+1]-1 times expert e's
    weights, w [E][N][K/2] with w_scales [E][N][K/32] (the layer's w13 and w2 as
    they are), offsets [E+1] int32. The rows are those of x, or with row_index
    [rows] int32 row row_index[i] // index_div of x for output row i. Rows of
    out that no expert takes are left as they are (as allocated, without out)."""
    _need(x.dim() == 2 and w.dim() == 3, "x: needs two dimensions, w three")
    dev = _device(x)
    (x_rows, half), (E, N, _) = x.shape, w.shape
    K = 2 * half
    rows = x_rows if row_index is None else row_index.numel()
    _int32(rows | x_rows | K | E | N, index_div)
    _check("x", x, dev, _NIBBLES, (x_rows, half), pitched=True)
    _check("x_scales", x_scales, dev, _E8M0, (x_rows, K // 32))
    _check("offsets", offsets, dev, _I32, (E + 1,))
    _check("w", w, dev, _NIBBLES, (E, N, half))
    _check("w_scales", w_scales, dev, _E8M0, (E, N, K // 32))
    if row_index is not None:
        _check("row_index", row_index, dev, _I32, (rows,))
    given = out
    out = _result(x, out, rows, N, out_dtype, dev, stream)
    _hold(stream, x, x_scales, offsets, w, w_scales, row_index, out)
    _run("moe_fp4_grouped", dev, stream, rows, E, N, K, offsets.data_ptr(), _ptr(row_index), index_div,
         x_rows, x.data_ptr(), _pitch(x), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
         out.data_ptr(), _pitch(out), _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


def sort_workspace_bytes(T: int, n_experts: int, top_k: int) -> int:
    _int32(T, n_experts, top_k)
    return int(lib().moe_sort_workspace_bytes(T, n_experts, top_k))


def sort_routes(ids: torch.Tensor, n_experts: int, first: int = 0, ws=None, stream=None) -> dict:
    """moe_sort_routes of ids [T][K] int32, for the experts first ..
    first + n_experts - 1 (routes to others are left out): a dict of int32
    tensors, offsets [n_experts+1], sorted [T*K], positions [T][K]. ws: a uint8
    workspace of sort_workspace_bytes, allocated here if None."""
    _need(ids.dim() == 2, "ids: needs two dimensions")
    dev = _device(ids)
    T, K = ids.shape
    _int32(T | K, n_experts, first)
    _check("ids", ids, dev, _I32, (T, K))
    _need(n_experts >= 0, "n_experts: negative")
    if ws is None:
        n = sort_workspace_bytes(T, n_experts, K)
        ws = _new(ids, n, torch.uint8, stream) if n else None
    else:
        _check("ws", ws, dev, (torch.uint8,), (ws.numel(),))
    offsets = _new(ids, n_experts + 1, torch.int32, stream)
    order = _new(ids, T * K, torch.int32, stream)
    positions = _new(ids, (T, K), torch.int32, stream)
    _hold(stream, ids, ws)
    _run("moe_sort_routes", dev, stream, T, n_experts, K, ids.data_ptr(), first, offsets.data_ptr(),
         order.data_ptr(), positions.data_ptr(), _ptr(ws), ws.numel() if ws is not None else 0)
    return dict(offsets=offsets, sorted=order, positions=positions)


def _int32_tensor(name: str, t: torch.Tensor, dev: torch.device, dims: int) -> torch.Tensor:
    if t.dtype != torch.int32 or t.device != dev or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name}: needs a dense int32 tensor of {dims} dimension(s) on {dev}, got {list(t.shape)} "
                         f"{t.dtype} on {t.device}, strides {t.stride()}")
    return t


def _positions(routes: dict, dev: torch.device, zero_rest: bool):
    """(positions, device address of the count of rows that are taken, or None; the tensor that holds it)."""
    positions = _int32_tensor("positions", routes["positions"], dev, 2)
    if not zero_rest:
        return positions, None, None
    offsets = _int32_tensor("offsets", routes["offsets"], dev, 1)
    _need(offsets.numel() > 0, "offsets: empty")
    return positions, offsets.data_ptr() + 4 * (offsets.numel() - 1), offsets


def _no_capture(t: torch.Tensor, what: str, instead: str) -> None:
    # (autograd would take the gradient to leaves whose accumulation is bound to the stream of an eager pass)
    with torch.cuda.device(_device(t)):
        _need(not torch.cuda.is_current_stream_capturing(),
              f"{what} requires a gradient: in a capture pass {what}.detach() and call {instead}")


def _once(what: str) -> None:
    if torch.is_grad_enabled():  # (create_graph: what comes back has no gradient of its own)
        raise RuntimeError(f"{what}: cannot differentiate twice")
    if torch.cuda.is_current_stream_capturing():  # (as _no_capture, for a forward pass that was not captured)
        raise RuntimeError(f"{what}: its gradient cannot be captured, call {what}_backward")


def gather_rows(x: torch.Tensor, routes: dict, out=None, zero_rest: bool = False, stream=None) -> torch.Tensor:
    """moe_gather_rows: x [T][cols] (bf16 or fp32, rows at any pitch) into the
    order of routes (sort_routes' dict as it came; offsets and positions are
    read): [T*K] rows, or into out [rows][cols]. Rows behind the last route are
    left as they are (as allocated, without out), or zeros with zero_rest.

    Where x requires a gradient, the rows carry it (once, on the stream that was
    current here), and those behind the last route are zeros; out is not taken.
    Not while a graph is captured: there pass x.detach() and call
    gather_rows_backward."""
    _no_tangent(x=x)
    if x.requires_grad and torch.is_grad_enabled():
        _no_capture(x, "x", "gather_rows_backward")
        _need(out is None, "out: not with an x that requires a gradient")
        return _GatherRows.apply(x, routes["offsets"], routes["positions"], stream)
    return _gather_rows(x, routes, out, zero_rest, stream)


def _gather_rows(x, routes, out, zero_rest, stream):
    _need(x.dim() == 2, "x: needs two dimensions")
    dev = _device(x)
    positions, taken, offsets = _positions(routes, dev, zero_rest)
    (T, K), cols = positions.shape, x.shape[1]
    rows = T * K if out is None else out.shape[0]
    _int32(T | K | rows | cols)
    _check("x", x, dev, _ANY_FLOAT, (T, cols), pitched=True)
    given = out
    if out is None:
        out = _new(x, (rows, cols), x.dtype, stream)
    else:
        _writable("out", out)
        _check("out", out, dev, (x.dtype,), (rows, cols), pitched=True)
    _hold(stream, x, positions, offsets, out)
    _run("moe_gather_rows", dev, stream, T, K, rows, cols, x.data_ptr(), _pitch(x), _FLOATS[x.dtype],
         positions.data_ptr(), taken, out.data_ptr(), _pitch(out))
    if given is not None:
        _written(given)
    return out


def gather_rows_backward(grad_rows: torch.Tensor, routes: dict, out_dtype=None, out=None, stream=None) -> torch.Tensor:
    """The gradient [T][cols] of gather_rows' x: the sum of its rows' gradients
    (moe_combine_rows without weights)."""
    return _combine_rows(grad_rows, routes, None, out_dtype, out, stream)


class _GatherRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, positions, stream):
        ctx.save_for_backward(offsets, positions)
        return _gather_rows(x, dict(offsets=offsets, positions=positions), None, True, stream)

    @staticmethod
    def backward(ctx, grad_rows):
        _once("gather_rows")
        offsets, positions = ctx.saved_tensors
        _hold(torch.cuda.current_stream(positions.device), positions)
        grad = _combine_rows(grad_rows.contiguous(), dict(offsets=offsets, positions=positions), None, None, None, None)
        return grad, None, None, None


def combine_rows(rows: torch.Tensor, routes: dict, w=None, out_dtype=None, out=None, stream=None) -> torch.Tensor:
    """moe_combine_rows: per token the sum of its routes' rows [rows][cols] (bf16
    or fp32, at any pitch), weighted with w [T][K] fp32 (None: 1): [T][cols] of
    out_dtype (None: that of rows), or into out.

    Where rows or w require a gradient, the result carries it (once, on the
    stream that was current here); rows behind the last route get zeros. out is
    not taken then, nor int16 (bf16 bits) for the result, and not while a graph
    is captured: there pass detached tensors and call combine_rows_backward."""
    _no_tangent(rows=rows, w=w)
    if torch.is_grad_enabled():
        for name, t in (("rows", rows), ("w", w)):
            if t is not None and t.requires_grad:
                _no_capture(rows, name, "combine_rows_backward")
                _need(out is None, "out: not with tensors that require a gradient")
                _need((rows.dtype if out_dtype is None else out_dtype) != torch.int16,
                      f"out_dtype: {name} requires a gradient, which int16 (bf16 bits) cannot carry")
                return _CombineRows.apply(rows, routes["offsets"], routes["positions"], w, out_dtype, stream)
    return _combine_rows(rows, routes, w, out_dtype, out, stream)


def _combine_rows(rows, routes, w, out_dtype, out, stream):
    _need(rows.dim() == 2, "rows: needs two dimensions")
    dev = _device(rows)
    positions, _, _ = _positions(routes, dev, False)
    (T, K), (n, cols) = positions.shape, rows.shape
    _int32(T | K | n | cols)
    _check("rows", rows, dev, _ANY_FLOAT, (n, cols), pitched=True)
    if w is not None:
        _check("w", w, dev, _F32, (T, K))
    given = out
    out = _result(rows, out, T, cols, rows.dtype if out_dtype is None else out_dtype, dev, stream)
    _hold(stream, rows, positions, w, out)
    _run("moe_combine_rows", dev, stream, T, K, n, cols, rows.data_ptr(), _pitch(rows), _FLOATS[rows.dtype],
         positions.data_ptr(), _ptr(w), out.data_ptr(), _pitch(out), _FLOATS[out.dtype])
    if given is not None:
        _written(given)
    return out


def combine_rows_backward(grad_out: torch.Tensor, rows: torch.Tensor, routes: dict, w=None, want_rows: bool = True,
                          want_w: bool = True, zero_rest: bool = False, grad_rows=None, stream=None):
    """moe_combine_rows_backward: (the gradient of rows, of their type, or into
    grad_rows; that of w [T][K] fp32) for grad_out [T][cols], or None for one not
    wanted. Rows behind the last route are left as they are (as allocated), or
    zeros with zero_rest."""
    _need(grad_out.dim() == 2 and rows.dim() == 2, "grad_out, rows: need two dimensions")
    dev = _device(rows)
    positions, taken, offsets = _positions(routes, dev, zero_rest)
    (T, K), (n, cols) = positions.shape, rows.shape
    _int32(T | K | n | cols)
    _check("grad_out", grad_out, dev, _ANY_FLOAT, (T, cols), pitched=True)
    _check("rows", rows, dev, _ANY_FLOAT, (n, cols), pitched=True)
    if w is not None:
        _check("w", w, dev, _F32, (T, K))
    given = grad_rows
    if grad_rows is not None:
        _need(want_rows, "grad_rows: given, but not wanted")
        _writable("grad_rows", grad_rows)
        _check("grad_rows", grad_rows, dev, (rows.dtype,), (n, cols), pitched=True)
    elif want_rows:
        grad_rows = _new(rows, (n, cols), rows.dtype, stream)
    grad_w = _new(rows, (T, K), torch.float32, stream) if want_w else None
    if not (want_rows or want_w):
        return None, None
    _hold(stream, grad_out, rows, positions, offsets, w, grad_rows)
    _run("moe_combine_rows_backward", dev, stream, T, K, n, cols, grad_out.data_ptr(), _pitch(grad_out),
         _FLOATS[grad_out.dtype], rows.data_ptr(), _pitch(rows), _FLOATS[rows.dtype], positions.data_ptr(), _ptr(w),
         taken, _ptr(grad_rows), _pitch(grad_rows) if want_rows else cols, _ptr(grad_w))
    if given is not None:
        _written(given)
    return grad_rows, grad_w


class _CombineRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, offsets, positions, w, out_dtype, stream):
        ctx.save_for_backward(rows, offsets, positions, w)
        return _combine_rows(rows, dict(offsets=offsets, positions=positions), w, out_dtype, None, stream)

    @staticmethod
    def backward(ctx, grad_out):
        _once("combine_rows")
        rows, offsets, positions, w = ctx.saved_tensors
        _hold(torch.cuda.current_stream(rows.device), rows, offsets, positions, w)
        grad_rows, grad_w = combine_rows_backward(
            grad_out.contiguous(), rows, dict(offsets=offsets, positions=positions), w, ctx.needs_input_grad[0],
            ctx.needs_input_grad[3], True)
        return grad_rows, None, None, grad_w, None, None


def balance_workspace_bytes(T: int, n_experts: int) -> int:
    _int32(T, n_experts)
    return int(lib().moe_balance_workspace_bytes(T, n_experts))


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, mask=None, ws=None, stream=None):
    """moe_balance_loss of logits [T][E] fp32 and ids [T][K] int32, mask [T]
    uint8 or bool (tokens that count; None: all): (losses [2] fp32: balance,
    z; counts [E+1] int32: routes per expert, tokens that counted). ws: a
    uint8 workspace of balance_workspace_bytes, allocated here if None.

    Where logits requires a gradient, the losses carry theirs (of this call's
    own counts, once, on the stream that was current here; without the router
    weights' part, which is balance_loss_backward's). Not while a graph is
    captured: there pass logits.detach() and call balance_loss_backward."""
    _no_tangent(logits=logits)
    if logits.requires_grad and torch.is_grad_enabled():
        # (autograd would take the gradient to leaves whose accumulation is bound to the stream of an eager pass)
        with torch.cuda.device(_device(logits)):
            _need(not torch.cuda.is_current_stream_capturing(),
                  "logits requires a gradient: in a capture pass logits.detach() and call balance_loss_backward")
        return _BalanceLoss.apply(logits, ids, mask, ws, stream)
    return _balance_loss(logits, ids, mask, ws, stream)


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, mask, ws, stream):
        losses, counts = _balance_loss(logits, ids, mask, ws, stream)
        ctx.save_for_backward(logits, ids, counts, mask)
        ctx.mark_non_differentiable(counts)
        return losses, counts

    @staticmethod
    def backward(ctx, grad_losses, _):
        if torch.is_grad_enabled():  # (create_graph: what comes back has no gradient of its own)
            raise RuntimeError("balance_loss: cannot differentiate twice")
        logits, ids, counts, mask = ctx.saved_tensors
        # (counts may be of a given stream's pool)
        _hold(torch.cuda.current_stream(counts.device), counts)
        return balance_loss_backward(logits, ids, counts, grad_losses.contiguous(), mask), None, None, None, None


def _balance_loss(logits, ids, mask, ws, stream):
    _need(logits.dim() == 2 and ids.dim() == 2, "logits, ids: need two dimensions")
    dev = _device(logits)
    (T, E), K = logits.shape, ids.shape[1]
    _int32(T | E | K)
    _check("logits", logits, dev, _F32, (T, E))
    _check("ids", ids, dev, _I32, (T, K))
    if mask is not None:
        _check("mask", mask, dev, _MASK, (T,))
    if ws is None:
        n = balance_workspace_bytes(T, E)
        ws = _empty(n, torch.uint8, dev, stream) if n else None
    else:
        _check("ws", ws, dev, (torch.uint8,), (ws.numel(),))
    losses = _empty(2, torch.float32, dev, stream)
    counts = _empty(E + 1, torch.int32, dev, stream)
    _hold(stream, logits, ids, mask, ws)
    _run("moe_balance_loss", dev, stream, T, E, K, logits.data_ptr(), ids.data_ptr(), _ptr(mask),
         counts.data_ptr(), losses.data_ptr(), _ptr(ws), ws.numel() if ws is not None else 0)
    return losses, counts


def balance_loss_backward(logits: torch.Tensor, ids: torch.Tensor, counts: torch.Tensor,
                          grad_losses: torch.Tensor, mask=None, w=None, grad_w=None, out=None,
                          stream=None) -> torch.Tensor:
    """moe_balance_loss_backward: the gradient [T][E] fp32 of the logits
    through both losses (grad_losses [2] fp32 on the device, counts as
    balance_loss gave them or summed over processes) and, with w and grad_w
    [T][K] fp32, through the router weights."""
    _need(logits.dim() == 2 and ids.dim() == 2, "logits, ids: need two dimensions")
    dev = _device(logits)
    (T, E), K = logits.shape, ids.shape[1]
    _int32(T | E | K)
    _check("logits", logits, dev, _F32, (T, E))
    _check("ids", ids, dev, _I32, (T, K))
    _check("counts", counts, dev, _I32, (E + 1,))
    _check("grad_losses", grad_losses, dev, _F32, (2,))
    if mask is not None:
        _check("mask", mask, dev, _MASK, (T,))
    _need((w is None) == (grad_w is None), "w, grad_w: both or neither")
    if w is not None:
        _check("w", w, dev, _F32, (T, K))
        _check("grad_w", grad_w, dev, _F32, (T, K))
    given = out
    if out is None:
        out = _empty((T, E), torch.float32, dev, stream)
    else:
        _writable("out", out)
        _check("out", out, dev, _F32, (T, E))
    _hold(stream, logits, ids, counts, grad_losses, mask, w, grad_w, out)
    _run("moe_balance_loss_backward", dev, stream, T, E, K, logits.data_ptr(), ids.data_ptr(), _ptr(mask),
         counts.data_ptr(), grad_losses.data_ptr(), _ptr(w), _ptr(grad_w), out.data_ptr())
    if given is not None:
        _written(given)
    return out


# ---- HIP events (timing of the stages on the stream they run on) ----------
_hip = None


def hip_runtime():
    global _hip
    if _hip is None:
        _hip = ctypes.CDLL("libamdhip64.so")
        _hip.hipEventCreate.argtypes = [ctypes.POINTER(_vp)]
        _hip.hipEventDestroy.argtypes = [_vp]
        _hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), _vp, _vp]
        _hip.hipEventSynchronize.argtypes = [_vp]
    return _hip


def create_events(n: int) -> list[int]:
    evs = []
    for _ in range(n):
        e = _vp()
        rc = hip_runtime().hipEventCreate(ctypes.byref(e))
        if rc != 0:
            raise RuntimeError(f"hipEventCreate failed: {rc}")
        evs.append(e.value)
    return evs


def elapsed_ms(e0: int, e1: int) -> float:
    ms = ctypes.c_float()
    rc = hip_runtime().hipEventElapsedTime(ctypes.byref(ms), e0, e1)
    if rc != 0:
        raise RuntimeError(f"hipEventElapsedTime failed: {rc}")
    return ms.value


def destroy_events(evs) -> None:
    for e in evs:
        hip_runtime().hipEventDestroy(e)
