"""Cases of 4-bit (MXFP4) rows with their products, and of the way into and out of expert order.

Six operators, as one user of the layer meets them:

* ``quantize``: rows to E2M1 codes with one power-of-two scale per 32 values, and back;
* ``linear``: a projection of rows that are quantised on the way in, weights kept in 4 bits;
* ``grouped``: the same for every expert over the routes that chose it (gate and up);
* ``down``: SwiGLU of the routes' gate and up values to 4 bits, then every expert's down projection (to bf16 rows: where a
  value lies next to a border of its 4-bit steps, another exponential's last bit moves it by a whole step);
* ``dispatch``: routes sorted by expert, the tokens' rows copied into that order, and the gradient of the tokens;
* ``combine``: the routes' rows weighted and summed per token, and the gradients of rows and weights.
"""
import math
from statistics import NormalDist

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # of codes 0 .. 7; 8 .. 15 are their negatives


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # the latent rows of 32 verified tokens before the experts: latency counts
        dict(name="quantize 32 x 4096", op="quantize", rows=32, cols=4096, type="bf16"),
        # the layer input of a 4096-token prefill before the pooler
        dict(name="quantize 4096 x 8192", op="quantize", rows=4096, cols=8192, type="bf16"),
        # the pooler for one decoded token
        dict(name="linear 1 token", op="linear", tokens=1, n=4096, k=8192, type="bf16"),
        # the pooler over a prefill
        dict(name="linear 4096 tokens", op="linear", tokens=4096, n=4096, k=8192, type="bf16"),
        # gate and up of one decoded token: its 8 routes' experts
        dict(name="gate/up 1 token", op="grouped", tokens=1, experts=256, top_k=8, n=8192, k=4096, type="bf16"),
        # gate and up of a ragged prefill on as many experts as one of eight processes holds
        dict(name="gate/up 1000 tokens", op="grouped", tokens=1000, experts=32, top_k=8, n=8192, k=4096, type="bf16"),
        # a 32-token verification step: nearly every touched expert has one or two rows
        dict(name="down 32 tokens", op="down", tokens=32, experts=256, top_k=8, n=4096, k=4096, type="f32"),
        # a prefill: about 128 rows per expert
        dict(name="down 4096 tokens", op="down", tokens=4096, experts=256, top_k=8, n=4096, k=4096, type="bf16"),
        # the latent rows of one micro-batch of training into expert order
        dict(name="dispatch 4096 tokens", op="dispatch", tokens=4096, experts=256, local=256, top_k=8, cols=4096,
             type="bf16"),
        # a short training batch of the reduced layer, on the experts that one of two processes holds
        dict(name="dispatch 61 tokens", op="dispatch", tokens=61, experts=16, local=8, top_k=4, cols=384, type="f32"),
        # the same batch's rows back
        dict(name="combine 61 tokens", op="combine", tokens=61, experts=16, local=8, top_k=4, cols=384, type="f32",
             out="bf16"),
        # the micro-batch's rows back
        dict(name="combine 4096 tokens", op="combine", tokens=4096, experts=256, local=256, top_k=8, cols=4096,
             type="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grouped", "down", "dispatch", "combine"])
    kind = rng.choice(["bf16", "f32"])
    if op == "quantize":
        cols = 32 * _log(rng, 2, 256)
        return dict(op=op, rows=_log(rng, 1, min(32768, 4096 * 8192 // cols)), cols=cols, type=kind)
    if op == "linear":
        return dict(op=op, tokens=_log(rng, 1, 4096), n=_log(rng, 64, 4096), k=32 * _log(rng, 2, 256), type=kind)
    experts = _log(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    if op in ("grouped", "down"):
        return dict(op=op, tokens=_log(rng, 1, 4096), experts=experts, top_k=top_k, n=_log(rng, 64, 4096),
                    k=32 * _log(rng, 2, 128), type=kind)
    cols = _log(rng, 16, 8192)
    if rng.random() < 0.7:
        cols = (cols + 7) // 8 * 8
    case = dict(op=op, tokens=_log(rng, 1, min(32767, 4096 * 4096 // cols)), experts=experts,
                local=experts if rng.random() < 0.5 else rng.randint(1, experts), top_k=top_k, cols=cols, type=kind)
    if op == "combine":
        case["out"] = rng.choice(["bf16", "f32"])
    return case


def work(case):
    op = case["op"]
    size = 2 if case["type"] == "bf16" else 4
    four = 0.5 + 1 / 32  # bytes of a 4-bit value with its share of the scale
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * 2 * size, "flops": n * 4}
    if op == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": t * k * size + n * k * four + t * n * size, "flops": 2 * t * n * k}
    if op in ("grouped", "down"):
        t, e, r, n, k = case["tokens"], case["experts"], case["tokens"] * case["top_k"], case["n"], case["k"]
        touched = e * (1 - (1 - case["top_k"] / e) ** t)  # of experts chosen at random
        rows, out = (t * k, size) if op == "grouped" else (r * 2 * k, 2)
        return {"bytes": touched * n * k * four + rows * size + r * n * out + 4 * r, "flops": 2 * r * n * k}
    t, k, c = case["tokens"], case["top_k"], case["cols"]
    taken = t * k * case["local"] / case["experts"]
    if op == "dispatch":  # x in, rows out; the rows' gradients in, x's out
        return {"bytes": (2 * t + t * k + taken) * c * size + 12 * t * k, "flops": taken * c}
    out = 2 if case["out"] == "bf16" else 4  # rows in, out out; rows and out's gradient in, rows' out
    return {"bytes": (2 * taken + t * k) * c * size + 2 * t * c * out + 16 * t * k, "flops": 5 * taken * c}


# ---- inputs -----------------------------------------------------------------------------------

def _activations(rows, cols, gen):
    """Normal, the rows' sizes spread, a few channels far larger than the others."""
    size = torch.exp(torch.randn((rows, 1), generator=gen, device="cuda"))
    channel = 1.0 + 30.0 * (torch.rand((1, cols), generator=gen, device="cuda") < 0.002)
    return torch.randn((rows, cols), generator=gen, device="cuda") * size * channel


def _pairs():
    """Bytes of two codes each, as normal weights scaled by their group's largest value give them."""
    edges = [(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])]
    codes = []
    for i in range(256):
        v = 2.2 * NormalDist().inv_cdf((i + 0.5) / 256)
        codes.append(sum(abs(v) > e for e in edges) + (8 if v < 0 else 0))
    c = torch.tensor(codes, dtype=torch.uint8, device="cuda")
    return (c[:, None] | (c[None, :] << 4)).reshape(-1)


def _weights(experts, n, k, gen):
    pairs = _pairs()
    codes = torch.empty((experts, n, k // 2), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        codes[e] = pairs[torch.randint(0, 65536, (n, k // 2), generator=gen, device="cuda", dtype=torch.int32)]
    about = 127 - 1 - int(round(math.log2(k) / 2))
    scales = torch.randint(about - 1, about + 2, (experts, n, k // 32), generator=gen, device="cuda",
                           dtype=torch.int32).to(torch.uint8)
    return codes, scales


def _ids(case, gen):
    """Routing as the router gives it: the best top_k of normal logits."""
    logits = torch.randn((case["tokens"], case["experts"]), generator=gen, device="cuda")
    return logits.topk(case["top_k"], dim=1).indices.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, kind = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op == "quantize":
        s["x"] = _activations(case["rows"], case["cols"], gen).to(kind)
        return s
    if op == "linear":
        s["x"] = _activations(case["tokens"], case["k"], gen).to(kind)
        w, ws = _weights(1, case["n"], case["k"], gen)
        s["w"], s["ws"] = w[0], ws[0]
        return s
    if op in ("grouped", "down"):
        ids = _ids(case, gen).reshape(-1).long()
        s["order"] = torch.argsort(ids, stable=True).to(torch.int32)  # routes t * top_k + j, grouped by expert
        counts = torch.bincount(ids, minlength=case["experts"])
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # rows of the fullest expert, for the plain form's padding
        rows = case["tokens"] if op == "grouped" else ids.numel()
        s["x"] = _activations(rows, case["k"] * (1 if op == "grouped" else 2), gen).to(kind)
        s["w"], s["ws"] = _weights(case["experts"], case["n"], case["k"], gen)
        return s
    t, k, c = case["tokens"], case["top_k"], case["cols"]
    s["ids"] = _ids(case, gen)
    s["first"] = (case["experts"] - case["local"]) // 2
    if op == "dispatch":
        s["x"] = torch.randn((t, c), generator=gen, device="cuda").to(kind)
        s["drows"] = torch.randn((t * k, c), generator=gen, device="cuda").to(kind)
        return s
    s["routes"] = _plain_sort(s["ids"], s["local"], s["first"])  # what the dispatch before has left
    s["rows"] = torch.randn((t * k, c), generator=gen, device="cuda").to(kind)
    s["weights"] = torch.softmax(torch.randn((t, k), generator=gen, device="cuda"), 1)
    s["dout"] = torch.randn((t, c), generator=gen, device="cuda").to(TYPES[case["out"]])
    return s


# ---- the operators ----------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from latent_mixture_experts_amd import binding as B

    op, kind = s["op"], TYPES[s["type"]]
    if op == "quantize":
        codes, scales = B.fp4_quantize(s["x"])
        return B.fp4_dequantize(codes, scales, kind)
    if op == "linear":
        codes, scales = B.fp4_quantize(s["x"])
        return B.fp4_linear(codes, scales, s["w"], s["ws"], kind)
    if op == "grouped":
        codes, scales = B.fp4_quantize(s["x"])
        return B.fp4_grouped(codes, scales, s["offsets"], s["w"], s["ws"], kind, row_index=s["order"],
                             index_div=s["top_k"])
    if op == "down":
        codes, scales = B.fp4_swiglu(s["x"])
        return B.fp4_grouped(codes, scales, s["offsets"], s["w"], s["ws"], torch.bfloat16)
    if op == "dispatch":
        routes = B.sort_routes(s["ids"], s["local"], s["first"])
        rows = B.gather_rows(s["x"], routes, zero_rest=True)
        return dict(routes, rows=rows, dx=B.gather_rows_backward(s["drows"], routes))
    out = B.combine_rows(s["rows"], s["routes"], s["weights"], TYPES[s["out"]])
    drows, dw = B.combine_rows_backward(s["dout"], s["rows"], s["routes"], s["weights"], zero_rest=True)
    return {"out": out, "drows": drows, "dweights": dw}


def _plain(s):
    op, kind = s["op"], TYPES[s["type"]]
    if op == "quantize":
        return _plain_round(s["x"].float()).to(kind)
    if op == "linear":
        return (_plain_round(s["x"].float()) @ _plain_values(s["w"], s["ws"]).t()).to(kind)
    if op == "grouped":
        token = torch.div(s["order"], s["top_k"], rounding_mode="floor")
        return _plain_experts(s, _plain_round(s["x"].float())[token]).to(kind)
    if op == "down":
        gate, up = s["x"].float().chunk(2, dim=1)
        return _plain_experts(s, _plain_round(gate / (1.0 + torch.exp(-gate)) * up)).to(torch.bfloat16)
    if op == "dispatch":
        return _plain_dispatch(s)
    return _plain_combine(s)


def _plain_round(v):
    """Every value to the nearest of its group's 4-bit values."""
    g = v.view(v.shape[0], -1, 32)
    amax = g.abs().amax(2, keepdim=True)
    # the exponent of the largest value, rounded to two significant bits as the codes are
    byte = ((amax.view(torch.int32) + 0x200000) >> 23).sub(2).clamp(1, 254)
    scale = (byte << 23).view(torch.float32)
    q = g / scale
    size = q.abs()
    step = torch.where(size < 2.0, 0.5, torch.where(size < 4.0, 1.0, 2.0))
    return (torch.round(q / step) * step * scale).view_as(v)


def _plain_values(codes, scales):
    """fp32 values of packed codes, two per byte, the first in the low half."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    at = torch.arange(256, device="cuda")
    pairs = torch.stack([table[at & 15], table[at >> 4]], 1)
    v = pairs[codes.int()].view(*codes.shape[:-1], -1, 32)
    return (v * (scales.int() << 23).view(torch.float32)[..., None]).view(*codes.shape[:-1], -1)


def _plain_experts(s, x):
    """Rows in expert order times their expert's weights: the touched experts at once, each with as many rows as the fullest."""
    start, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    touched = (end > start).nonzero()[:, 0]
    at = start[touched, None] + torch.arange(s["most"], device="cuda")
    live = at < end[touched, None]
    rows = x[torch.where(live, at, 0)]
    w = _plain_values(s["w"][touched], s["ws"][touched])
    out = torch.bmm(w, rows.transpose(1, 2).contiguous()).transpose(1, 2)
    return out[live]


def _plain_sort(ids, local, first):
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < local), flat, local)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(local, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    at = torch.arange(flat.numel(), device="cuda")
    positions = torch.empty_like(order)
    positions[order] = at
    sorted_routes = torch.where(at < offsets[-1], order, -1)
    positions = torch.where(key < local, positions, -1).view(ids.shape)
    return {k: v.to(torch.int32) for k, v in dict(offsets=offsets, sorted=sorted_routes, positions=positions).items()}


def _plain_dispatch(s):
    routes = _plain_sort(s["ids"], s["local"], s["first"])
    order, at = routes["sorted"].long(), routes["positions"].long()
    token = torch.div(order.clamp(min=0), s["top_k"], rounding_mode="floor")
    rows = torch.where((order >= 0)[:, None], s["x"][token], 0)
    parts = s["drows"].float()[at.clamp(min=0)]  # [tokens][top_k][cols]
    dx = torch.where((at >= 0)[:, :, None], parts, 0.0).sum(1)
    return dict(routes, rows=rows, dx=dx.to(s["drows"].dtype))


def _plain_combine(s):
    order, at = s["routes"]["sorted"].long(), s["routes"]["positions"].long()
    rows, dout, w = s["rows"].float(), s["dout"].float(), s["weights"]
    mine = torch.where((at >= 0)[:, :, None], rows[at.clamp(min=0)], 0.0)  # [tokens][top_k][cols]
    out = (w[:, :, None] * mine).sum(1)
    dw = (dout[:, None, :] * mine).sum(2)
    route = order.clamp(min=0)
    token = torch.div(route, s["top_k"], rounding_mode="floor")
    drows = torch.where((order >= 0)[:, None], w.reshape(-1)[route][:, None] * dout[token], 0.0)
    return {"out": out.to(s["dout"].dtype), "drows": drows.to(s["rows"].dtype), "dweights": dw}


# ---- from the definitions, in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_round(s["x"].double())
    if op == "linear":
        return _exact_round(s["x"].double()) @ _exact_values(s["w"], s["ws"]).t()
    if op in ("grouped", "down"):
        if op == "grouped":
            x = _exact_round(s["x"].double())[s["order"].long() // case["top_k"]]
        else:
            v, half = s["x"].double(), case["k"]
            x = _exact_round(v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:])
        out = torch.empty((x.shape[0], case["n"]), dtype=torch.float64, device="cuda")
        bounds = s["offsets"].tolist()
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if b > a:
                out[a:b] = x[a:b] @ _exact_values(s["w"][e], s["ws"][e]).t()
        return out
    t, k = case["tokens"], case["top_k"]
    local = (s["ids"] >= s["first"]) & (s["ids"] < s["first"] + case["local"])
    if op == "dispatch":
        keyed = sorted((int(e), r) for r, e in enumerate(s["ids"].reshape(-1).tolist())
                       if s["first"] <= e < s["first"] + case["local"])
        order = torch.tensor([r for _, r in keyed], dtype=torch.int64, device="cuda")
        rows = torch.zeros((t * k, case["cols"]), dtype=torch.float64, device="cuda")
        rows[:order.numel()] = s["x"].double()[order // k]
        dx = torch.zeros((t, case["cols"]), dtype=torch.float64, device="cuda")
        dx.index_add_(0, order // k, s["drows"][:order.numel()].double())
        return {"offsets": None, "sorted": None, "positions": None, "rows": rows, "dx": dx}
    out = torch.zeros((t, case["cols"]), dtype=torch.float64, device="cuda")
    drows = torch.zeros((t * k, case["cols"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        who = local[:, j].nonzero()[:, 0]
        at = s["routes"]["positions"][who, j].long()
        weight, mine, above = s["weights"][who, j].double()[:, None], s["rows"][at].double(), s["dout"][who].double()
        out[who] += weight * mine
        drows[at] = weight * above
        dw[who, j] = (mine * above).sum(1)
    return {"out": out, "drows": drows, "dweights": dw}


def _exact_round(v):
    out = torch.empty_like(v)
    values = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for a in range(0, v.shape[1], 32):
        g = v[:, a:a + 32]
        top = g.abs().amax(1, keepdim=True).clamp(min=2.0 ** -124)
        scale = torch.exp2(torch.floor(torch.log2(top)) - 2)
        scale = torch.where(top / scale >= 7, 2 * scale, scale)
        size = g.abs() / scale
        # the nearest value; of two as near the one with the even code
        low = (torch.searchsorted(values, size.contiguous(), right=True) - 1).clamp(0, 6)
        down, up = size - values[low], values[low + 1] - size
        code = torch.where((up < down) | ((up == down) & (low % 2 == 1)), low + 1, low)
        out[:, a:a + 32] = torch.sign(g) * values[code] * scale
    return out


def _exact_values(codes, scales):
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    v = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = table[(codes & 15).long()], table[(codes >> 4).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
