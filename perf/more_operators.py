"""The operators of a mixture-of-experts layer in 8-bit floating point as they are measured: their inputs, plain
forms, exact forms and work.

Operators (op): "product" gemm_f8_tn, C = A B^T of two 8-bit matrices with an FP32 scale for each block of 128 along K
(of a row, or of a band of 128 rows); "experts" gemm_f8_tn_experts, the same for rows sorted by expert and a weight
matrix an expert; "quantize" quantize_f8 / swiglu_f8, rows in that form; "dispatch" sort_by_expert and
gather_by_expert(_f8), tokens to expert order, with the gradient where they train; "combine" combine_experts, back
with the router's weights applied, and combine_experts_grad.  What is held in 8 bits is returned as the values it
stands for (dequantize_f8, to 16 bits), beside the scales.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # the largest value of either type
BLOCK = 128


def listed():
    return [
        # one token through one projection: the latency of decoding, bound by the weights' bytes
        {"name": "product_1x8192x4096", "op": "product", "m": 1, "n": 8192, "k": 4096, "out": "bf16", "a": "e4m3", "wgrad": False, "bias": False},
        # a weight's gradient added up in FP32: scales a row on either side, e5m2 gradients, a ragged number of tokens
        {"name": "product_2048x4096x1000_wgrad", "op": "product", "m": 2048, "n": 4096, "k": 1000, "out": "f32", "a": "e5m2", "wgrad": True, "bias": False},
        # a long prompt: bound by the tensor cores
        {"name": "product_8192x8192x4096", "op": "product", "m": 8192, "n": 8192, "k": 4096, "out": "bf16", "a": "e4m3", "wgrad": False, "bias": False},
        # a decoding batch of 16 tokens, 8 of 64 experts each: a few rows an expert, bound by the weights' bytes
        {"name": "experts_16x8of64", "op": "experts", "tokens": 16, "top": 8, "e": 64, "n": 4096, "k": 2048, "out": "bf16", "padded": False},
        # a long prompt through the same layer: about a thousand rows an expert, some with far more
        {"name": "experts_8192x8of64", "op": "experts", "tokens": 8192, "top": 8, "e": 64, "n": 4096, "k": 2048, "out": "bf16", "padded": False},
        # the gated activation of a decoding batch's sorted rows
        {"name": "swiglu_128x2048", "op": "quantize", "form": "swiglu", "m": 128, "k": 2048, "type": "bf16", "f8": "e4m3"},
        # activations for the weight's gradient: groups of 128 tokens down each column, sizes ragged
        {"name": "quantize_8191x4104_transposed", "op": "quantize", "form": "transposed", "m": 8191, "k": 4104, "type": "bf16", "f8": "e4m3"},
        # a weight matrix at load: blocks of 128 x 128
        {"name": "quantize_16384x8192_blocks", "op": "quantize", "form": "blocks", "m": 16384, "k": 8192, "type": "f32", "f8": "e4m3"},
        # the decoding batch's tokens to expert order in 8 bits, a quarter of it padding
        {"name": "dispatch_16x8of64_f8", "op": "dispatch", "tokens": 16, "top": 8, "e": 64, "k": 4096, "type": "bf16", "train": False, "padded": True},
        # a training batch to expert order in 16 bits, and its gradient back
        {"name": "dispatch_8192x8of64_train", "op": "dispatch", "tokens": 8192, "top": 8, "e": 64, "k": 4096, "type": "bf16", "train": True, "padded": False},
        # the decoding batch's rows back, added to the residual stream
        {"name": "combine_16x8", "op": "combine", "tokens": 16, "top": 8, "e": 64, "k": 4096, "type": "bf16", "train": False, "padded": True},
        # a training batch's rows back and the gradients of the rows and the router's weights
        {"name": "combine_8192x8_train", "op": "combine", "tokens": 8192, "top": 8, "e": 64, "k": 4096, "type": "bf16", "train": True, "padded": False},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row's length: a multiple of 128, as most models have, or any."""
    k = _log(rng, low, high)
    return k if rng.random() < 0.4 else max(128, k // 128 * 128)


def draw(rng):
    op = rng.choice(["product", "product", "product", "experts", "experts", "quantize", "dispatch", "combine"])
    if op == "product":
        m, n, k = _log(rng, 1, 8192), _width(rng, 512, 16384), _width(rng, 512, 16384)
        wgrad = rng.random() < 0.3
        k = max(128, min(k, 8192 * 8192 * 4096 // (m * n)))
        return {"op": op, "m": m, "n": n, "k": k, "out": "f32" if wgrad else rng.choice(["bf16", "bf16", "f16", "f32"]),
                "a": "e5m2" if wgrad else "e4m3", "wgrad": wgrad, "bias": not wgrad and rng.random() < 0.4}
    if op == "quantize":
        form = rng.choice(["rows", "swiglu", "transposed", "blocks"])
        case = {"op": op, "form": form, "k": _width(rng, 512, 16384), "type": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "f8": rng.choice(["e4m3", "e4m3", "e5m2"])}
        case["m"] = min(_log(rng, 1, 16384), 8192 * 8192 // case["k"])
        return case
    e = rng.choice([8, 16, 60, 64, 128, 256])
    case = {"op": op, "tokens": _log(rng, 1, 8192), "top": rng.choice([1, 2, 4, 6, 8]), "e": e, "padded": rng.random() < 0.3}
    if op == "experts":
        case["n"], case["k"] = _width(rng, 512, 8192), _width(rng, 512, 4096)
        while e * case["n"] * case["k"] > 64 * 4096 * 2048:
            case["n"], case["k"] = max(512, case["n"] // 2), max(512, case["k"] // 2)
            case["e"] = e = e if case["n"] > 512 else max(8, e // 2)
        case["tokens"] = max(1, min(case["tokens"], 65536 * 4096 * 2048 // (case["top"] * case["n"] * case["k"])))
        case["out"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        return case
    case["k"] = _width(rng, 512, 8192)
    case["tokens"] = max(1, min(case["tokens"], 65536 * 4096 // (case["top"] * case["k"])))
    case["type"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if case["type"] == "f32":
        case["tokens"] = max(1, case["tokens"] // 2)
    case["train"] = rng.random() < 0.5
    return case


def _pitched(rows, cols, dtype):
    """A rows x cols matrix whose rows start 16 bytes aligned, as a program lays out rows of any length."""
    step = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros((rows, -(-cols // step) * step), dtype=dtype, device="cuda")[:, :cols]


def _blocks(k):
    return -(-k // BLOCK)


def _padded(x, rows, cols):
    """x with zeros up to multiples of rows and cols."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _quantized(x, rows, f8):
    """(Q, scale) of FP32 rows, a scale for each rows x 128 values, by elementary operations."""
    m, k = x.shape
    y = _padded(x, rows, BLOCK)
    y = y.view(y.shape[0] // rows, rows, y.shape[1] // BLOCK, BLOCK)
    a = y.abs().amax((1, 3))
    inv = torch.where(a > 0, TOP[f8] / a, 0.0)
    q = (y * inv[:, None, :, None]).view(y.shape[0] * rows, -1)[:m, :k].to(F8[f8])
    return q, a / TOP[f8]


def _spread(scale, rows, m, k):
    """A scale for each value."""
    s = scale.repeat_interleave(BLOCK, -1)[..., :k]
    return s.repeat_interleave(rows, -2)[..., :m, :] if rows > 1 else s


def _held(q):
    out = _pitched(q.shape[0], q.shape[1], q.dtype)
    out.copy_(q)
    return out


def _routing(case, g):
    """(experts, weights) of each token: the top of the router's logits, some experts liked more than others."""
    t, e, top = case["tokens"], case["e"], case["top"]
    logits = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
    best, experts = torch.topk(logits, top, dim=1)
    experts, weights = experts.to(torch.int32), torch.softmax(best, 1)
    if case["padded"]:  # the batch's last quarter is padding
        experts[t - t // 4:] = -1
    return experts.contiguous(), weights.contiguous()


def _sorted(experts, e):
    """(offsets, position) of the pairs (token, choice) sorted by expert, in their order within an expert."""
    flat = experts.reshape(-1).long()
    keys = torch.where((flat >= 0) & (flat < e), flat, e)
    keys, order = torch.sort(keys, stable=True)
    offsets = torch.searchsorted(keys, torch.arange(e + 1, device=keys.device))
    row = torch.arange(keys.numel(), device=keys.device)
    position = torch.empty_like(row).scatter_(0, order, torch.where(keys < e, row, -1))
    return offsets.to(torch.int32), position.view(experts.shape).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, k = case["op"], case["k"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def activations(m, cols=k):
        # normal, some channels several times louder than the rest
        x = normal(m, cols)
        x[:, torch.rand(cols, generator=g, device="cuda") < 0.004] *= 6.0
        return x

    if op == "product":
        m, n = case["m"], case["n"]
        a, sa = _quantized(activations(m), 1, case["a"])
        b, sb = _quantized(normal(n, k) / math.sqrt(k), 1 if case["wgrad"] else BLOCK, "e4m3")
        c = _pitched(m, n, TYPES[case["out"]])
        if case["wgrad"]:
            c.copy_(normal(m, n))
        return {"op": op, "a": _held(a), "b": _held(b), "sa": sa, "sb": sb, "rows": 1 if case["wgrad"] else BLOCK,
                "bias": normal(n) * 0.1 if case["bias"] else None, "beta": 1.0 if case["wgrad"] else 0.0, "c": c,
                "c0": c.clone()}
    if op == "quantize":
        m, form, dtype, f8 = case["m"], case["form"], TYPES[case["type"]], F8[case["f8"]]
        x = _pitched(m, k, dtype)
        x.copy_(normal(m, k) / math.sqrt(k) if form == "blocks" else activations(m))
        qm, qk, rows = (k, m, 1) if form == "transposed" else (m, k, BLOCK if form == "blocks" else 1)
        s = {"op": op, "form": form, "f8": case["f8"], "x": x, "u": None, "q": _pitched(qm, qk, f8),
             "scale": torch.zeros(-(-qm // rows), _blocks(qk), device="cuda"),
             "v": _pitched(qm, qk, torch.float16 if dtype == torch.float16 else torch.bfloat16)}
        if form == "swiglu":
            s["u"] = _pitched(m, k, dtype)
            s["u"].copy_(activations(m))
        return s
    experts, weights = _routing(case, g)
    offsets, position = _sorted(experts, case["e"])
    rows = case["tokens"] * case["top"]
    if op == "experts":
        e, n = case["e"], case["n"]
        a, sa = _quantized(activations(rows), 1, "e4m3")
        w = normal(e, n, k) / math.sqrt(k)
        w = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK))  # blocks do not cross experts
        b, sb = _quantized(w.view(-1, w.shape[2]), BLOCK, "e4m3")
        held = torch.zeros((e, n, -(-k // 16) * 16), dtype=b.dtype, device="cuda")[:, :, :k]
        held.copy_(b.view(w.shape)[:, :n, :k])
        return {"op": op, "a": _held(a), "sa": sa, "b": held, "sb": sb.view(e, -1, sb.shape[1]), "offsets": offsets,
                "most": int((offsets[1:] - offsets[:-1]).max()), "c": _pitched(rows, n, TYPES[case["out"]])}
    dtype = TYPES[case["type"]]

    def held(m, x=None):
        y = _pitched(m, k, dtype)
        return y if x is None else y.copy_(x)

    if op == "dispatch":
        s = {"op": op, "train": case["train"], "e": case["e"], "experts": experts, "x": held(case["tokens"], activations(case["tokens"])),
             "offsets": torch.empty_like(offsets), "position": torch.empty_like(position)}
        if case["train"]:
            return {**s, "y": held(rows), "dy": held(rows, normal(rows, k)), "dx": held(case["tokens"])}
        return {**s, "q": _pitched(rows, k, torch.float8_e4m3fn), "scale": torch.zeros(rows, _blocks(k), device="cuda"),
                "v": _pitched(rows, k, torch.float16 if dtype == torch.float16 else torch.bfloat16)}
    s = {"op": op, "train": case["train"], "y": held(rows, normal(rows, k)), "position": position, "weights": weights,
         "x": held(case["tokens"], 2.0 * normal(case["tokens"], k))}
    s["x0"] = s["x"].clone()
    if case["train"]:
        s.update(dx=held(case["tokens"], normal(case["tokens"], k)), dy=held(rows), dw=torch.empty_like(weights))
    return s


def _plain_product(s):
    m, k = s["a"].shape
    a = s["a"].float() * _spread(s["sa"], 1, m, k)
    b = s["b"].float() * _spread(s["sb"], s["rows"], s["b"].shape[0], k)
    y = a @ b.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["beta"]:
        y = y + s["beta"] * s["c0"].float()
    return y.to(s["c"].dtype)


def _places(offsets, rows):
    """(expert, place within the expert, whether it has one) of each sorted row."""
    row = torch.arange(rows, device=offsets.device, dtype=offsets.dtype)
    expert = (torch.searchsorted(offsets, row, right=True) - 1).clamp_(max=offsets.numel() - 2)
    return expert, (row - offsets[expert]).long(), row < offsets[-1]


def _plain_experts(s):
    (m, k), (_, n, _) = s["a"].shape, s["b"].shape
    a = s["a"].float() * _spread(s["sa"], 1, m, k)
    b = s["b"].float() * _spread(s["sb"], BLOCK, n, k)
    at = s["offsets"][:-1, None] + torch.arange(max(s["most"], 1), device=a.device)
    y = torch.bmm(a[at.clamp(max=m - 1)], b.transpose(1, 2))
    expert, place, real = _places(s["offsets"], m)
    y = y[expert, place.clamp(0, y.shape[1] - 1)]
    return torch.where(real[:, None], y, 0.0).to(s["c"].dtype)


def _plain_quantize(s):
    x = s["x"].float()
    if s["form"] == "swiglu":
        x = x / (1.0 + torch.exp(-x)) * s["u"].float()
    elif s["form"] == "transposed":
        x = x.t()
    rows = BLOCK if s["form"] == "blocks" else 1
    q, scale = _quantized(x, rows, s["f8"])
    return {"values": (q.float() * _spread(scale, rows, *x.shape)).to(s["v"].dtype), "scale": scale}


def _to_rows(x, position, rows):
    """Row position[t, j] = x[t]; the others 0."""
    flat = position.reshape(-1).long()
    out = torch.zeros(rows + 1, x.shape[1], dtype=x.dtype, device=x.device)
    out[torch.where(flat >= 0, flat, rows)] = x.repeat_interleave(position.shape[1], 0)
    return out[:rows]


def _from_rows(y, position, weights):
    """The sum over j of weights[t, j] y[position[t, j]], in FP32."""
    part = torch.where(position[..., None] >= 0, y[position.long().clamp(min=0)].float(), 0.0)
    return part.sum(1) if weights is None else (part * weights[..., None]).sum(1)


def _plain_dispatch(s):
    offsets, position = _sorted(s["experts"], s["e"])
    out = {"offsets": offsets, "position": position}
    if s["train"]:
        out["y"] = _to_rows(s["x"], position, s["y"].shape[0])
        out["dx"] = _from_rows(s["dy"], position, None).to(s["dx"].dtype)
        return out
    q, scale = _quantized(s["x"].float(), 1, "e4m3")
    scale = _to_rows(scale, position, s["q"].shape[0])
    q = _to_rows(q.float(), position, s["q"].shape[0])
    out["values"], out["scale"] = (q * _spread(scale, 1, *q.shape)).to(s["v"].dtype), scale
    return out


def _plain_combine(s):
    out = {"x": (_from_rows(s["y"], s["position"], s["weights"]) + (0.0 if s["train"] else s["x0"].float())).to(s["x"].dtype)}
    if s["train"]:
        dx, real = s["dx"].float(), s["position"] >= 0
        dy = _to_rows(dx, s["position"], s["dy"].shape[0])
        w = _to_rows(s["weights"].reshape(-1, 1), s["position"].reshape(-1, 1), s["dy"].shape[0])
        out["dy"] = (dy * w).to(s["dy"].dtype)
        y = s["y"][s["position"].long().clamp(min=0)].float()
        out["dw"] = torch.where(real, (y * dx[:, None, :]).sum(2), 0.0)
    return out


def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"product": _plain_product, "experts": _plain_experts, "quantize": _plain_quantize, "dispatch": _plain_dispatch,
                "combine": _plain_combine}[op](s)
    import dense_gemm_09_gb300 as dg

    if op == "product":
        if s["beta"]:
            s["c"].copy_(s["c0"])  # a pass adds to the same gradient each time
        return dg.gemm_f8_tn(s["a"], s["b"], s["c"], s["sa"], s["sb"], bias=s["bias"], beta=s["beta"])
    if op == "experts":
        return dg.gemm_f8_tn_experts(s["a"], s["b"], s["c"], s["sa"], s["sb"], s["offsets"])
    if op == "quantize":
        if s["form"] == "swiglu":
            dg.swiglu_f8(s["x"], s["u"], s["q"], s["scale"])
        else:
            dg.quantize_f8(s["x"], s["q"], s["scale"], transposed=s["form"] == "transposed")
        return {"values": dg.dequantize_f8(s["q"], s["scale"], s["v"]), "scale": s["scale"]}
    if op == "dispatch":
        dg.sort_by_expert(s["experts"], s["offsets"], s["position"])
        out = {"offsets": s["offsets"], "position": s["position"]}
        if s["train"]:
            out["y"] = dg.gather_by_expert(s["x"], s["position"], s["y"])
            out["dx"] = dg.combine_experts(s["dy"], s["position"], None, s["dx"])
        else:
            dg.gather_by_expert_f8(s["x"], s["position"], s["q"], s["scale"])
            out["values"], out["scale"] = dg.dequantize_f8(s["q"], s["scale"], s["v"]), s["scale"]
        return out
    if s["train"]:
        out = {"x": dg.combine_experts(s["y"], s["position"], s["weights"], s["x"])}
        out["dy"], out["dw"] = dg.combine_experts_grad(s["dx"], s["y"], s["position"], s["weights"], s["dy"], s["dw"])
        return out
    s["x"].copy_(s["x0"])  # a pass adds to the same residual stream each time
    return {"x": dg.combine_experts(s["y"], s["position"], s["weights"], s["x"], beta=1.0)}


def _to_step(q, f8):
    """q on the grid of an 8-bit type, ties to even."""
    bits, least = (3, -6) if f8 == "e4m3" else (2, -14)
    step = torch.exp2((torch.frexp(q)[1].double() - 1).clamp(min=least) - bits)
    return (torch.round(q / step) * step).clamp(-TOP[f8], TOP[f8])


def _exact_groups(y, rows, f8):
    """(values, scale) of rows in 64 bits."""
    m, k = y.shape
    z = torch.nn.functional.pad(y, (0, -k % BLOCK, 0, -m % rows))
    z = z.reshape(z.shape[0] // rows, rows, -1, BLOCK).transpose(1, 2)
    top = torch.maximum(z.amax((2, 3)), -z.amin((2, 3)))
    q = _to_step(TOP[f8] * z / torch.where(top > 0, top, 1.0)[:, :, None, None], f8)
    v = (q * (top / TOP[f8])[:, :, None, None]).transpose(1, 2).reshape(z.shape[0] * rows, -1)
    return v[:m, :k], top / TOP[f8]


def exact(case, seed):
    op = case["op"]
    flops = work(case)["flops"]
    if op in ("product", "experts") and flops > 1e13:
        return None  # 64-bit products run at about a teraflop a second
    s = prepare(case, seed)
    if op == "product":
        m, k = s["a"].shape
        a = torch.einsum("mk,mk->mk", s["a"].double(), _spread(s["sa"].double(), 1, m, k))
        b = torch.einsum("nk,nk->nk", s["b"].double(), _spread(s["sb"].double(), s["rows"], s["b"].shape[0], k))
        y = torch.einsum("mk,nk->mn", a, b) + s["beta"] * s["c0"].double()
        return y if s["bias"] is None else y + s["bias"].double()[None, :]
    if op == "experts":
        y = torch.zeros(s["c"].shape, dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                k, n = s["a"].shape[1], s["b"].shape[1]
                a = s["a"][lo:hi].double() * _spread(s["sa"][lo:hi].double(), 1, hi - lo, k)
                y[lo:hi] = a @ (s["b"][e].double() * _spread(s["sb"][e].double(), BLOCK, n, k)).t()
        return y
    if op == "quantize":
        y = s["x"].double()
        if s["form"] == "swiglu":
            y = y * torch.special.expit(y) * s["u"].double()
        elif s["form"] == "transposed":
            y = y.t().contiguous()
        values, scale = _exact_groups(y, BLOCK if s["form"] == "blocks" else 1, case["f8"])
        return {"values": values, "scale": scale}
    if op == "dispatch":
        _, position = _sorted(s["experts"], case["e"])
        rows = case["tokens"] * case["top"]
        out = {"offsets": None, "position": None}
        pairs = position.reshape(-1).long()
        kept = pairs >= 0
        token = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["top"])

        def place(x):
            y = torch.zeros(rows, x.shape[1], dtype=torch.float64, device="cuda")
            y[pairs[kept]] = x.double()[token[kept]]
            return y

        if case["train"]:
            dx = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
            return {**out, "y": place(s["x"]), "dx": dx.index_add_(0, token[kept], s["dy"].double()[pairs[kept]])}
        values, scale = _exact_groups(s["x"].double(), 1, "e4m3")
        return {**out, "values": place(values), "scale": place(scale)}
    pairs = s["position"].reshape(-1).long()
    kept = pairs >= 0
    token = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["top"])[kept]
    w, at = s["weights"].reshape(-1)[kept].double(), pairs[kept]
    x = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda") if case["train"] else s["x0"].double()
    x = x.index_add(0, token, s["y"].double()[at] * w[:, None])
    if not case["train"]:
        return {"x": x}
    dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device="cuda")
    dy[at] = s["dx"].double()[token] * w[:, None]
    dw = torch.zeros(pairs.numel(), dtype=torch.float64, device="cuda")
    dw[kept] = torch.einsum("pk,pk->p", s["dx"].double()[token], s["y"].double()[at])
    return {"x": x, "dy": dy, "dw": dw.view(s["dw"].shape)}


def work(case):
    k = case["k"]
    if case["op"] == "product":
        m, n = case["m"], case["n"]
        c = TYPES[case["out"]].itemsize * m * n * (2 if case["wgrad"] else 1)
        scales = 4 * _blocks(k) * (m + (n if case["wgrad"] else _blocks(n)))
        return {"bytes": (m + n) * k + scales + c + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if case["op"] == "quantize":
        m, e = case["m"], TYPES[case["type"]].itemsize
        each = (2 if case["form"] == "swiglu" else 1) * e + 2  # the rows, the values
        return {"bytes": each * m * k + 4 * m * k // BLOCK, "flops": (9 if case["form"] == "swiglu" else 4) * m * k}
    tokens = case["tokens"] - (case["tokens"] // 4 if case["padded"] else 0)
    rows = tokens * case["top"]
    if case["op"] == "experts":
        e, n = case["e"], case["n"]
        used = e * (1.0 - (1.0 - min(1.0, case["top"] / e)) ** tokens)  # experts with a row, on average
        weights = used * (n * k + 4 * _blocks(n) * _blocks(k))
        return {"bytes": weights + rows * (k + 4 * _blocks(k) + TYPES[case["out"]].itemsize * n), "flops": 2 * rows * n * k}
    e = TYPES[case["type"]].itemsize
    if case["op"] == "dispatch":
        pairs = 8 * case["tokens"] * case["top"]  # ids and positions
        if case["train"]:
            return {"bytes": pairs + 2 * e * (tokens + rows) * k, "flops": rows * k}
        return {"bytes": pairs + e * tokens * k + 2 * rows * k + 4 * rows * _blocks(k), "flops": 4 * tokens * k}
    if case["train"]:  # rows, their gradient, tokens out and their gradient in
        return {"bytes": 2 * e * (tokens + rows) * k, "flops": 5 * rows * k}
    return {"bytes": e * (2 * tokens + rows) * k, "flops": 2 * rows * k}
