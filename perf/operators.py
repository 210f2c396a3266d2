"""The 8-bit linear-layer operators as they are measured: their inputs, plain forms, exact forms and work.

Operators (op): "norm" rmsnorm_i8, "swiglu" swiglu_i8, "quantize" quantize_i8 -- each writes int8 rows with one FP32
scale a row -- and "product" gemm_i8_tn, the product of two such matrices.  What is held in 8 bits is returned as the
values it stands for (dequantize_i8, to 16 bits), beside the scales.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token through one projection: the latency of decoding, bound by the weights' bytes
        {"name": "product_1x8192x4096", "op": "product", "m": 1, "n": 8192, "k": 4096, "out": "bf16", "bias": False},
        # a small decoding batch into a projection with a bias
        {"name": "product_16x4096x8192", "op": "product", "m": 16, "n": 4096, "k": 8192, "out": "bf16", "bias": True},
        # a large decoding batch or a short prompt: few rows, a wide projection
        {"name": "product_127x12288x4096", "op": "product", "m": 127, "n": 12288, "k": 4096, "out": "f16", "bias": False},
        # logits of part of a prompt in FP32; every size ragged, rows at a padded pitch
        {"name": "product_1023x8193x4095", "op": "product", "m": 1023, "n": 8193, "k": 4095, "out": "f32", "bias": True},
        # a long prompt: bound by the tensor cores
        {"name": "product_8192x8192x4096", "op": "product", "m": 8192, "n": 8192, "k": 4096, "out": "bf16", "bias": False},
        # the norm before a projection: one token, a ragged batch, a long prompt
        {"name": "norm_1x4096", "op": "norm", "m": 1, "k": 4096, "type": "bf16", "residual": True},
        {"name": "norm_333x8191", "op": "norm", "m": 333, "k": 8191, "type": "f16", "residual": False},
        {"name": "norm_8192x8192", "op": "norm", "m": 8192, "k": 8192, "type": "bf16", "residual": True},
        # the gated activation between the projections of a feed-forward layer: a decoding batch, a long prompt
        {"name": "swiglu_16x12288", "op": "swiglu", "m": 16, "k": 12288, "type": "bf16"},
        {"name": "swiglu_8192x12288", "op": "swiglu", "m": 8192, "k": 12288, "type": "bf16"},
        # the operand of the output projection in a decoding batch; a weight matrix at load, a row for each channel
        {"name": "quantize_127x4096", "op": "quantize", "m": 127, "k": 4096, "type": "f16"},
        {"name": "quantize_8192x8192", "op": "quantize", "m": 8192, "k": 8192, "type": "f32"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row's length: a multiple of 64, as most models have, or any."""
    k = _log(rng, low, high)
    return k if rng.random() < 0.4 else max(64, k // 64 * 64)


def draw(rng):
    op = rng.choice(["product", "product", "product", "norm", "norm", "swiglu", "quantize"])
    if op == "product":
        m, n, k = _log(rng, 1, 8192), _width(rng, 512, 16384), _width(rng, 512, 16384)
        k = max(64, min(k, 8192 * 8192 * 4096 // (m * n)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "f16", "f32"]), "bias": rng.random() < 0.4}
    case = {"op": op, "k": _width(rng, 512, 16384), "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    case["m"] = min(_log(rng, 1, 8192), 8192 * 8192 // case["k"])
    if op == "norm":
        case["residual"] = rng.random() < 0.7
    return case


def _pitched(rows, cols, dtype):
    """A rows x cols matrix whose rows start 16 bytes aligned, as a program lays out rows of any length."""
    step = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, -(-cols // step) * step), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op == "product":
        n, out = case["n"], TYPES[case["out"]]
        # rows as the quantisation leaves them: the largest of some thousand normal values stands at 127
        a, b = _pitched(m, k, torch.int8), _pitched(n, k, torch.int8)
        a.copy_((normal(m, k) * 32).round_().clamp_(-127, 127))
        b.copy_((normal(n, k) * 36).round_().clamp_(-127, 127))
        return {"op": op, "a": a, "b": b, "sa": (0.02 + 0.02 * torch.rand(m, generator=g, device="cuda")),
                "sb": (0.5 + torch.rand(n, generator=g, device="cuda")) / (36 * math.sqrt(k)),
                "bias": normal(n) * 0.1 if case["bias"] else None, "c": _pitched(m, n, out)}
    dtype = TYPES[case["type"]]

    def rows(scale, loud):
        # activations: normal, some channels several times louder than the rest
        x = normal(m, k) * scale
        x[:, torch.rand(k, generator=g, device="cuda") < 0.004] *= loud
        y = _pitched(m, k, dtype)
        return y.copy_(x)

    s = {"op": op, "x": rows(1.0, 6.0), "q": _pitched(m, k, torch.int8), "scale": torch.empty(m, device="cuda"),
         "v": _pitched(m, k, torch.float16 if dtype == torch.float16 else torch.bfloat16)}
    if op == "norm":
        s["gamma"] = (1.0 + 0.1 * normal(k)).to(dtype)
        s["r"] = rows(2.0, 8.0) if case["residual"] else None
        s["h"] = _pitched(m, k, dtype) if case["residual"] else None
    if op == "swiglu":
        s["u"] = rows(1.0, 4.0)
    return s


def _plain_product(s):
    y = (s["a"].float() @ s["b"].float().t()) * s["sa"][:, None] * s["sb"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["c"].dtype)


def _plain_rows(s):
    x = s["x"].float()
    if s["op"] == "norm":
        if s["r"] is not None:
            x = x + s["r"].float()
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
    elif s["op"] == "swiglu":
        y = x / (1.0 + torch.exp(-x)) * s["u"].float()
    else:
        y = x
    scale = y.abs().amax(1) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]).to(torch.int8)
    out = {"values": (q.float() * scale[:, None]).to(s["v"].dtype), "scale": scale}
    if s["op"] == "norm" and s["r"] is not None:
        out["h"] = x.to(s["h"].dtype)
    return out


def run(state):
    s = state
    if not own:
        return _plain_product(s) if s["op"] == "product" else _plain_rows(s)
    import dense_gemm_09_gb300 as dg

    if s["op"] == "product":
        return dg.gemm_i8_tn(s["a"], s["b"], s["c"], s["sa"], s["sb"], bias=s["bias"])
    if s["op"] == "norm":
        dg.rmsnorm_i8(s["x"], s["gamma"], s["q"], s["scale"], residual=s["r"], H=s["h"], eps=EPS)
    elif s["op"] == "swiglu":
        dg.swiglu_i8(s["x"], s["u"], s["q"], s["scale"])
    else:
        dg.quantize_i8(s["x"], s["q"], s["scale"])
    out = {"values": dg.dequantize_i8(s["q"], s["scale"], s["v"]), "scale": s["scale"]}
    if s["op"] == "norm" and s["r"] is not None:
        out["h"] = s["h"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        a, b = s["a"].double(), s["b"].double()
        y = torch.einsum("mk,nk->mn", a, b)  # whole numbers below 2^53: no rounding at all
        y = torch.einsum("mn,m,n->mn", y, s["sa"].double(), s["sb"].double())
        return y if s["bias"] is None else y + s["bias"].double()[None, :]
    h = s["x"].double()
    out = {}
    if case["op"] == "norm":
        if s["r"] is not None:
            h = h + s["r"].double()
            out["h"] = h
        root = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["k"] + EPS).sqrt()
        y = h / root[:, None] * s["gamma"].double()
    elif case["op"] == "swiglu":
        y = h * torch.special.expit(h) * s["u"].double()
    else:
        y = h
    top = torch.maximum(y.amax(1), -y.amin(1))
    steps = torch.round(127.0 * y / torch.where(top > 0, top, 1.0)[:, None])
    out["values"] = steps * (top / 127.0)[:, None]
    out["scale"] = top / 127.0
    return out


def work(case):
    m, k = case["m"], case["k"]
    if case["op"] == "product":
        n = case["n"]
        e = TYPES[case["out"]].itemsize
        return {"bytes": (m + n) * k + 4 * (m + n) + (4 * n if case["bias"] else 0) + e * m * n, "flops": 2 * m * n * k}
    e = TYPES[case["type"]].itemsize
    read = {"norm": 2 if case.get("residual") else 1, "swiglu": 2, "quantize": 1}[case["op"]] * e * m * k
    write = (e * m * k if case.get("residual") else 0) + 2 * m * k + 4 * m  # the residual stream, the values, the scales
    each = {"norm": 8, "swiglu": 9, "quantize": 4}[case["op"]]
    return {"bytes": read + write + (e * k if case["op"] == "norm" else 0), "flops": each * m * k}
