"""A mixture-of-experts feed-forward layer in 8-bit floating point, from this library's calls.

    h[t] += sum_j weight[t, j] * down_e( silu(gate_e(x[t])) * up_e(x[t]) ),   e = expert[t, j]

as an inference program runs it: weights quantised once, in blocks of 128 x 128; activations
with a scale for each 128 values, where they are made.  Six launches a layer: the pairs
(token, expert) are sorted, tokens quantised on their way to their rows, multiplied by each
expert's gate and up projections, gated, multiplied by its down projection, and brought back
with the router's weights; on buffers laid out once, so a step can be captured in a CUDA graph.

    python -m dense_gemm_09_gb300.moe [--hidden 4096] [--ffn 2048] [--experts 64] [--top 8] [--tokens 1 16 2048]

prints each batch's time eager and as a graph, and the error of the layer's update against FP32
on the unquantised weights.
"""
from __future__ import annotations

import argparse

import torch

import dense_gemm_09_gb300 as dg
from dense_gemm_09_gb300.w8a8 import _rows, _settle, _time

F8 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return -(-n // 128)


def quantize_experts(w: torch.Tensor):
    """(Q, scale) of weights (experts x out x in), a scale for each 128 x 128 of them."""
    e, n, k = w.shape
    q = torch.empty((e, n, -(-k // 16) * 16), dtype=F8, device=w.device)[:, :, :k]  # rows on 16-byte boundaries
    scale = torch.empty((e, _blocks(n), _blocks(k)), dtype=torch.float32, device=w.device)
    for i in range(e):
        dg.quantize_f8(w[i], q[i], scale[i])
    return q, scale


class ExpertMlp:
    """The layer.  w_gate, w_up: experts x ffn x hidden; w_down: experts x hidden x ffn (float32,
    float16 or bfloat16).

    Like GatedMlp it may be called from several streams and threads at once, and replayed in
    graphs beside them: each call's rows are its own, allocated on the current stream.  The
    weights are laid out when the constructor returns (made in a capture, the layer belongs to
    that graph's stream)."""

    def __init__(self, w_gate, w_up, w_down, dtype=torch.bfloat16):
        self.experts, self.ffn, self.hidden = w_gate.shape
        # the two projections of the same rows are one product
        self.w1, self.s1 = quantize_experts(torch.cat([w_gate, w_up], 1))
        self.w2, self.s2 = quantize_experts(w_down)
        self.dtype = dtype
        _settle(w_gate.device)  # the first call may come on any stream

    def __call__(self, x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, h: torch.Tensor) -> torch.Tensor:
        """h (tokens x hidden, the residual stream) is updated and returned.  x: the tokens, normed;
        experts (int32 or int64), weights (float32): tokens x top, an expert out of range (padding)
        adds nothing."""
        rows, dev = experts.numel(), x.device
        offsets = torch.empty(self.experts + 1, dtype=torch.int32, device=dev)
        position = torch.empty(experts.shape, dtype=torch.int32, device=dev)
        dg.sort_by_expert(experts, offsets, position)
        q1, t1 = _rows(rows, self.hidden, F8, dev), torch.empty((rows, _blocks(self.hidden)), dtype=torch.float32, device=dev)
        dg.gather_by_expert_f8(x, position, q1, t1)
        gu = _rows(rows, 2 * self.ffn, self.dtype, dev)
        dg.gemm_f8_tn_experts(q1, self.w1, gu, t1, self.s1, offsets)
        q2, t2 = _rows(rows, self.ffn, F8, dev), torch.empty((rows, _blocks(self.ffn)), dtype=torch.float32, device=dev)
        dg.swiglu_f8(gu[:, :self.ffn], gu[:, self.ffn:], q2, t2)  # (rows of no expert: whatever they hold)
        y = _rows(rows, self.hidden, self.dtype, dev)
        dg.gemm_f8_tn_experts(q2, self.w2, y, t2, self.s2, offsets)
        return dg.combine_experts(y, position, weights, h, beta=1.0)


def plain(x, experts, weights, w_gate, w_up, w_down):
    """The layer's update of h, in the inputs' precision, on the unquantised weights."""
    out = torch.zeros_like(x)
    for e in range(w_gate.shape[0]):
        token, choice = torch.nonzero(experts == e, as_tuple=True)
        y = (torch.nn.functional.silu(x[token] @ w_gate[e].t()) * (x[token] @ w_up[e].t())) @ w_down[e].t()
        out.index_add_(0, token, y * weights[token, choice][:, None].to(y.dtype))
    return out


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top", type=int, default=8)
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 2048])
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    w = [normal(a.experts, a.ffn, a.hidden) / a.hidden ** 0.5 for _ in range(2)]
    w.append(normal(a.experts, a.hidden, a.ffn) / a.ffn ** 0.5)
    layer = ExpertMlp(*w)
    for m in a.tokens:
        x = normal(m, a.hidden).bfloat16()
        best, experts = torch.topk(normal(m, a.experts), a.top, dim=1)
        weights = torch.softmax(best, 1)
        h = torch.zeros_like(x)
        layer(x, experts, weights, h)
        want = plain(x.float(), experts, weights, *w)
        err = ((h.float() - want).norm() / want.norm()).item()
        eager = _time(lambda: layer(x, experts, weights, h))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(x, experts, weights, h)
        us = _time(graph.replay)
        print("%5d tokens: eager %8.1f us, graph %8.1f us, %7.1f TFLOP/s, error of the update %.4f"
              % (m, eager, us, 6.0 * m * a.top * a.hidden * a.ffn / us / 1e6, err))


if __name__ == "__main__":
    main()
