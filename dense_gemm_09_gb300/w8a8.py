"""A gated feed-forward layer in 8-bit integers, from this library's calls.

    h += down( silu(gate(n)) * up(n) ),   n = rmsnorm(h)

as an inference program runs it: weights quantised once, a channel at a time;
activations quantised a token at a time where they are made.  Four launches a
layer: norm -> product -> gated activation -> product with the residual's
addition (two quantised matrices and the gate / up rows in between), on
buffers laid out once, so a step can be captured in a CUDA graph.

    python -m dense_gemm_09_gb300.w8a8 [--hidden 4096] [--ffn 12288] [--tokens 1 16 2048]

prints each batch's time eager and as a graph, and the error of the layer's
update against FP32 on the unquantised weights.
"""
from __future__ import annotations

import argparse

import torch

import dense_gemm_09_gb300 as dg


def _rows(n: int, cols: int, dtype, device) -> torch.Tensor:
    """n x cols with rows on 16-byte boundaries (the fast kernels' condition)."""
    step = 16 // dtype.itemsize
    if cols % step == 0:
        return torch.empty((n, cols), dtype=dtype, device=device)
    return torch.empty((n, -(-cols // step) * step), dtype=dtype, device=device)[:, :cols]


def quantize_weights(w: torch.Tensor):
    """Int8 rows and scales of a weight matrix (a row for each output channel)."""
    q = _rows(w.shape[0], w.shape[1], torch.int8, w.device)
    return dg.quantize_i8(w, q, torch.empty(w.shape[0], dtype=torch.float32, device=w.device))


class GatedMlp:
    """The layer, for up to `most` tokens at a time.  gamma: the norm's weights;
    w_gate, w_up: ffn x hidden; w_down: hidden x ffn (float32, float16 or
    bfloat16, as nn.Linear stores them).

    A layer may be called from several streams and threads at once, and replayed
    in graphs beside them: each call's rows are its own, allocated on the
    current stream (in a capture, in the graph's memory) as torch allocates any
    tensor.  q1, t1, gu, q2, t2 are the last call's, to look at."""

    q1 = t1 = gu = q2 = t2 = None

    def __init__(self, gamma, w_gate, w_up, w_down, most: int, dtype=torch.bfloat16, eps: float = 1e-6):
        dev, (ffn, hidden) = w_gate.device, w_gate.shape
        self.gamma, self.eps, self.ffn = gamma.to(dtype), eps, ffn
        # the two projections of the same rows are one product
        self.w1, self.s1 = quantize_weights(torch.cat([w_gate, w_up]))
        self.w2, self.s2 = quantize_weights(w_down)
        self.hidden, self.dtype, self.most = hidden, dtype, most

    def __call__(self, h: torch.Tensor) -> torch.Tensor:
        """h (tokens x hidden, the residual stream) is updated and returned."""
        m, ffn, dev = h.shape[0], self.ffn, h.device
        if m > self.most:
            raise ValueError("%d tokens, the layer was made for %d" % (m, self.most))
        q1, t1 = _rows(m, self.hidden, torch.int8, dev), torch.empty(m, dtype=torch.float32, device=dev)
        dg.rmsnorm_i8(h, self.gamma, q1, t1, eps=self.eps)
        gu = _rows(m, 2 * ffn, self.dtype, dev)
        dg.gemm_i8_tn(q1, self.w1, gu, t1, self.s1)
        q2, t2 = _rows(m, ffn, torch.int8, dev), torch.empty(m, dtype=torch.float32, device=dev)
        dg.swiglu_i8(gu[:, :ffn], gu[:, ffn:], q2, t2)
        dg.gemm_i8_tn(q2, self.w2, h, t2, self.s2, beta=1.0)
        self.q1, self.t1, self.gu, self.q2, self.t2 = q1, t1, gu, q2, t2
        return h


def plain(h, gamma, w_gate, w_up, w_down, eps: float = 1e-6):
    """The layer's update of h, in the inputs' precision, on the unquantised weights."""
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * gamma
    return (torch.nn.functional.silu(n @ w_gate.t()) * (n @ w_up.t())) @ w_down.t()


def _time(f, reps: int = 20) -> float:
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=12288)
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 2048])
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    gamma = 1 + 0.1 * normal(a.hidden)
    w = [normal(a.ffn, a.hidden) / a.hidden ** 0.5 for _ in range(2)] + [normal(a.hidden, a.ffn) / a.ffn ** 0.5]
    layer = GatedMlp(gamma, *w, most=max(a.tokens))
    for m in a.tokens:
        h0 = normal(m, a.hidden).bfloat16()
        h = h0.clone()
        layer(h)
        want = plain(h0.float(), layer.gamma.float(), *w)
        err = ((h.float() - h0.float() - want).norm() / want.norm()).item()
        eager = _time(lambda: layer(h))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(h)
        us = _time(graph.replay)
        print("%5d tokens: eager %8.1f us, graph %8.1f us, %7.1f TFLOP/s, error of the update %.4f"
              % (m, eager, us, 6.0 * m * a.hidden * a.ffn / us / 1e6, err))


if __name__ == "__main__":
    main()
