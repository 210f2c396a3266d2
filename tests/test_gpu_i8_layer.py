"""The 8-bit calls together: the gated feed-forward layer of w8a8.py."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu


def _weights(hidden, ffn, seed):
    g = torch.Generator().manual_seed(seed)
    gamma = 1 + 0.1 * torch.randn(hidden, generator=g)
    w = [torch.randn((ffn, hidden), generator=g) / hidden ** 0.5 for _ in range(2)]
    return gamma, w + [torch.randn((hidden, ffn), generator=g) / ffn ** 0.5], torch.randn((300, hidden), generator=g)


def _exact(layer, h, m):
    """The layer's new h in float64 from the device's own quantised weights and
    activations: what the two products and the residual's addition make of them."""
    q2, t2 = layer.q2[:m].cpu().double(), layer.t2[:m].cpu().double()
    w2, s2 = layer.w2.cpu().double(), layer.s2.cpu().double()
    return h.double() + (q2 * t2[:, None]) @ (w2 * s2[:, None]).t()


@pytest.mark.parametrize("hidden,ffn", [(512, 1024), (1000, 2056), (257, 515)])
@pytest.mark.parametrize("m", [1, 3, 12, 100, 300])
def test_layer(hidden, ffn, m):
    from dense_gemm_09_gb300 import w8a8
    gamma, w, h0 = _weights(hidden, ffn, hidden + m)
    h0 = h0[:m].bfloat16()
    layer = w8a8.GatedMlp(gamma.cuda(), *[x.cuda() for x in w], most=300)
    h = w8a8._rows(m, hidden, torch.bfloat16, "cuda")
    h.copy_(h0)
    assert layer(h) is h
    # the quantised norm, gate / up rows and gated rows are each the formula's
    _, y, delta = ref.norm_rows(h0, layer.gamma.cpu(), None, 1e-6)
    ref.check_rows(y, delta, layer.q1[:m].cpu(), layer.t1[:m].cpu())
    gu, mag = ref.product(layer.q1[:m].cpu(), layer.w1.cpu(), layer.t1[:m].cpu(), layer.s1.cpu())
    ref.check_product(layer.gu[:m].cpu(), gu, mag)  # (K <= 1024: exact sums)
    got = layer.gu[:m].cpu()
    y, delta = ref.swiglu_rows(got[:, :ffn], got[:, ffn:])
    ref.check_rows(y, delta, layer.q2[:m].cpu(), layer.t2[:m].cpu())
    want = _exact(layer, h0, m)
    # FP32 sums of <= 2056 products, the scales, the addition, one rounding to bf16
    off = (h.cpu().double() - want).abs()
    assert bool((off <= ref.U[torch.bfloat16] * want.abs() + 300 * ref.E * (want.abs() + h0.double().abs() + 1)).all())
    # 8 bits a value: each of the three quantisations leaves ~1/2 % (rms) of a
    # normal row of this length (a step is max / 127, ~3.5 rms / 127, off by up
    # to a half: 0.8 %), and the products average over K
    full = w8a8.plain(h0.double(), layer.gamma.cpu().double(), *[x.double() for x in w])
    rel = ((want - h0.double() - full).norm() / full.norm()).item()
    assert rel < 0.05, rel


def test_layer_in_a_graph():
    from dense_gemm_09_gb300 import w8a8
    gamma, w, h0 = _weights(512, 1024, 9)
    layer = w8a8.GatedMlp(gamma.cuda(), *[x.cuda() for x in w], most=300)
    for m in (1, 40, 300):
        start = h0[:m].bfloat16().cuda()
        want = layer(start.clone())
        h = start.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(h)
        for _ in range(3):
            h.copy_(start)
            graph.replay()
            assert torch.equal(h, want)


def test_calls_follow_the_stream():
    # launches start beside the previous kernel's end: a chain in which each
    # call reads what the one before it wrote, many times over, and torch
    # kernels between them
    import dense_gemm_09_gb300 as dg
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((64, 2048), generator=g, device="cuda").bfloat16()
    w = (torch.randn((2048, 2048), generator=g, device="cuda") * 40).round().clamp(-127, 127).to(torch.int8)
    s = torch.full((2048,), 1 / (127 * 40 * 2048 ** 0.5) * 30, device="cuda")

    def chain(sync):
        h, q, t = x.clone(), torch.empty((64, 2048), dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")
        one = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
        for i in range(60):
            n = (64, 1, 7, 30)[i % 4]
            dg.rmsnorm_i8(h[:n], one, q[:n], t[:n])
            sync()
            dg.gemm_i8_tn(q[:n], w, h[:n], t[:n], s, beta=0.5)
            sync()
            if i % 5 == 0:
                h.mul_(0.5)
                sync()
            dg.quantize_i8(h, q, t)
            sync()
            dg.dequantize_i8(q, t, h)
            sync()
        return h

    a = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert torch.equal(chain(lambda: None), a)
