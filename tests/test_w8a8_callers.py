"""GatedMlp called by several callers at once: each call's rows are its own.

No GPU: the library's calls are stood in for by plain torch on the CPU, and two
threads take turns call by call, as two streams may."""
import threading

import pytest
import torch


def _quantize(y, Q, scale):
    a = y.abs().amax(1)
    scale.copy_(a / 127)
    Q.copy_(torch.round(127 * y / torch.where(a > 0, a, 1.0)[:, None]))
    return Q, scale


@pytest.fixture
def turns(monkeypatch):
    """Stand-ins for the calls; each waits until the other thread has made its
    own, once `turns.barrier` is set."""
    import dense_gemm_09_gb300 as dg

    class Turns:
        barrier = None

    def turn(f):
        def call(*a, **k):
            if Turns.barrier is not None:
                Turns.barrier.wait(timeout=60)
            out = f(*a, **k)
            if Turns.barrier is not None:
                Turns.barrier.wait(timeout=60)
            return out
        return call

    def norm(X, gamma, Q, scale, residual=None, H=None, eps=1e-6):
        x = X.float()
        return _quantize(x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * gamma.float(), Q, scale)

    def swiglu(G, U, Q, scale):
        return _quantize(torch.nn.functional.silu(G.float()) * U.float(), Q, scale)

    def gemm(A, B, C, sa, sb, bias=None, beta=0.0):
        y = (A.float() @ B.float().t()) * sa[:, None] * sb
        return C.copy_(y + beta * C.float() if beta else y)

    monkeypatch.setattr(dg, "quantize_i8", lambda X, Q, scale: _quantize(X.float(), Q, scale))
    monkeypatch.setattr(dg, "rmsnorm_i8", turn(norm))
    monkeypatch.setattr(dg, "swiglu_i8", turn(swiglu))
    monkeypatch.setattr(dg, "gemm_i8_tn", turn(gemm))
    return Turns


def _layer(most=8):
    from dense_gemm_09_gb300 import w8a8
    g = torch.Generator().manual_seed(1)
    w = [torch.randn(s, generator=g) / 4 for s in ((40, 24), (40, 24), (24, 40))]
    return w8a8.GatedMlp(torch.ones(24), *w, most=most, dtype=torch.float32), g


@pytest.mark.parametrize("sizes", [(5, 5), (3, 8), (8, 1)])
def test_two_callers_in_turn(turns, sizes):
    layer, g = _layer()
    hs = [torch.randn((m, 24), generator=g) for m in sizes]
    alone = [layer(h.clone()) for h in hs]
    turns.barrier = threading.Barrier(2)
    got = [h.clone() for h in hs]
    threads = [threading.Thread(target=layer, args=(h,)) for h in got]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, alone):
        assert torch.equal(a, b)


def test_more_tokens_than_laid_out_for(turns):
    layer, g = _layer(most=4)
    layer(torch.randn((4, 24), generator=g))
    with pytest.raises(ValueError):
        layer(torch.randn((5, 24), generator=g))
