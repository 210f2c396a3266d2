"""One GatedMlp on several streams, in several threads and in graphs at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _layer(hidden=1024, ffn=2048):
    from dense_gemm_09_gb300 import w8a8
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [torch.randn(s, generator=g, device="cuda") / s[1] ** 0.5 for s in ((ffn, hidden), (ffn, hidden), (hidden, ffn))]
    layer = w8a8.GatedMlp(torch.ones(hidden, device="cuda"), *w, most=512)
    hs = [torch.randn((m, hidden), generator=g, device="cuda").bfloat16() for m in (300, 512, 64, 1, 300)]
    return layer, hs


def _steps(layer, h, n=12):
    for _ in range(n):
        layer(h)
        h.mul_(0.75)  # (keeps the stream's size)
    return h


def test_streams_threads_and_a_graph():
    layer, hs = _layer()
    want = [_steps(layer, h.clone()) for h in hs]
    captured = hs[4].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _steps(layer, captured)
    for _ in range(3):
        got = [h.clone() for h in hs[:4]]
        captured.copy_(hs[4])
        streams = [torch.cuda.Stream() for _ in range(5)]
        torch.cuda.synchronize()

        def work(h, s):
            with torch.cuda.stream(s):
                _steps(layer, h)

        threads = [threading.Thread(target=work, args=a) for a in zip(got, streams)]
        for t in threads:
            t.start()
        with torch.cuda.stream(streams[4]):
            graph.replay()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for a, b in zip(got + [captured], want):
            assert torch.equal(a, b)


def test_streams_from_one_thread():
    layer, hs = _layer()
    want = [_steps(layer, h.clone()) for h in hs]
    got = [h.clone() for h in hs]
    streams = [torch.cuda.Stream() for _ in hs]
    torch.cuda.synchronize()
    for _ in range(12):  # one step of each stream in turn
        for h, s in zip(got, streams):
            with torch.cuda.stream(s):
                _steps(layer, h, 1)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rows_of_the_last_call():
    layer, hs = _layer()
    assert layer.q1 is None
    layer(hs[2])
    assert layer.q1.shape == (64, 1024) and layer.gu.shape == (64, 4096) and layer.t2.shape == (64,)
    with pytest.raises(ValueError):
        layer(torch.zeros((513, 1024), dtype=torch.bfloat16, device="cuda"))
