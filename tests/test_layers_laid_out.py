"""The layers' weights are laid out when a constructor returns, so that a first call may come on
any stream.  (No GPU: the library's calls and the streams are stood in for.)"""
import pytest
import torch


def test_waits_for_the_current_stream(monkeypatch):
    from dense_gemm_09_gb300 import w8a8
    done, capturing = [], [False]

    class Stream:
        def __init__(self, device):
            self.device = device

        def synchronize(self):
            done.append(self.device)

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    w8a8._settle(torch.device("cuda", 1))
    assert done == [torch.device("cuda", 1)]
    w8a8._settle(torch.device("cpu"))
    capturing[0] = True  # (a wait would end the capture with an error)
    w8a8._settle(torch.device("cuda", 1))
    assert len(done) == 1


def weights(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(1))


@pytest.fixture
def calls(monkeypatch):
    """The names of the calls that lay a layer out, and of the wait, in their order."""
    import dense_gemm_09_gb300 as dg
    from dense_gemm_09_gb300 import moe, w8a8
    names = []
    for name in ("quantize_i8", "quantize_f8"):
        monkeypatch.setattr(dg, name, lambda x, q, scale, *a, name=name, **k: names.append(name) or (q, scale))
    for module in (w8a8, moe):
        monkeypatch.setattr(module, "_settle", lambda device: names.append("settle " + device.type))
    return names


def test_a_mixture_of_experts(calls):
    from dense_gemm_09_gb300.moe import ExpertMlp
    ExpertMlp(weights(3, 40, 24), weights(3, 40, 24), weights(3, 24, 40))
    assert calls == 6 * ["quantize_f8"] + ["settle cpu"]


def test_a_gated_layer(calls):
    from dense_gemm_09_gb300.w8a8 import GatedMlp
    GatedMlp(torch.ones(24), weights(40, 24), weights(40, 24), weights(24, 40), most=4)
    assert calls == 2 * ["quantize_i8"] + ["settle cpu"]
