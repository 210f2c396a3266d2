"""A layer called at once on another stream than the one that it was made on, which still has
work before the weights' quantisation."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def first_call(make, call):
    """What the layer gives on another stream as soon as it is made, and later."""
    torch.full((1 << 28,), 0x7F, dtype=torch.uint8, device="cuda")  # (what is laid out lands on other values)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    layer = make()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(layer)
    torch.cuda.synchronize()
    return got, call(layer)


def test_a_mixture_of_experts(dg):
    from dense_gemm_09_gb300.moe import ExpertMlp
    w = [torch.randn(4, *s, device="cuda") / 16 for s in ((256, 384), (256, 384), (384, 256))]
    x = torch.randn(50, 384, device="cuda").bfloat16()
    ids, share = torch.arange(100, device="cuda").view(50, 2) % 4, torch.full((50, 2), 0.5, device="cuda")
    got, want = first_call(lambda: ExpertMlp(*w), lambda layer: layer(x, ids, share, torch.zeros_like(x)))
    assert torch.equal(got, want) and bool(want.isfinite().all()) and bool((want != 0).any())


def test_a_gated_layer(dg):
    from dense_gemm_09_gb300.w8a8 import GatedMlp
    w = [torch.randn(*s, device="cuda") / 16 for s in ((256, 384), (256, 384), (384, 256))]
    h, gamma = torch.randn(50, 384, device="cuda").bfloat16(), torch.ones(384, device="cuda")
    got, want = first_call(lambda: GatedMlp(gamma, *w, most=50), lambda layer: layer(h.clone()))
    assert torch.equal(got, want) and bool(want.isfinite().all()) and bool((want != h).any())
