"""Calls of which one size is 0: what does not depend on it is still written, and nothing else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_no_pairs(dg):
    for shape in ((0, 4), (4, 0)):
        offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
        dg.sort_by_expert(empty(*shape, dtype=torch.int64), offsets, empty(*shape, dtype=torch.int32))
        assert not bool(offsets.any())


@pytest.mark.parametrize("rows", [0, 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_choices(dg, dtype, rows):
    y, position, weights = torch.ones(rows, 300, dtype=dtype, device="cuda"), empty(7, 0, dtype=torch.int32), empty(7, 0)
    x = torch.randn(7, 300, device="cuda").to(dtype)
    want = -0.5 * x
    assert torch.equal(dg.combine_experts(y, position, weights, x, beta=-0.5), want)
    assert not bool(dg.combine_experts(y, position, None, x.fill_(float("nan"))).any())
    assert torch.equal(dg.gather_by_expert(want, position, y), torch.ones_like(y))


def test_no_rows(dg):
    position = torch.tensor([[0, -1], [3, 1]], dtype=torch.int32, device="cuda")
    x, weights, dw = torch.randn(2, 300, device="cuda"), torch.rand(2, 2, device="cuda"), torch.full((2, 2), 9.0, device="cuda")
    y = empty(0, 300)
    dg.gather_by_expert(x, position, y)
    assert not bool(dg.combine_experts(y, position, weights, x.clone()).any())
    dg.combine_experts_grad(x, y, position, weights, y, dw)
    assert not bool(dw.any())


def test_no_columns(dg):
    position = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    dw = torch.full((2, 2), 9.0, device="cuda")
    dg.combine_experts_grad(empty(2, 0), empty(4, 0), position, torch.rand(2, 2, device="cuda"), empty(4, 0), dw)
    assert not bool(dw.any())
    x = empty(2, 0)
    assert dg.combine_experts(empty(4, 0), position, None, x) is x


def test_no_tokens(dg):
    position, weights, dw = empty(0, 2, dtype=torch.int32), empty(0, 2), empty(0, 2)
    y = torch.ones(4, 300, device="cuda")
    dg.gather_by_expert(empty(0, 300), position, y)
    dg.combine_experts_grad(empty(0, 300), y, position, weights, y, dw)
    assert bool((y == 1).all()) and dg.device_status() == dg.OK
