"""gemm_f8_tn_experts on as many rows as a call may have: an expert's last tile then ends past
2^31, wherever the expert begins."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


@pytest.mark.parametrize("begin", [0, 2 ** 31 - 100], ids=["all rows", "the last rows"])
def test_the_last_tile_ends_past_2_31(dg, begin):
    m = 2 ** 31 - 1
    a = (torch.arange(7, device="cuda", dtype=torch.uint8) + 0x38).repeat(m // 7 + 1)[:m].view(E4M3)[:, None]  # 1, 1.125 .. 1.75
    b = torch.tensor([2.0, 4.0], device="cuda").to(E4M3).view(2, 1, 1)
    one = torch.ones(1, 1, device="cuda")
    c = torch.full((m, 1), 5.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([begin, m - 40, m], dtype=torch.int32, device="cuda")
    dg.gemm_f8_tn_experts(a, b, c, one.expand(m, 1), one.expand(2, 1, 1), offsets)
    assert "any" in dg.last_kernel() and dg.device_status() == dg.OK
    step = 1 << 28
    for lo in range(0, m, step):
        rows = torch.arange(lo, min(lo + step, m), device="cuda")
        want = a[lo:lo + step, 0].to(torch.bfloat16) * torch.where(rows < m - 40, 2, 4).to(torch.bfloat16)
        want = torch.where(rows < begin, 5.0, want)
        assert torch.equal(c[lo:lo + step, 0], want)


@pytest.mark.parametrize("kernel", [None, (1, 0, 1), (2, 128, 1), (2, 256, 1), (3, 64, 1)], ids=str)
def test_the_most_rows_of_the_tensor_cores(dg, kernel):
    m, k = 2 ** 31 - 1 - 512, 16
    a = torch.empty(m, k, dtype=torch.uint8, device="cuda")  # 34 GB, of which the last rows are used
    a[-64:] = torch.arange(64, device="cuda", dtype=torch.uint8)[:, None] % 7 + 0x38
    b = torch.tensor([2.0, 4.0], device="cuda").to(E4M3).view(2, 1, 1).expand(2, 1, k).contiguous()
    one = torch.ones(1, 1, device="cuda")
    c = torch.full((m, 1), 5.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([m - 40, m - 17, m], dtype=torch.int32, device="cuda")
    if kernel:
        dg.tune_f8_next(*kernel)
    dg.gemm_f8_tn_experts(a.view(E4M3), b, c, one.expand(m, 1), one.expand(2, 1, 1), offsets)
    assert dg.device_status() == dg.OK
    assert kernel is None or ("any" in dg.last_kernel()) == (kernel[0] == 1)
    want = a[-64:].view(E4M3).float().sum(1) * torch.where(torch.arange(64, device="cuda") < 47, 2.0, 4.0)
    assert torch.equal(c[-40:, 0].float(), want[-40:])
    assert bool((c[:-40] == 5).all())
