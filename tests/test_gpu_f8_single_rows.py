"""gemm_f8_tn and gemm_f8_tn_experts on operands of one row: the pitch of a single row is never
used, so a contiguous one of any length takes the kernels for rows on 16-byte boundaries; and
what lies behind a row's last value (here NaNs) is not part of it."""
import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def row(q):
    """A contiguous row with NaNs behind it."""
    k = q.shape[1]
    y = torch.full((k + 64,), 0x7F, dtype=torch.uint8, device="cuda")[:k].view(1, k)
    y.copy_(q.view(torch.uint8))
    return y.view(q.dtype)


def rows(q):
    """Rows on 16-byte boundaries with NaNs in between."""
    m, k = q.shape
    y = torch.full((m, -(-k // 16) * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda")[:, :k]
    y.copy_(q.view(torch.uint8))
    return y.view(q.dtype)


def close(c, a, sa, b, sb, rb):
    want, mag = ref.product(a, sa, 1, b, sb, rb)
    return bool(((c.double() - want).abs() <= (ref.product_error(a.shape[1]) + ref.E) * mag).all())


K = [1, 15, 17, 100, 130, 1000, 4101]


@pytest.mark.parametrize("kernel", [None, (4, 0, 4), (4, 0, 8), (3, 16, 1), (2, 128, 1)], ids=str)
@pytest.mark.parametrize("k", K)
@pytest.mark.parametrize("m,n", [(1, 700), (1, 1), (7, 1), (300, 1)])
def test_one_row(dg, m, n, k, kernel):
    g = torch.Generator(device="cuda").manual_seed(k)
    rb = 128 if n > 1 else 1
    a, sa = ref.operand(m, k, 1, torch.float8_e4m3fn, g)
    b, sb = ref.operand(n, k, rb, torch.float8_e4m3fn, g)
    c = torch.empty(m, n, device="cuda")
    if kernel:
        dg.tune_f8_next(*kernel)
    dg.gemm_f8_tn((row if m == 1 else rows)(a), (row if n == 1 else rows)(b), c, sa, sb)
    assert "any" not in dg.last_kernel() and close(c, a, sa, b, sb, rb)
    assert dg.device_status() == dg.OK


@pytest.mark.parametrize("k", K)
def test_one_row_by_expert(dg, k):
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa = ref.operand(1, k, 1, torch.float8_e4m3fn, g)
    b, sb = ref.operand(2 * 130, k, 1, torch.float8_e4m3fn, g)
    held = rows(b)
    step = held.stride(0)
    c = torch.empty(1, 130, device="cuda")
    dg.gemm_f8_tn_experts(row(a), held.as_strided((2, 130, k), (130 * step, step, 1)), c, sa, sb.view(2, 130, -1),
                          torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"))
    assert "any" not in dg.last_kernel() and close(c, a, sa, b[130:], sb[130:], 1)
    # experts of one channel, at 16-byte boundaries from each other
    m = 50
    a, sa = ref.operand(m, k, 1, torch.float8_e4m3fn, g)
    b, sb = ref.operand(2, k, 1, torch.float8_e4m3fn, g)
    held = rows(b)
    c = torch.empty(m, 1, device="cuda")
    dg.gemm_f8_tn_experts(rows(a), held.as_strided((2, 1, k), (step, k, 1)), c, sa, sb.view(2, 1, -1),
                          torch.tensor([0, 30, m], dtype=torch.int32, device="cuda"))
    assert "any" not in dg.last_kernel()
    assert close(c[:30], a[:30], sa[:30], b[:1], sb[:1], 1) and close(c[30:], a[30:], sa[30:], b[1:], sb[1:], 1)
