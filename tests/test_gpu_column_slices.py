"""Outputs that are columns of a wider matrix, at rows on 16-byte boundaries, whose last column
lies inside a 16-byte word: the neighbouring columns stay as they were."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES = [(128, 33, 64), (300, 257, 256), (600, 2065, 192), (1100, 1030, 128), (2304, 4099, 64), (127, 4103, 512)]


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def wide(m, n, dtype):
    """(matrix, what lies beside it)."""
    s = torch.full((m, (n + 31) // 16 * 16), 77, device="cuda", dtype=dtype)
    return s[:, :n], s[:, n:]


def padded(t):
    """t at a pitch on 16-byte boundaries."""
    s = torch.zeros(t.shape[0], (t.shape[1] + 15) // 16 * 16, device="cuda", dtype=t.dtype)
    s[:, :t.shape[1]] = t
    return s[:, :t.shape[1]]


def ints(m, n):
    return torch.randint(-4, 5, (m, n), device="cuda").float()


# (small whole numbers: every product and sum is exact in FP32, and rounded once)
@pytest.mark.parametrize("beta", [0.0, 1.0])
@pytest.mark.parametrize("name", ["gemm_f32", "gemm_tf32", "gemm_f16_tn", "gemm_f16_nn", "gemm_bf16_tn", "gemm_bf16_nn"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm(dg, m, n, k, name, beta):
    dtype = torch.float16 if "f16" in name and "bf16" not in name else torch.bfloat16 if "bf16" in name else torch.float32
    a, b = ints(m, k), ints(k, n)
    c, beside = wide(m, n, dtype)
    want = (a.double() @ b.double() + beta * 77).to(dtype)
    operand = padded((b.t() if name.endswith("tn") else b).to(dtype))
    getattr(dg, name)(padded(a.to(dtype)), operand, c, beta=beta)
    assert torch.equal(c, want) and bool((beside == 77).all()), dg.last_kernel()


@pytest.mark.parametrize("beta", [0.0, 1.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_eight_bits(dg, m, n, k, dtype, beta):
    a, b = ints(m, k), ints(n, k)
    want = (a.double() @ b.double().t() + beta * 77).to(dtype)
    c, beside = wide(m, n, dtype)
    dg.gemm_i8_tn(padded(a.to(torch.int8)), padded(b.to(torch.int8)), c, torch.ones(m, device="cuda"), torch.ones(n, device="cuda"), beta=beta)
    assert torch.equal(c, want) and bool((beside == 77).all()), dg.last_kernel()
    f8 = [padded(t.to(torch.float8_e4m3fn).view(torch.uint8)).view(torch.float8_e4m3fn) for t in (a, b)]
    scales = [torch.ones(rows, -(-k // 128), device="cuda") for rows in (m, n)]
    for kernel in (None, (2, 128, 1), (2, 256, 1), (3, 64, 1)):
        c, beside = wide(m, n, dtype)
        if kernel:
            dg.tune_f8_next(*kernel)
        dg.gemm_f8_tn(*f8, c, *scales, beta=beta)
        assert torch.equal(c, want) and bool((beside == 77).all()), dg.last_kernel()


def test_experts(dg):
    a, b = ints(600, 256), ints(3 * 300, 256)
    off = torch.tensor([0, 256, 411, 600], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for n in (257, 299):
            w = b.view(3, 300, 256)[:, :n]
            want = torch.cat([a[o:e].double() @ w[i].double().t() for i, (o, e) in enumerate(((0, 256), (256, 411), (411, 600)))]).to(dtype)
            c, beside = wide(600, n, dtype)
            dg.gemm_f8_tn_experts(a.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), c, torch.ones(600, 2, device="cuda"),
                                  torch.ones(3, n, 2, device="cuda"), off)
            assert torch.equal(c, want) and bool((beside == 77).all()), dg.last_kernel()
