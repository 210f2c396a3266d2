"""The input gradient of gemm_f8_tn_experts: the same call on each expert's transposed weights,
whose 128 x 128 scales transpose with them, as a view."""
import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


@pytest.mark.parametrize("kernel", [None, (1, 0, 1), (2, 128, 1), (2, 256, 1), (3, 16, 1), (3, 64, 1)], ids=str)
@pytest.mark.parametrize("n,k", [(256, 384), (130, 200), (700, 1000)])
@pytest.mark.parametrize("f8", ref.F8)
def test_input_gradient(dg, f8, n, k, kernel):
    e, offsets = 4, [0, 40, 40, 171, 300]
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randn(e, n, k, generator=g, device="cuda") / k ** 0.5
    q, s = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(e, ref.blocks(n), ref.blocks(k), device="cuda")
    for i in range(e):
        dg.quantize_f8(w[i], q[i], s[i])
    dy = torch.randn(300, n, generator=g, device="cuda")
    qd, sd = torch.empty(300, -(-n // 16) * 16, dtype=ref.F8[f8], device="cuda")[:, :n], torch.empty(300, ref.blocks(n), device="cuda")
    dg.quantize_f8(dy, qd, sd)
    back = torch.zeros(e, k, -(-n // 16) * 16, dtype=torch.uint8, device="cuda")[:, :, :n]
    back.copy_(q.view(torch.uint8).transpose(1, 2))
    dx = torch.full((320, k), 5.0, device="cuda")
    if kernel:
        dg.tune_f8_next(*kernel)
    dg.gemm_f8_tn_experts(qd, back.view(q.dtype), dx[:300], sd, s.transpose(1, 2), torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert bool((dx[300:] == 5).all()) and dg.device_status() == dg.OK
    # <dX, T> is the derivative of <dY, X W^T> along T, in float64 on the values held
    values = qd.double() * ref.spread(sd.double(), 1, 300, n)
    t = torch.randn(300, k, generator=g, device="cuda").double()
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if lo == hi:
            continue
        wi = q[i].double() * ref.spread(s[i].double(), 128, n, k)
        want, mag = values[lo:hi] @ wi, values[lo:hi].abs() @ wi.abs()
        tol = (ref.product_error(n) + ref.E) * mag
        assert bool(((dx[lo:hi].double() - want).abs() <= tol).all())
        along = (values[lo:hi] * (t[lo:hi] @ wi.t())).sum()
        assert abs((dx[lo:hi].double() * t[lo:hi]).sum() - along) <= (tol * t[lo:hi].abs()).sum()
