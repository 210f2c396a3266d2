"""rmsnorm_i8 with eps = 0 (or next to it): rows whose squares leave FP32's range
downwards, and rows of zeros, in every kernel."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu

# binary exponents of a row's values, on both sides of where squares turn
# subnormal (-63), vanish (-75), and values do (-126)
EXPONENTS = [0, -20, -38, -39, -40, -41, -42, -50, -60, -63, -64, -70, -75, -80, -100, -126, -140]
ZERO = len(EXPONENTS)  # the row of zeros after them


def _rows(rows, cols, dtype, seed, pad, offset):
    g = torch.Generator().manual_seed(seed)
    e = torch.tensor([EXPONENTS[i % len(EXPONENTS)] for i in range(rows)], dtype=torch.float64)
    x = torch.randn((rows, cols), generator=g, dtype=torch.float64) * 2.0 ** e[:, None]
    x[:, 0] += 2.0 ** e  # (no row of one column is nearly 0)
    x[ZERO::40] = 0.0
    d, _ = ref.pitched(rows, cols, dtype, pad, offset)
    return d.copy_(x)


def _check(rows, cols, dtype, eps, residual=False, pad=0, offset=0, into_x=False):
    import dense_gemm_09_gb300 as dg
    x = _rows(rows, cols, dtype, cols, pad, offset)
    # the residual halves the rows exactly: h = x - x / 2 keeps their sizes
    r = (x * -0.5) if residual else None
    if residual:
        r2, _ = ref.pitched(rows, cols, dtype, pad, offset)
        r = r2.copy_(r)
    gamma = (1.0 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(dtype).cuda()
    x0, r0 = x.clone(), r.clone() if residual else None
    q, _ = ref.pitched(rows, cols, torch.int8, pad, offset)
    s = torch.full((rows,), -1.0, device="cuda")
    H = x if into_x else None
    dg.rmsnorm_i8(x, gamma, q, s, residual=r, H=H, eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    h, y, delta = ref.norm_rows(x0, gamma, r0, eps)
    zero = (h == 0).all(1)
    assert bool(zero.any()) or rows <= ZERO
    assert bool((s[zero] == 0).all()) and bool((q[zero] == 0).all())
    ref.check_rows(y[~zero], delta, q[~zero], s[~zero])
    if into_x:
        assert bool(((x.double() - h).abs() <= (ref.U[dtype] + 2 * ref.E) * h.abs() + ref.TINY[dtype]).all())


SIZES = [(40, 1), (40, 5), (40, 100), (40, 1000), (40, 4096), (40, 8191), (40, 12300), (20, 33000),
         (2000, 300), (8003, 1000), (1301, 8184), (700, 12304), (317, 32760)]


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_no_eps(rows, cols, ty):
    _check(rows, cols, ref.TYPES[ty], 0.0, pad=(-cols) % 8, into_x=True)
    _check(rows, cols, ref.TYPES[ty], 0.0, residual=True, pad=(-cols) % 8)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-38, 2.0 ** -101])
def test_smallest_eps(eps, ty):
    for rows, cols in ((40, 1000), (40, 12300), (20, 33000), (8003, 1000)):
        _check(rows, cols, ref.TYPES[ty], eps, pad=(-cols) % 8, into_x=True)


def test_unaligned_and_f16():
    for cols in (100, 1000, 9001, 33001):
        _check(40, cols, torch.float32, 0.0, residual=True, pad=3, offset=1, into_x=True)
        import dense_gemm_09_gb300 as dg
        x = torch.randn((3, cols), generator=torch.Generator().manual_seed(1)).half().cuda() * 2.0 ** -10
        x[1] = 0.0
        q, s = torch.empty((3, cols), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
        gamma = torch.ones(cols, dtype=torch.float16, device="cuda")
        dg.rmsnorm_i8(x, gamma, q, s, eps=0.0)
        _, y, delta = ref.norm_rows(x[[0, 2]], gamma, None, 0.0)
        ref.check_rows(y, delta, q[[0, 2]], s[[0, 2]])
        assert float(s[1]) == 0.0 and not bool(q[1].any())


@pytest.mark.parametrize("cols", [100, 4096, 33000])
def test_rows_that_are_not_finite_stay_marked(cols):
    import dense_gemm_09_gb300 as dg
    x = torch.full((4, cols), 2.0 ** -100, device="cuda")
    x[0, cols - 1], x[1, 0], x[2, 5] = float("nan"), float("inf"), float("-inf")
    q, s = torch.empty((4, cols), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    dg.rmsnorm_i8(x, torch.ones(cols, device="cuda"), q, s, eps=0.0)
    assert torch.isnan(s).tolist() == [True, True, True, False]
    assert not bool(q[:3].any()) and bool((q[3] == 127).all())
