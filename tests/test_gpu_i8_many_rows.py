"""The 8-bit row operators on more rows than the GPU runs at once, where a block
takes several rows one after another, against their formulas in float64."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu

# a warp to a row, then blocks of 160 to 1024 threads; 1.1 to 3 rounds of rows
SIZES = [(8003, 1000), (2101, 4104), (1301, 8191), (700, 12300), (401, 16384), (317, 32760)]


def _rows(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    d, _ = ref.pitched(rows, cols, dtype, (-cols) % 8 + 8, 0)
    return d.copy_(torch.randn((rows, cols), generator=g) * scale)


def _out(rows, cols):
    pad = (-cols) % 16 + 16
    q, storage = ref.pitched(rows, cols, torch.int8, pad, 0, fill=77)
    return q, storage, pad, torch.full((rows,), -1.0, device="cuda")


def _check(y, delta, q, storage, pad, s):
    rows, cols = q.shape
    ref.check_rows(y, delta, q.cpu(), s.cpu())
    assert bool((storage[:rows * (cols + pad)].view(rows, cols + pad)[:, cols:] == 77).all())


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(rows, cols, ty):
    import dense_gemm_09_gb300 as dg
    x = _rows(rows, cols, ref.TYPES[ty], 1)
    x[rows - 2] = 0.0
    q, st, pad, s = _out(rows, cols)
    dg.quantize_i8(x, q, s)
    _check(x.cpu().double(), 0.0, q, st, pad, s)
    assert float(s[rows - 2]) == 0.0


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_swiglu(rows, cols, ty):
    import dense_gemm_09_gb300 as dg
    g, u = _rows(rows, cols, ref.TYPES[ty], 2, 2.0), _rows(rows, cols, ref.TYPES[ty], 3)
    q, st, pad, s = _out(rows, cols)
    dg.swiglu_i8(g, u, q, s)
    _check(*ref.swiglu_rows(g.cpu(), u.cpu()), q, st, pad, s)


@pytest.mark.parametrize("f32_gamma", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rmsnorm(rows, cols, residual, f32_gamma):
    import dense_gemm_09_gb300 as dg
    dt = torch.bfloat16
    x = _rows(rows, cols, dt, 4)
    r = _rows(rows, cols, dt, 5, 3.0) if residual else None
    gamma = (1.0 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(6))).cuda()
    gamma = gamma if f32_gamma else gamma.to(dt)
    h, y, delta = ref.norm_rows(x.cpu(), gamma.cpu(), r.cpu() if residual else None, 1e-6)
    q, st, pad, s = _out(rows, cols)
    # H in place of the residual, or of X
    dg.rmsnorm_i8(x, gamma, q, s, residual=r, H=r if residual else x)
    _check(y, delta, q, st, pad, s)
    stored = (r if residual else x).cpu().double()
    assert bool(((stored - h).abs() <= (ref.U[dt] + 2 * ref.E) * h.abs() + ref.TINY[dt]).all())


@pytest.mark.parametrize("rows,cols", SIZES)
def test_rows_that_are_not_finite_mark_themselves_alone(rows, cols):
    import dense_gemm_09_gb300 as dg
    x = _rows(rows, cols, torch.bfloat16, 7)
    x[3, 5], x[rows - 3, cols - 1], x[rows // 2, 0] = float("nan"), float("inf"), float("-inf")
    bad = {3, rows - 3, rows // 2}
    ones = torch.ones(cols, device="cuda", dtype=torch.bfloat16)
    for call in (lambda q, s: dg.quantize_i8(x, q, s), lambda q, s: dg.rmsnorm_i8(x, ones, q, s),
                 lambda q, s: dg.swiglu_i8(x, x, q, s)):
        q, _, _, s = _out(rows, cols)
        call(q, s)
        marked = set(torch.isnan(s).nonzero().flatten().tolist())
        assert marked == bad
        assert all(int(q[i].abs().max()) == 0 for i in bad)
