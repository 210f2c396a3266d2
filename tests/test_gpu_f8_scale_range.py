"""Scales whose product with each other is out of FP32's normal range, of sums that bring the
result back into it.  The CTA pairs multiply the scales of weights in bands with each other
first, and so take products within that range; the other kernels give all of them.  Rows and
bands out of the range change no others."""
import pytest
import torch

from tests import f8_reference as ref
from tests.test_gpu_f8_gemm import KERNELS, held, tune

pytestmark = pytest.mark.gpu

# (of A, of B, the values' products): products of ~2^-140 (denormal) and ~2^-145 * 1.1 (0 or
# denormal), of sums around 2^22; of ~2^130 (infinite), of sums around 2^-8; and of 2^-126 and
# 2^127, just in the range
OUT = {"denormal": (1.37 * 2.0 ** -80, 1.61 * 2.0 ** -60, 1.0), "zero": (1.37 * 2.0 ** -81, 1.61 * 2.0 ** -64, 1.0),
       "infinite": (1.37 * 2.0 ** 70, 1.61 * 2.0 ** 60, 2.0 ** -16)}
IN = {"least": (2.0 ** -66, 2.0 ** -60, 1.0), "most": (2.0 ** 67, 2.0 ** 60, 2.0 ** -14)}
SCALES = {**OUT, **IN}


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def check(c, a, sa, b, sb, rb, rows=slice(None)):
    # in float64, on scales brought near 1 by powers of two
    up = [2.0 ** -torch.frexp(s.abs().max())[1].item() for s in (sa, sb)]
    want, mag = ref.product(a, sa.double() * up[0], 1, b, sb.double() * up[1], rb)
    tol = ref.product_error(a.shape[1]) * mag
    # denormal results are rounded to a multiple of 2^-149, and so is each block's term
    tol = tol + ref.U[torch.float32] * want.abs() + 2.0 ** -150 * up[0] * up[1] * (ref.blocks(a.shape[1]) + 1)
    err = (c.double() * up[0] * up[1] - want).abs()
    assert bool((err <= tol)[rows].all()), (err / tol)[rows].max().item()


def operands(m, n, k, name, rb, others):
    """Values of one size and sign, so that sums are of the size that the scales want; `others`: some
    rows and bands have other scales, or 0."""
    x, y, small = SCALES[name]
    g = torch.Generator(device="cuda").manual_seed(k)
    a, b = ((torch.rand(r, k, generator=g, device="cuda") + 1) * (256 if small == 1 else small ** 0.5) for r in (m, n))
    sa, sb = torch.full((m, ref.blocks(k)), x, device="cuda"), torch.full((-(-n // rb), ref.blocks(k)), y, device="cuda")
    if others:
        sa[::3] *= 1.25
        sa[1::7] = 0.0
        sb[1::2, ::2] = 0.0
    return a.to(torch.float8_e5m2), sa, b.to(torch.float8_e5m2), sb


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("name", SCALES)
@pytest.mark.parametrize("others", [False, True])
@pytest.mark.parametrize("m,n,k", [(6, 300, 400), (300, 520, 1300)])
def test_products(dg, m, n, k, others, name, kernel):
    for rb in (1, 128):
        a, sa, b, sb = operands(m, n, k, name, rb, others)
        c = torch.empty(m, n, device="cuda")
        tune(dg, kernel)
        dg.gemm_f8_tn(held(a), held(b), c, sa, sb)
        if name in IN or rb == 1 or "pair" not in dg.last_kernel():
            check(c, a, sa, b, sb, rb)


@pytest.mark.parametrize("kernel", [(2, 128, 1), (2, 256, 1)], ids=str)
@pytest.mark.parametrize("name", OUT)
def test_rows_out_of_the_range_change_no_others(dg, name, kernel):
    a, sa, b, sb = operands(300, 512, 640, name, 128, False)
    fine = torch.arange(300, device="cuda") % 5 != 2
    sa[fine] = 2.0 ** -torch.frexp(sb[0, 0])[1].item()
    c = torch.empty(300, 512, device="cuda")
    dg.tune_f8_next(*kernel)
    dg.gemm_f8_tn(a, b, c, sa, sb)
    check(c[fine], a[fine], sa[fine], b, sb, 128)
