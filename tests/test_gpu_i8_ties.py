"""The steps of quantize_i8 against their definition, value by value:
q = rint(127 y / a), ties to even, a the row's largest |y|.

In float64 127 y is exact, and the quotient of an FP32 (FP16, BF16) row is a tie
(a whole number and a half) exactly where its rounded value is one: other
quotients are at least 2^-33 (relative) away from a tie, and float64 rounds by
2^-53.  So the steps are compared for equality, the scale with a / 127 rounded
once."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu


def _check(x, pad=0, offset=0):
    import dense_gemm_09_gb300 as dg
    rows, cols = x.shape
    q, _ = ref.pitched(rows, cols, torch.int8, pad, offset)
    s = torch.empty(rows, device="cuda")
    dg.quantize_i8(x, q, s)
    y = x.double()
    a = y.abs().amax(1)
    want = torch.round(127.0 * y / a[:, None])
    off = q.double() != want
    assert int(off.sum()) == 0, "%d of %d steps, first at %s" % (int(off.sum()), off.numel(), off.nonzero()[0].tolist())
    assert torch.equal(s, (a / 127.0).float())


def _near_ties(dtype, rows, cols, seed, exponent=0):
    """rows x cols values: a row's largest is random (or 127 times a whole
    number, whose ties all exist in the type), the others are the values of
    the type nearest to its ties, of either sign, with their neighbours."""
    g = torch.Generator().manual_seed(seed)
    a = (1.0 + torch.rand(rows, generator=g, dtype=torch.float64)).to(dtype).double()
    a[::3] = 127.0 / 128.0 * (1 + torch.randint(0, 2 if dtype == torch.bfloat16 else 8, a[::3].shape, generator=g))
    m = torch.randint(0, 127, (rows, cols), generator=g)
    y = ((m + 0.5) * a[:, None] / 127.0).to(dtype)
    bits = y.view(torch.int32 if dtype == torch.float32 else torch.int16)
    bits += torch.randint(-1, 2, bits.shape, generator=g).to(bits.dtype)
    y = y.double().clamp(max=a[:, None]) * (1 - 2 * torch.randint(0, 2, y.shape, generator=g))
    y[:, cols // 2] = a
    return (y * 2.0 ** exponent).to(dtype)


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("rows,cols", [(5, 9), (40, 255), (40, 512), (40, 1000), (40, 4096), (9, 9001), (3, 33000)])
def test_near_ties(rows, cols, ty, pad, offset):
    x, _ = ref.pitched(rows, cols, ref.TYPES[ty], pad, offset)
    _check(x.copy_(_near_ties(ref.TYPES[ty], rows, cols, cols)), pad, offset)


# more rows than run at once
@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("rows,cols", [(8003, 1000), (1301, 8191), (700, 12300), (317, 32760)])
def test_near_ties_in_many_rows(rows, cols, ty):
    pad = (-cols) % 16
    x, _ = ref.pitched(rows, cols, ref.TYPES[ty], pad)
    _check(x.copy_(_near_ties(ref.TYPES[ty], rows, cols, cols)), pad)


@pytest.mark.parametrize("ty,exponents", [("f32", (-140, -126, -110, -101, -100, -99, 60, 99, 100, 101, 124)),
                                          ("bf16", (-125, -101, -100, 100, 101, 126)), ("f16", (-14, 12))])
def test_near_ties_of_small_and_large_rows(ty, exponents):
    for e in exponents:
        _check(_near_ties(ref.TYPES[ty], 60, 512, 7, e).cuda())


def test_half_of_the_largest():
    # every FP16 and BF16 mantissa of the largest value; 63.5 goes to 64
    for dt, n in ((torch.float16, 1024), (torch.bfloat16, 128), (torch.float32, 1024)):
        a = torch.arange(n, 2 * n, dtype=torch.float64)
        x = torch.stack([a, a / 2, -a / 2, a / 4], 1).to(dt).cuda()
        _check(x)


def test_halves_in_a_norm():
    # half of a row's largest value stays a tie through the norm, whatever the norm is
    import dense_gemm_09_gb300 as dg
    a = torch.arange(1024, 2048, dtype=torch.float64)
    for cols in (4, 300, 9000):
        x = torch.zeros((1024, cols), dtype=torch.float16, device="cuda")
        x[:, :4] = torch.stack([a / 2, a, -a / 2, a / 4], 1).to(torch.float16)
        q, s = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(1024, device="cuda")
        dg.rmsnorm_i8(x, torch.ones(cols, dtype=torch.float16, device="cuda"), q, s)
        assert bool((q[:, :4] == torch.tensor([64, 127, -64, 32], dtype=torch.int8, device="cuda")).all())
        assert not bool(q[:, 4:].any())


@pytest.mark.parametrize("ty", ref.TYPES)
def test_normal_rows(ty):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1000, 3136), generator=g, device="cuda")
    x[:, torch.rand(3136, generator=g, device="cuda") < 0.004] *= 6.0
    _check(x.to(ref.TYPES[ty]))
