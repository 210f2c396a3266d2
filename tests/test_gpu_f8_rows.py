"""quantize_f8, swiglu_f8 and dequantize_f8 on a GPU."""
import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 128), (1, 4096), (2, 127), (3, 129), (128, 128), (129, 257), (255, 640), (300, 1000), (1, 16384),
          (2000, 384), (4096, 2056)]


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def values(m, k, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, k, generator=g, device="cuda") * torch.exp2(4 * torch.randn(m, 1, generator=g, device="cuda"))
    return x.to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8)


def scales(rows, blocks, k_major):
    """rows x blocks of scales, by either stride order, in a larger storage of 7s."""
    s = torch.full((blocks + 1, rows + 1) if k_major else (rows + 1, blocks + 1), 7.0, device="cuda")
    return (s.t() if k_major else s)[:rows, :blocks], s


def check_quantize(dg, x, form, f8, pad=0, offset=0, k_major=False):
    m, k = x.shape
    rows = ref.BLOCK if form == "blocks" else 1
    qm, qk = (k, m) if form == "transposed" else (m, k)
    q, store = ref.pitched(qm, qk, torch.uint8, pad, offset, fill=99)
    scale, sstore = scales(-(-qm // rows), ref.blocks(qk), k_major)
    got = dg.quantize_f8(x, q.view(f8), scale, transposed=form == "transposed")
    assert got[1] is scale
    y = x.float().t() if form == "transposed" else x.float()
    want, ws = ref.quantized(y, rows, f8)
    assert torch.equal(scale.nan_to_num(-1.0), ws.nan_to_num(-1.0))
    assert torch.equal(q, bits(want).view(qm, qk))
    q.fill_(99)
    scale.fill_(7.0)
    assert bool((store == 99).all()) and bool((sstore == 7.0).all())  # nothing beside them was written


@pytest.mark.parametrize("form", ["rows", "blocks", "transposed"])
@pytest.mark.parametrize("f8", ref.F8)
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("m,k", SHAPES)
def test_quantize(dg, m, k, dtype, f8, form):
    check_quantize(dg, values(m, k, ref.TYPES[dtype]), form, ref.F8[f8])


@pytest.mark.parametrize("form", ["rows", "blocks", "transposed"])
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("pad,offset,xpad,xoffset", [(0, 1, 0, 0), (3, 0, 0, 0), (8, 8, 8, 8), (0, 0, 1, 0), (5, 3, 3, 1)])
def test_quantize_layouts(dg, dtype, form, pad, offset, xpad, xoffset):
    x, _ = ref.pitched(200, 333, ref.TYPES[dtype], xpad, xoffset)
    x.copy_(values(200, 333, ref.TYPES[dtype], 1))
    for k_major in (False, True):
        check_quantize(dg, x, form, torch.float8_e4m3fn, pad, offset, k_major)


@pytest.mark.parametrize("form", ["rows", "blocks", "transposed"])
@pytest.mark.parametrize("dtype", ref.TYPES)
def test_quantize_what_is_not_ordinary(dg, dtype, form):
    """Zeros, infinities, NaN, the types' smallest and largest values, and values next
    to them."""
    t = ref.TYPES[dtype]
    x = values(600, 300, t, 2)
    x[:130] = 0.0
    x[131, 5] = float("inf")
    x[140, 200] = float("-inf")
    x[300, 299] = float("nan")
    x[400:410] = ref.TINY[t]
    x[410:500, :200] *= 2.0 ** -120  # (subnormal or zero in 16 bits)
    x[520] = torch.finfo(t).max
    x[521] = -torch.finfo(t).max
    check_quantize(dg, x, form, torch.float8_e4m3fn)
    check_quantize(dg, x, form, torch.float8_e5m2)


def test_many_rows(dg):
    """More blocks than one grid's worth, of one short block each."""
    check_quantize(dg, values(300000, 3, torch.bfloat16), "rows", torch.float8_e4m3fn)


def test_nothing_to_do(dg):
    for m, k in ((0, 128), (5, 0), (0, 0)):
        x = torch.empty(m, k, device="cuda")
        q, s = torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(m, ref.blocks(k), device="cuda")
        assert dg.quantize_f8(x, q, s)[0] is q
        dg.swiglu_f8(x, x, q, s)
        dg.dequantize_f8(q, s, x)


@pytest.mark.parametrize("f8", ref.F8)
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("m,k,pad", [(1, 1, 0), (16, 2048, 0), (130, 300, 0), (130, 300, 4), (77, 129, 1), (3000, 512, 0)])
def test_swiglu(dg, m, k, pad, dtype, f8):
    t, f8 = ref.TYPES[dtype], ref.F8[f8]
    gu, _ = ref.pitched(m, 2 * k, t, pad)  # column slices of one matrix
    gu.copy_(values(m, 2 * k, t, 3))
    if k > 1:
        gu[0, :2] = torch.tensor([100.0, -100.0], device="cuda")
    g, u = gu[:, :k], gu[:, k:]
    q, s = torch.empty(m, k, dtype=f8, device="cuda"), torch.empty(m, ref.blocks(k), device="cuda")
    dg.swiglu_f8(g, u, q, s)
    y = g.double() / (1 + torch.exp(-g.double())) * u.double()
    # each value: g's exponent one rounding in the exponential's argument (|g| log2 e
    # up to 2^8: 2^8 E), ex2 2^-22, the sum, rcp 2^-23, three products
    delta = (2 ** 8 + 4 + 2 + 5) * ref.E
    tiny = 2.0 ** -126 * u.double().abs() + 2.0 ** -149  # gates whose quotient is flushed
    top, a = ref.TOP[f8], torch.nn.functional.pad(y.abs(), (0, -k % 128)).view(m, -1, 128).amax(2)
    assert bool(((s.double() - a / top).abs() <= (delta + 2 * ref.E) * a / top + 2.0 ** -126).all())
    # half a step of the 8-bit type (2^-4, 2^-3 of the value; of the smallest normal one below it)
    half, least = (2.0 ** -4, 2.0 ** -6) if f8 == torch.float8_e4m3fn else (2.0 ** -3, 2.0 ** -14)
    sy = ref.spread(a / top, 1, m, k)
    got = q.double() * ref.spread(s.double(), 1, m, k)
    bound = half * torch.maximum(y.abs(), least * sy) * (1 + 4 * delta) + 4 * delta * y.abs() + tiny
    assert bool(((got - y).abs() <= bound).all())


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("f8", ref.F8)
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("m,k,pad,offset", [(1, 1, 0, 0), (130, 300, 4, 0), (130, 300, 0, 1), (257, 1024, 0, 0), (5000, 136, 0, 0)])
def test_dequantize(dg, m, k, pad, offset, dtype, f8, rows):
    """Every bit pattern, NaN and e5m2's infinities among them."""
    t, f8 = ref.TYPES[dtype], ref.F8[f8]
    q, _ = ref.pitched(m, k, torch.uint8, pad, offset)
    q.copy_(torch.arange(m * k, device="cuda").view(m, k) * 7 % 256)
    g = torch.Generator(device="cuda").manual_seed(4)
    s = torch.exp2(8 * torch.randn(-(-m // rows), ref.blocks(k), generator=g, device="cuda"))
    x, store = ref.pitched(m, k, t, pad, offset, fill=3)
    assert dg.dequantize_f8(q.view(f8), s, x) is x
    want = (q.contiguous().view(f8).float() * ref.spread(s, rows, m, k)).to(t)
    assert torch.equal(x.float().nan_to_num(1e30, 2e38, -2e38), want.float().nan_to_num(1e30, 2e38, -2e38))
    x.fill_(3)
    assert bool((store == 3).all())


def test_broadcast_scales(dg):
    """A scale read through strides of 0."""
    q = torch.randn(300, 400, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((1, 1), 0.5, device="cuda")
    x = torch.empty(300, 400, device="cuda")
    dg.dequantize_f8(q, s.expand(300, 4), x)
    assert torch.equal(x, q.float() * 0.5)
