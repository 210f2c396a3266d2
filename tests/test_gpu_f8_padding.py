"""What lies between an operand's rows and behind its last one is no part of it: with NaNs there
the calls give the bits that they give with zeros."""
import pytest
import torch

from tests import f8_reference as ref
from tests.test_gpu_f8_gemm import KERNELS, tune

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def among(t, pad, fill):
    """t at a pitch `pad` elements past a 16-byte boundary, and `fill` (a byte) all around it."""
    m, k = t.shape
    per = 16 // t.element_size()
    ld = -(-k // per) * per + pad
    store = torch.full(((m + 2) * ld * t.element_size() + 64,), fill, dtype=torch.uint8, device="cuda")
    out = store[16 * 4:].view(t.dtype)[:m * ld].view(m, ld)[:, :k]
    return out.copy_(t.view(t.dtype))


def both(f):
    """f with zeros in the padding and with bytes of 0x7F and of 0xFF: NaNs, or FP32's and bfloat16's
    largest values."""
    zeros = f(0)
    for fill in (0x7F, 0xFF):
        for a, b in zip(zeros, f(fill)):
            kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
            assert torch.equal(a.view(kind), b.view(kind))
    return zeros


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("k", [1, 5, 15, 16, 17, 100, 127, 130, 250, 257, 1001])
@pytest.mark.parametrize("fa", ref.F8)
@pytest.mark.parametrize("m,n", [(1, 40), (6, 130), (40, 300)])
def test_products(dg, m, n, k, fa, kernel):
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa = ref.operand(m, k, 1, ref.F8[fa], g)
    b, sb = ref.operand(n, k, 128, torch.float8_e4m3fn, g)

    def run(fill):
        c = torch.empty(m, n, device="cuda")
        tune(dg, kernel)
        return [dg.gemm_f8_tn(among(a, 0, fill), among(b, 16, fill), c, sa, sb)]

    c, = both(run)
    assert bool(c.isfinite().all()) and dg.device_status() == dg.OK


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("k", [5, 127, 130, 1001])
def test_products_by_expert(dg, k, kernel):
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa = ref.operand(90, k, 1, torch.float8_e4m3fn, g)
    b, sb = ref.operand(3 * 70, k, 1, torch.float8_e4m3fn, g)
    off = torch.tensor([0, 20, 21, 90], dtype=torch.int32, device="cuda")

    def run(fill):
        w = among(b, 0, fill)
        ld = w.stride(0)
        tune(dg, kernel)
        return [dg.gemm_f8_tn_experts(among(a, 0, fill), w.as_strided((3, 70, k), (70 * ld, ld, 1)), torch.empty(90, 70, device="cuda"),
                                      sa, sb.view(3, 70, -1), off)]

    c, = both(run)
    assert bool(c.isfinite().all())


@pytest.mark.parametrize("t", ref.TYPES)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 127), (130, 130), (257, 1001)])
def test_rows(dg, m, k, pad, t):
    g = torch.Generator(device="cuda").manual_seed(k)
    x, u = (torch.randn(m, k, generator=g, device="cuda").to(ref.TYPES[t]) for _ in range(2))
    position = torch.randperm(m, device="cuda").to(torch.int32).view(m, 1)
    f8 = torch.float8_e4m3fn

    def run(fill):
        out = []
        for form in ("rows", "blocks", "transposed", "swiglu", "gather"):
            qm, qk = (k, m) if form == "transposed" else (m, k)
            rows = -(-qm // 128) if form == "blocks" else qm
            q, s = among(torch.zeros(qm, qk, device="cuda").to(f8), pad, fill), torch.empty(rows, ref.blocks(qk), device="cuda")
            if form == "swiglu":
                dg.swiglu_f8(among(x, pad, fill), among(u, pad, fill), q, s)
            elif form == "gather":
                dg.gather_by_expert_f8(among(x, pad, fill), position, q, s)
            else:
                dg.quantize_f8(among(x, pad, fill), q, s, transposed=form == "transposed")
            back = dg.dequantize_f8(q, s, torch.empty(qm, qk, device="cuda"))
            assert bool(back.isfinite().all())
            out += [q.contiguous(), s, back]
        y = among(torch.zeros_like(x), pad, fill)
        dg.gather_by_expert(among(x, pad, fill), position, y)
        w, dw = torch.full((m, 1), 0.5, device="cuda"), torch.empty(m, 1, device="cuda")
        dy = torch.empty_like(x)
        dg.combine_experts_grad(among(x, pad, fill), y, position, w, dy, dw)
        return out + [y.contiguous(), dg.combine_experts(y, position, w, among(u, pad, fill), beta=1.0).contiguous(), dy, dw]

    both(run)
