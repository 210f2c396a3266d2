"""What one warp of the 8-bit floating-point products hands to another, many times over in one
launch.  (Small whole numbers: every product and sum is exact in FP32 and rounded once, so
that values of another turn show.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def ints(*shape, most=4):
    return torch.randint(-most, most + 1, shape, device="cuda").float()


def turns(rows, blocks):
    """Scales that differ from block to block and from row to row."""
    return ((torch.arange(blocks, device="cuda") + 3 * torch.arange(rows, device="cuda")[:, None]) % 7 + 1).float()


def product(a, sa, b, sb, rb):
    k = a.shape[1]
    wide = [s.double().repeat_interleave(128, 1)[:, :k] for s in (sa, sb.repeat_interleave(rb, 0)[:b.shape[0]])]
    return (a.double() * wide[0]) @ (b.double() * wide[1]).t()


@pytest.mark.parametrize("kernel", [(3, 16, 1), (3, 16, 4), (3, 32, 1), (3, 32, 2), (3, 64, 1), (3, 64, 8)], ids=str)
@pytest.mark.parametrize("rb", [1, 128])
@pytest.mark.parametrize("k", [128, 1024, 1152, 5248])
def test_scales_of_many_turns(dg, k, rb, kernel):
    """The scales' ring is written many times over, by a tile's blocks and from tile to tile."""
    for m, n in ((kernel[1] - 3, 700), (kernel[1] * 3 + 1, 700 if kernel[2] > 1 else 30000)):
        a, b = ints(m, k), ints(n, k)
        sa, sb = turns(m, -(-k // 128)), turns(-(-n // rb), -(-k // 128))
        want = product(a, sa, b, sb, rb).float()
        c = torch.empty(m, n, device="cuda")
        a8, b8 = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
        for _ in range(5):
            dg.tune_f8_next(*kernel)
            dg.gemm_f8_tn(a8, b8, c.fill_(float("nan")), sa, sb)
            assert torch.equal(c, want), dg.last_kernel()
    assert dg.device_status() == dg.OK


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [129, 1030, 1097])
def test_the_old_c_behind_an_edge(dg, n, out):
    """Several tiles a CTA of which some end inside a 16-byte word: their box is stored by the
    warp, and takes the old C of a later tile by TMA."""
    m, k = 20000, 256
    a, b = ints(m, k), ints(n, k)
    c0 = ints(m, n, most=200)
    want = (a.double() @ b.double().t() - 2 * c0.double()).to(out)
    store = torch.full((m, n + 16 - n % 16), 77.0, device="cuda").to(out)
    c = store[:, :n]
    a8, b8 = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    ones = [torch.ones(m, 2, device="cuda"), torch.ones(n, 2, device="cuda")]
    for rb in (1, 128):
        for _ in range(5):
            c.copy_(c0)
            dg.tune_f8_next(2, 128, 1)
            dg.gemm_f8_tn(a8, b8, c, ones[0], ones[1][:-(-n // rb)], beta=-2.0)
            assert torch.equal(c, want), dg.last_kernel()
    assert bool((store[:, n:] == 77).all()) and dg.device_status() == dg.OK
