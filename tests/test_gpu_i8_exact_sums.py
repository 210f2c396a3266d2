"""gemm_i8_tn: sums are exact wherever sum |a| |b| < 2^24, however long K is, in
every kernel; and how far they may be off beyond it."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu

# (variant, bn, split) of dgemm_tune_i8_next, most tokens
KERNELS = [((0, 0, 1), 600), ((1, 0, 1), 600), ((2, 64, 1), 600), ((2, 192, 1), 600), ((2, 256, 1), 600), ((3, 64, 1), 600),
           ((3, 192, 1), 600), ((3, 256, 1), 600), ((4, 32, 1), 600), ((4, 64, 4), 600), ((4, 128, 8), 600), ((5, 0, 8), 32),
           ((5, 0, 16), 32), ((6, 0, 1), 2)]
IDS = ["%d-%d-%d" % k[0] for k in KERNELS]


def _sums(tune, A, B):
    """A B^T in FP32 with scales of 1, and the true sums."""
    import dense_gemm_09_gb300 as dg
    M, N = A.shape[0], B.shape[0]
    C = torch.empty((M, N), device="cuda")
    dg.tune_i8_next(*tune)
    dg.gemm_i8_tn(A, B, C, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"))
    return C.double(), A.double() @ B.double().t()


def _normal(rows, K, spread, g):
    return (torch.randn((rows, K), generator=g, device="cuda") * spread).round().clamp(-127, 127).to(torch.int8)


@pytest.mark.parametrize("tune,most", KERNELS, ids=IDS)
def test_exact_below_2_24(tune, most):
    g = torch.Generator(device="cuda").manual_seed(1)
    for M, N, K, spread in ((300, 700, 4096, 40.0), (70, 300, 8192, 30.0), (20, 130, 16384, 24.0), (2, 70, 65536, 11.0)):
        M = min(M, most)
        A, B = _normal(M, K, spread, g), _normal(N, K, spread, g)
        size = A.double().abs() @ B.double().abs().t()
        assert float(size.max()) < 2.0 ** 24 and K > 1024
        got, want = _sums(tune, A, B)
        assert torch.equal(got, want)


@pytest.mark.parametrize("tune,most", KERNELS, ids=IDS)
def test_exact_whatever_the_order(tune, most):
    # a sum just below 2^24 from the first (or last, or every 8th) products, and
    # ones of either sign around it
    g = torch.Generator(device="cuda").manual_seed(2)
    M, N, K = min(40, most), 150, 8192
    for where in (slice(0, 1024), slice(K - 1024, K), slice(0, K, 8)):
        A = torch.randint(-1, 2, (M, K), generator=g, device="cuda", dtype=torch.int8)
        B = torch.randint(-1, 2, (N, K), generator=g, device="cuda", dtype=torch.int8)
        A[:, where] = 127
        B[:, where] = 127
        B[1::2, where] = -127
        size = A.double().abs() @ B.double().abs().t()
        assert float(size.max()) < 2.0 ** 24
        got, want = _sums(tune, A, B)
        assert torch.equal(got, want)


@pytest.mark.parametrize("tune,most", KERNELS, ids=IDS)
def test_past_2_24(tune, most):
    # integer kernels round once; the tensor-core kernels may lose a unit in the
    # last place of the running sum at each of their K / 16 steps
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = min(40, most), 150, 16384
    sign = torch.randint(0, 2, (N, 1), generator=g, device="cuda", dtype=torch.int8) * 2 - 1
    one_signed = (torch.randint(80, 128, (M, K), generator=g, device="cuda", dtype=torch.int8),
                  torch.randint(80, 128, (N, K), generator=g, device="cuda", dtype=torch.int8) * sign)
    # the second half takes back what the first has summed, up to small values
    half = torch.randint(80, 128, (M, K // 2), generator=g, device="cuda", dtype=torch.int8)
    other = torch.randint(80, 127, (N, K // 2), generator=g, device="cuda", dtype=torch.int8)
    more = other + torch.randint(0, 2, (N, K // 2), generator=g, device="cuda", dtype=torch.int8)
    cancelling = torch.cat([half, -half], 1), torch.cat([other, more], 1)
    for name, (A, B) in (("one sign", one_signed), ("cancelling", cancelling)):
        got, want = _sums(tune, A, B)
        size = A.double().abs() @ B.double().abs().t()
        err = (got - want).abs()
        print("%s %s: off by %.3g of the sum of sizes, %.3g of the sum"
              % (tune, name, float((err / size).max()), float((err / want.abs().clamp(min=1.0)).max())))
        if tune[0] in (1, 5, 6):  # exact int32, rounded once
            assert bool((err <= ref.E * want.abs()).all())
        else:
            assert bool((err <= (K / 16 + 16) * 2 * ref.E * size).all())
