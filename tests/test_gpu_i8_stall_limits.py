"""A stalled tensor-core launch of gemm_i8_tn whose waits run out while its
loads are still in flight: with a limit of a nanosecond to some microseconds,
every role gives up at another point, some after the producer has issued
its last load.  The launch waits for what it has in flight, ends with
DGEMM_ERR_TIMEOUT, and the next call is ordinary again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# (variant, bn, split), M, N: pairs of either kind, single CTAs, clusters that
# share a tile; several tiles a CTA
KINDS = [((2, 128, 1), 300, 700), ((2, 192, 1), 4096, 8192), ((3, 64, 1), 60, 1000), ((3, 192, 1), 2048, 16384),
         ((4, 32, 1), 30, 700), ((4, 64, 4), 60, 1000), ((4, 128, 8), 100, 300)]


@pytest.mark.parametrize("K", [128, 256, 384, 2048])
@pytest.mark.parametrize("tune,M,N", KINDS, ids=["%d-%d-%d_%dx%d" % (t + (m, n)) for t, m, n in KINDS])
def test_waits_that_run_out_at_once(tune, M, N, K):
    import dense_gemm_09_gb300 as dg
    g = torch.Generator(device="cuda").manual_seed(K)
    A = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    C, want = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    dg.tune_i8_next(*tune)
    dg.gemm_i8_tn(A, B, want, sa, sb)
    assert dg.device_status(clear=True) == dg.OK
    name = dg.last_kernel()
    assert "umma" in name
    for limit in (0, 1, 300, 1000, 3000, 20000):
        for _ in range(3):
            dg.tune_i8_next(*tune)
            dg.test_inject_stall(limit)
            dg.gemm_i8_tn(A, B, C, sa, sb)
            assert dg.last_kernel() == name
            st = dg.device_status(clear=True)  # synchronises
            assert st == dg.ERR_TIMEOUT, dg.status_string(st)
        dg.tune_i8_next(*tune)
        dg.gemm_i8_tn(A, B, C.zero_(), sa, sb)
        assert dg.device_status(clear=True) == dg.OK
        assert torch.equal(C, want)
