"""A stalled tensor-core launch whose waits run out while its loads are still in
flight (limits from a nanosecond on; K short, so that the producer has issued
its last load, and long): the launch waits for what it has in flight, ends with
DGEMM_ERR_TIMEOUT, and the next call is ordinary again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# path, dgemm_tune_next's variant, bn and split (whole tiles only), M, N
KINDS = [("f16_tn", (1, 256, 1), 300, 700), ("f16_tn", (5, 256, 1), 300, 700), ("f16_nn", (1, 256, 1), 4096, 6144),
         ("f16_tn", (6, 256, 1), 300, 700), ("f16_tn", (2, 128, 1), 300, 700), ("f16_tn", (2, 256, 1), 300, 700),
         ("f16_tn", (3, 64, 4), 100, 300), ("f16_tn", (8, 128, 1), 100, 700), ("f16_nn", (8, 256, 1), 100, 704),
         ("tf32", (1, 256, 1), 300, 704), ("tf32", (2, 256, 1), 300, 704), ("tf32", (3, 64, 4), 100, 320)]


@pytest.mark.parametrize("K", [64, 256, 2048])
@pytest.mark.parametrize("path,tune,M,N", KINDS, ids=["%s-%d-%d-%d" % ((p,) + t) for p, t, _, _ in KINDS])
def test_waits_that_run_out_at_once(path, tune, M, N, K):
    import dense_gemm_09_gb300 as dg
    g = torch.Generator(device="cuda").manual_seed(K)
    dt = torch.float32 if path == "tf32" else torch.float16
    call = {"f16_tn": dg.gemm_f16_tn, "f16_nn": dg.gemm_f16_nn, "tf32": dg.gemm_tf32}[path]
    A = torch.randn((M, K), generator=g, device="cuda").to(dt)
    B = torch.randn((N, K) if path == "f16_tn" else (K, N), generator=g, device="cuda").to(dt)
    C, want = torch.empty((M, N), dtype=dt, device="cuda"), torch.empty((M, N), dtype=dt, device="cuda")
    dg.tune_next(*tune)
    call(A, B, want)
    assert dg.device_status(clear=True) == dg.OK
    name = dg.last_kernel()
    assert "cpasync" not in name and "ldst" not in name, name
    for limit in (0, 1, 300, 1000, 3000, 20000):
        for _ in range(3):
            dg.tune_next(*tune)
            dg.test_inject_stall(limit)
            call(A, B, C)
            assert dg.last_kernel() == name
            st = dg.device_status(clear=True)  # synchronises
            assert st == dg.ERR_TIMEOUT, dg.status_string(st)
        dg.tune_next(*tune)
        call(A, B, C.zero_())
        assert dg.device_status(clear=True) == dg.OK
        assert torch.equal(C, want)
