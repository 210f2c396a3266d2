"""The tuning hook of gemm_i8_tn holds for the next call and no other."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _operands(M, N, K):
    return (torch.ones((M, K), dtype=torch.int8, device="cuda"), torch.ones((N, K), dtype=torch.int8, device="cuda"),
            torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.empty((M, N), device="cuda"))


def _mma():
    import dense_gemm_09_gb300 as dg
    return dg.last_kernel().startswith("i8_mma")


def test_a_call_with_nothing_to_do_takes_the_request():
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, C = _operands(100, 300, 256)
    dg.tune_i8_next(dg.TUNE_I8_MMA)
    dg.gemm_i8_tn(A[:0], B, C[:0], sa[:0], sb)
    dg.gemm_i8_tn(A, B, C, sa, sb)
    assert not _mma()
    assert bool((C == 256).all())


def test_a_refused_call_takes_the_request():
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, C = _operands(100, 300, 256)
    # by the library
    dg.tune_i8_next(dg.TUNE_I8_MMA)
    assert dg.lib().gemm_i8_tn(-1, 1, 1, None, 1, None, None, 1, None, None, 0.0, None, 1, 0, None) == dg.ERR_INVALID_ARG
    dg.gemm_i8_tn(A, B, C, sa, sb)
    assert not _mma()
    # by the binding
    for bad in ((A, B[:, :8], C, sa, sb), (A.float(), B, C, sa, sb), (A, B, C, sa[:3], sb)):
        dg.tune_i8_next(dg.TUNE_I8_MMA)
        with pytest.raises((TypeError, ValueError)):
            dg.gemm_i8_tn(*bad)
        dg.gemm_i8_tn(A, B, C, sa, sb)
        assert not _mma()
    # and an ordinary call still gets what it asked for
    dg.tune_i8_next(dg.TUNE_I8_MMA)
    dg.gemm_i8_tn(A, B, C, sa, sb)
    assert _mma()


@pytest.mark.parametrize("K,ran", [(128, 1), (300, 3), (1024, 8), (2000, 8)])
def test_the_name_tells_the_split_that_ran(K, ran):
    # a tile of fewer K blocks (of 128) than asked for has one CTA a block
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, C = _operands(60, 200, (K + 15) // 16 * 16)
    dg.tune_i8_next(dg.TUNE_I8_SPLIT, 64, 8)
    dg.gemm_i8_tn(A[:, :K], B[:, :K], C, sa, sb)
    assert dg.last_kernel() == "i8_umma_128x64_channels_split8" + ("" if ran == 8 else "_ran_%d" % ran)
    assert bool((C == K).all())
