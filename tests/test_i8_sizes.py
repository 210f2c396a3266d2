"""gemm_i8_tn refuses more than 2^31 - 1 tiles of 64 x 64, up to the largest sizes
there are (no GPU: the pointers are never read)."""
import pytest
import torch

P = 0x1000
MAX = 2 ** 63 - 1


@pytest.mark.parametrize("M,N", [(MAX, 1), (MAX - 60, 1), (MAX - 63, 1), (1, MAX), (MAX, MAX), (MAX, 64), (2 ** 62, 2 ** 62),
                                 (64 * (2 ** 31 - 1) + 1, 1), (64 * 2 ** 16, 64 * 2 ** 15), (65, 64 * 2 ** 30)])
def test_too_many_tiles(M, N):
    import dense_gemm_09_gb300 as dg
    dg.build()
    assert dg.lib().gemm_i8_tn(M, N, 8, P, 8, P, P, 8, P, None, 0.0, P, N, 0, None) == dg.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on a GPU")
@pytest.mark.parametrize("M,N", [(64 * (2 ** 31 - 1), 1), (64, 64 * (2 ** 31 - 1)), (64 * 2 ** 15, 64 * (2 ** 16 - 1))])
def test_the_most_tiles(M, N):
    import dense_gemm_09_gb300 as dg
    dg.build()
    assert dg.lib().gemm_i8_tn(M, N, 8, P, 8, P, P, 8, P, None, 0.0, P, N, 0, None) == dg.ERR_UNSUPPORTED_DEVICE
