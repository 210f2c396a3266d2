"""The 8-bit kernels' failure detection and bounds checks on the GPU.

A stalled tensor-core launch (the test hook of test_gpu_timeout.py) ends by
itself with DGEMM_ERR_TIMEOUT and leaves the context usable; and in the checked
build (test_gpu_checked.py) no index any kernel computes leaves its extent, at
the sizes where it could, with results that are right."""
import time

import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu


def _operands(M, N, K, seed, pad=0):
    g = torch.Generator().manual_seed(seed)

    def ints(rows):
        d, _ = ref.pitched(rows, K, torch.int8, pad)
        d.copy_(torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int8))
        return d

    return ints(M), ints(N), torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()


STALLS = [((2, 128, 1), (300, 700, 512), "_tokens"), ((2, 192, 1), (2048, 12288, 256), "_tokens"),
          ((3, 64, 1), (60, 1000, 2048), "256x64_channels"), ((4, 32, 1), (30, 700, 512), "split1"),
          ((4, 64, 4), (60, 1000, 2048), "split4")]


@pytest.mark.parametrize("tune,shape,name", STALLS, ids=["%s-%dx%dx%d" % ((n.strip("_"),) + s) for _, s, n in STALLS])
def test_a_stalled_launch_times_out_cleanly(tune, shape, name):
    import dense_gemm_09_gb300 as dg
    M, N, K = shape
    A, B, sa, sb = _operands(M, N, K, 3)
    C = torch.empty((M, N), device="cuda")
    torch.cuda.synchronize()
    assert dg.device_status(clear=True) == dg.OK
    dg.tune_i8_next(*tune)
    dg.test_inject_stall(20_000_000)  # 20 ms
    t0 = time.monotonic()
    dg.gemm_i8_tn(A, B, C, sa, sb)
    st = dg.device_status(clear=True)  # synchronises
    assert name in dg.last_kernel()
    assert st == dg.ERR_TIMEOUT, dg.status_string(st)
    assert time.monotonic() - t0 < 10.0
    # the next call is ordinary again
    dg.tune_i8_next(*tune)
    dg.gemm_i8_tn(A, B, C, sa, sb)
    torch.cuda.synchronize()
    assert dg.device_status(clear=True) == dg.OK
    y, mag = ref.product(A.cpu(), B.cpu(), sa.cpu(), sb.cpu())
    err = ref.partial_error(A, B)
    smag = (A.cpu().double().abs() @ B.cpu().double().abs().t()) * sa.cpu().double()[:, None] * sb.cpu().double()
    ref.check_product(C.cpu(), y, mag, smag, err)


@pytest.fixture(scope="module")
def checked():
    """The binding on the checked library, and its status word clear."""
    import dense_gemm_09_gb300 as dg
    from dense_gemm_09_gb300 import _build
    _build.build(checked=True)
    normal = dg.lib()
    dg._lib = dg.lib_checked()
    torch.cuda.synchronize()
    assert dg.device_status() == dg.OK
    yield dg
    dg._lib = normal


def _passed(dg):
    L = dg.lib()
    st, site = L.dgemm_device_status(0), L.dgemm_check_site()
    L.dgemm_device_status(1)
    assert st == dg.OK and site == 0, "%s at site %d" % (dg.status_string(st), site)


SHAPES = [(1, 1, 1), (1, 300, 513), (2, 37, 700), (3, 129, 2000), (5, 17, 129), (8, 300, 300), (9, 65, 4000),
          (17, 129, 127), (31, 500, 1000), (33, 127, 255), (64, 1000, 2100), (127, 129, 640), (128, 256, 256),
          (129, 300, 1000), (256, 700, 128), (257, 1000, 500), (700, 2065, 384)]


@pytest.mark.parametrize("aligned", [True, False])
def test_products_pass_every_check(checked, aligned):
    dg = checked
    for M, N, K in SHAPES:
        A, B, sa, sb = _operands(M, N, K, M + N + K, pad=(-K) % 16 if aligned else 1)
        for ty, beta, cpad in (("f32", 0.5, 0), ("bf16", 0.0, 3), ("f16", 0.0, 8)):
            C, _ = ref.pitched(M, N, ref.TYPES[ty], cpad, fill=2)
            c0 = C.cpu()
            dg.gemm_i8_tn(A, B, C, sa * 1e-3, sb * 1e-2, bias=sb, beta=beta)
            _passed(dg)
            y, mag = ref.product(A.cpu(), B.cpu(), sa.cpu() * 1e-3, sb.cpu() * 1e-2, sb.cpu(), beta, c0)
            a, b = A.cpu().double().abs(), B.cpu().double().abs()
            smag = (a @ b.t()) * (sa.cpu() * 1e-3).double()[:, None] * (sb.cpu() * 1e-2).double()
            ref.check_product(C.cpu(), y, mag, smag, ref.partial_error(A, B))


TUNES = [(1, 0, 1), (2, 64, 1), (2, 192, 1), (2, 256, 1), (3, 32, 1), (3, 160, 1), (3, 256, 1), (4, 16, 1), (4, 48, 5),
         (4, 128, 8), (5, 0, 8), (5, 0, 16), (6, 0, 1)]


@pytest.mark.parametrize("tune", TUNES, ids=["%d-%d-%d" % t for t in TUNES])
def test_every_kernel_passes_every_check(checked, tune):
    dg = checked
    for M, N, K in ((300, 700, 1300), (20, 300, 2064), (4, 129, 5000), (2600, 4200, 256)):
        if M > {5: 32, 6: 2}.get(tune[0], M):
            continue
        A, B, sa, sb = _operands(M, N, K, 5, pad=(-K) % 16)
        C = torch.empty((M, N), device="cuda")
        dg.tune_i8_next(*tune)
        dg.gemm_i8_tn(A, B, C, sa, sb)
        _passed(dg)
        want = A.double() @ B.double().t() * sa.double()[:, None] * sb.double()
        assert bool(((C.double() - want).abs() <= 1e-5 * want.abs().max()).all())


def test_row_operators_pass_every_check(checked):
    dg = checked
    for rows, cols in ((1, 1), (3, 7), (5, 8), (6, 255), (2, 513), (400, 1024), (3, 4095), (700, 8192), (2, 16391),
                       (3, 32768), (2, 40001)):
        for dt in ref.TYPES.values():
            for pad, off in ((0, 0), (8, 8), (3, 1)):
                x, _ = ref.pitched(rows, cols, dt, pad, off)
                x.copy_(torch.randn(rows, cols))
                q, _ = ref.pitched(rows, cols, torch.int8, pad, off)
                s = torch.empty(rows, device="cuda")
                dg.rmsnorm_i8(x, torch.ones(cols, dtype=dt, device="cuda"), q, s, residual=x, H=x)
                _passed(dg)
                dg.swiglu_i8(x, x, q, s)
                _passed(dg)
                dg.quantize_i8(x, q, s)
                _passed(dg)
                ref.check_rows(x.cpu().double(), 0.0, q.cpu(), s.cpu())
                dg.dequantize_i8(q, s, x)
                _passed(dg)
                assert torch.equal(x.cpu(), (q.cpu().float() * s.cpu()[:, None]).to(dt))
