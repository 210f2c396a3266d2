"""gemm_i8_tn on the GPU against its formula in float64."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu


def _operands(M, N, K, seed, pad=(0, 0), offset=(0, 0), spread=40.0):
    g = torch.Generator().manual_seed(seed)

    def ints(rows, k, lay):
        v = (torch.randn((rows, k), generator=g) * spread).round_().clamp_(-128, 127).to(torch.int8)
        d, _ = ref.pitched(rows, k, torch.int8, *lay)
        d.copy_(v)
        return d

    A, B = ints(M, K, (pad[0], offset[0])), ints(N, K, (pad[1], offset[1]))
    sa = (torch.rand(M, generator=g) * 0.02 + 0.01).cuda()
    sb = (torch.rand(N, generator=g) * 0.02 + 0.01).cuda()
    return A, B, sa, sb, torch.randn(N, generator=g).cuda() * 3, torch.randn((M, N), generator=g) * 2


def _check(M, N, K, ty="f32", bias=False, beta=0.0, pad=(0, 0), offset=(0, 0), c_pad=0, c_offset=0, seed=0, call=None,
           operands=None):
    """One call against float64; returns the kernel's name."""
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, bv, c0 = operands or _operands(M, N, K, seed or M * 3 + N * 5 + K, pad, offset)
    dt = ref.TYPES[ty]
    C, Cs = ref.pitched(M, N, dt, c_pad, c_offset, fill=77)
    if beta != 0.0:
        C.copy_(c0)
    else:
        C.fill_(float("nan"))  # never read
    c0 = C.cpu()
    out = (call or dg.gemm_i8_tn)(A, B, C, sa, sb, bias=bv if bias else None, beta=beta)
    torch.cuda.synchronize()
    assert out is C
    name = dg.last_kernel()
    a, b = A.cpu(), B.cpu()
    y, mag = ref.product(a, b, sa.cpu(), sb.cpu(), bv.cpu() if bias else None, beta, c0)
    err = ref.partial_error(a, b)
    smag = (a.double().abs() @ b.double().abs().t()) * sa.cpu().double()[:, None] * sb.cpu().double() if err else None
    ref.check_product(C.cpu(), y, mag, smag, err)
    # nothing outside C's elements was written
    s = Cs.clone()
    s[c_offset:c_offset + M * (N + c_pad)].view(M, N + c_pad)[:, :N] = 77
    assert bool((s == 77).all()), name
    return name


# every kernel and tile width on request: (variant, bn, split), name
KERNELS = [((1, 0, 1), "i8_mma_"), ((2, 64, 1), "pair_256x64_tokens"), ((2, 128, 1), "pair_256x128_tokens"),
           ((2, 192, 1), "pair_256x192_tokens"), ((2, 256, 1), "pair_256x256_tokens"),
           ((3, 32, 1), "pair_256x32_channels"), ((3, 160, 1), "pair_256x160_channels"),
           ((3, 96, 1), "pair_256x96_channels"), ((3, 128, 1), "pair_256x128_channels"),
           ((3, 192, 1), "pair_256x192_channels"), ((3, 256, 1), "pair_256x256_channels"),
           ((4, 16, 1), "128x16_channels_split1"),
           ((4, 48, 3), "128x48_channels_split3"), ((4, 64, 8), "128x64_channels_split8"),
           ((4, 112, 5), "128x112_channels_split5"), ((4, 128, 2), "128x128_channels_split2"),
           ((5, 0, 8), "decode_16_channels_8"), ((5, 0, 16), "decode_16_channels_16"),
           ((6, 0, 1), "dot_4_channels")]
MOST_TOKENS = {5: 32, 6: 2}  # of the kernels for few


@pytest.mark.parametrize("tune,name", KERNELS, ids=[n for _, n in KERNELS])
def test_every_kernel(tune, name):
    import dense_gemm_09_gb300 as dg

    def call(*a, **k):
        dg.tune_i8_next(*tune)
        return dg.gemm_i8_tn(*a, **k)

    # one K block (whole, half, a tail in either half), many; one tile, ragged
    # edges both ways, several tiles
    for M, N, K in ((128, 128, 128), (1, 1, 16), (16, 128, 64), (30, 500, 48), (130, 129, 80), (256, 192, 1024),
                    (100, 300, 2064), (257, 513, 1000), (300, 700, 4096), (2, 37, 4100), (3, 300, 9000), (4, 70, 513),
                    (7, 33, 3000), (9, 17, 130), (24, 300, 2500)):
        if M > MOST_TOKENS.get(tune[0], M):
            continue
        for ty, bias, beta in (("f32", True, 0.5), ("bf16", False, 0.0)):
            got = _check(M, N, K, ty, bias, beta, pad=((-K) % 16, (-K) % 16), call=call)
            split = tune[2]
            if tune[0] == 4 and (-(-M // tune[1])) * (-(-N // 128)) * split > 128:
                continue  # more clusters than fit at once: the automatic choice
            assert name in got, got
    assert dg.device_status() == dg.OK


@pytest.mark.parametrize("tune,name", KERNELS[1:], ids=[n for _, n in KERNELS[1:]])
@pytest.mark.parametrize("c_pad,c_offset", [(0, 0), (1, 0), (8, 3)])
def test_every_kernel_stores_any_pitch(tune, name, c_pad, c_offset):
    import dense_gemm_09_gb300 as dg

    def call(*a, **k):
        dg.tune_i8_next(*tune)
        return dg.gemm_i8_tn(*a, **k)

    M = min(70, MOST_TOKENS.get(tune[0], 70))
    for ty in ref.TYPES:
        assert name in _check(M, 333, 256, ty, True, 0.5, c_pad=c_pad, c_offset=c_offset, call=call)


def test_tune_refusals():
    import dense_gemm_09_gb300 as dg
    for bad in ((-1, 0, 1), (7, 0, 1), (2, 32, 1), (2, 320, 1), (3, 16, 1), (3, 288, 1), (4, 8, 1), (4, 144, 1), (4, 64, 0),
                (4, 64, 9), (5, 0, 4), (6, 0, 2), (6, 0, 8)):
        with pytest.raises(dg.DgemmError):
            dg.tune_i8_next(*bad)
    # what the next call cannot take is ignored
    A, B, sa, sb, _, _ = _operands(100, 300, 256, 3)
    C = torch.empty((100, 300), device="cuda")
    dg.tune_i8_next(6, 0, 1)
    dg.gemm_i8_tn(A, B, C, sa, sb)
    assert "dot" not in dg.last_kernel()
    dg.tune_i8_next(1)
    dg.tune_i8_next(0)
    dg.gemm_i8_tn(A, B, C, sa, sb)
    assert "mma" not in dg.last_kernel().replace("umma", "")


SMALL = [(1, 1, 1), (1, 1, 64), (2, 3, 5), (7, 9, 33), (16, 16, 16), (17, 65, 129), (64, 64, 64), (65, 63, 127),
         (128, 128, 128), (129, 127, 255), (31, 300, 1024), (200, 33, 1000)]


@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("bias,beta", [(False, 0.0), (True, 0.0), (True, -0.5)])
def test_small_shapes(ty, bias, beta):
    for M, N, K in SMALL:
        _check(M, N, K, ty, bias, beta)


# rows of tokens around every tile edge x channels x features, as decoding and
# prompts have them; tails in every direction
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 192,
                               255, 256, 257, 383, 512, 700])
@pytest.mark.parametrize("N,K", [(512, 1024), (1000, 528), (1536, 2048)])
def test_tokens(M, N, K):
    ty = ("f32", "f16", "bf16")[M % 3]
    _check(M, N, K, ty, bias=M % 2 == 0)


@pytest.mark.parametrize("M,N,K", [(300, 5000, 4096), (2048, 2048, 1024), (1000, 4097, 999), (2500, 1111, 640),
                                   (4096, 1024, 512), (129, 9000, 2000), (96, 4096, 8192), (5, 4096, 14336),
                                   (16, 100, 16384), (64, 128, 9000), (600, 600, 7000)])
def test_larger_shapes(M, N, K):
    for ty, bias, beta in (("bf16", False, 0.0), ("f32", True, 0.25)):
        _check(M, N, K, ty, bias, beta, pad=((-K) % 16, (-K) % 16))


@pytest.mark.parametrize("pad,offset", [((1, 0), (0, 0)), ((0, 3), (0, 0)), ((4, 8), (0, 4)), ((16, 16), (1, 0)),
                                        ((16, 16), (0, 2)), ((5, 7), (3, 9)), ((32, 16), (16, 32))])
@pytest.mark.parametrize("M", [1, 13, 130])
def test_pitches_and_offsets(M, pad, offset):
    for N, K in ((70, 100), (300, 512)):
        _check(M, N, K, "bf16", True, 0.5, pad=pad, offset=offset, c_pad=3, c_offset=1)


@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("c_pad,c_offset", [(0, 0), (1, 0), (0, 1), (7, 5), (8, 8)])
@pytest.mark.parametrize("M,N,K", [(1, 257, 512), (12, 257, 512), (100, 520, 512), (600, 2065, 256)])
def test_outputs_of_any_pitch(ty, c_pad, c_offset, M, N, K):
    _check(M, N, K, ty, True, 0.5, c_pad=c_pad, c_offset=c_offset)


@pytest.mark.parametrize("M", [1, 6, 16, 40, 128, 300, 1100])
@pytest.mark.parametrize("K", [512, 1024])
def test_sums_are_exact_up_to_1024_deep(M, K):
    # scales of 1 and FP32 output: every sum is a whole number below 2^24
    import dense_gemm_09_gb300 as dg
    N = 1100
    A, B, _, _, _, _ = _operands(M, N, K, 5, spread=200.0)  # most values at the ends
    A[0] = -128
    B[0] = -128
    C = torch.empty((M, N), device="cuda")
    dg.gemm_i8_tn(A, B, C, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"))
    want = A.cpu().double() @ B.cpu().double().t()
    assert torch.equal(C.cpu().double(), want)


@pytest.mark.parametrize("M", [1, 16, 100, 600])
def test_sums_past_2_24(M):
    # every product of one sign: the sum outgrows FP32's whole numbers
    K, N = 16384, 700
    A = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    B = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    B[1::2] = -128
    one = torch.ones(max(M, N), device="cuda")
    _check(M, N, K, "f32", operands=(A, B, one[:M].clone(), one[:N].clone(), one[:N], torch.zeros(M, N)))


def test_a_sum_past_int32():
    # K * 128 * 128 is past 2^31
    import dense_gemm_09_gb300 as dg
    for K in (140000, 140001):
        A = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
        B = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
        C = torch.empty((3, 5), device="cuda")
        dg.gemm_i8_tn(A, B, C, torch.ones(3, device="cuda"), torch.ones(5, device="cuda"))
        want = K * 128.0 * 128.0
        assert bool(((C - want).abs() <= want * (K / 16 + 16) * 2 * ref.E).all())


@pytest.mark.parametrize("M", [1, 20, 200])
def test_scales_that_are_not_numbers_mark_their_rows(M):
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, _, _ = _operands(M, 300, 256, 3)
    sa[0] = float("nan")
    A[0] = 0
    sb[7] = float("inf")
    C = torch.empty((M, 300), device="cuda")
    dg.gemm_i8_tn(A, B, C, sa, sb)
    c = C.cpu()
    assert bool(torch.isnan(c[0]).all())
    assert not bool(torch.isfinite(c[1:, 7]).any())
    ok = torch.ones(300, dtype=torch.bool)
    ok[7] = False
    assert bool(torch.isfinite(c[1:, ok]).all())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_zero_scales_and_no_features(M):
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, bias, c0 = _operands(M, 300, 256, 3)
    sa.zero_()
    C = torch.full((M, 300), 5.0, device="cuda")
    dg.gemm_i8_tn(A, B, C, sa, sb, bias=bias)
    assert torch.equal(C.cpu(), bias.cpu().expand(M, 300))
    # K == 0: bias + beta * C
    C.copy_(c0)
    dg.gemm_i8_tn(A[:, :0], B[:, :0], C, sa, sb, bias=bias, beta=2.0)
    want = bias.cpu().double() + 2.0 * c0.double()
    assert bool(((C.cpu().double() - want).abs() <= 4 * ref.E * (bias.cpu().abs() + 2 * c0.abs())).all())
    dg.gemm_i8_tn(A[:0], B, C[:0], sa[:0], sb)
    dg.gemm_i8_tn(A, B[:0], C[:, :0], sa, sb[:0])


def test_f16_outputs_past_the_range_are_infinite():
    import dense_gemm_09_gb300 as dg
    for M in (1, 30, 300):
        A = torch.full((M, 512), 100, dtype=torch.int8, device="cuda")
        B = torch.full((64, 512), 100, dtype=torch.int8, device="cuda")
        C = torch.empty((M, 64), dtype=torch.float16, device="cuda")
        dg.gemm_i8_tn(A, B, C, torch.ones(M, device="cuda"), torch.ones(64, device="cuda"))
        assert bool(torch.isinf(C).all())


def test_the_same_inputs_give_the_same_bits():
    import dense_gemm_09_gb300 as dg
    for M, N, K in ((1, 4096, 4096), (16, 1000, 8192), (100, 2000, 4096), (700, 1500, 2000)):
        A, B, sa, sb, _, _ = _operands(M, N, K, 4)
        C0, C1 = (torch.empty((M, N), device="cuda") for _ in range(2))
        dg.gemm_i8_tn(A, B, C0, sa, sb)
        for _ in range(3):
            dg.gemm_i8_tn(A, B, C1.zero_(), sa, sb)
            assert torch.equal(C0, C1)


def test_offsets_past_2_31_bytes():
    # B of more than 2^31 bytes, and rows of C far apart
    import dense_gemm_09_gb300 as dg
    N, K = 140000, 16384
    B = torch.empty((N, K), dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, N, 10000):
        B[i:i + 10000] = torch.randint(-50, 51, (10000, K), generator=g, device="cuda", dtype=torch.int8)
    for M in (1, 5, 40, 300):
        A = torch.randint(-50, 51, (M, K), generator=g, device="cuda", dtype=torch.int8)
        C = torch.empty((M, N), device="cuda")
        dg.gemm_i8_tn(A, B, C, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"))
        for cols in (slice(0, 300), slice(131000, 131200), slice(N - 300, N)):
            want = A.double() @ B[cols].double().t()
            assert torch.equal(C[:, cols].double(), want), (M, cols)


def test_streams_and_graphs():
    import dense_gemm_09_gb300 as dg
    probs = []
    for M, N, K in ((1, 2048, 2048), (24, 1000, 4096), (120, 3000, 1024), (900, 2000, 512)):
        A, B, sa, sb, bias, _ = _operands(M, N, K, 9)
        C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        dg.gemm_i8_tn(A, B, C, sa, sb, bias=bias)
        probs.append((A, B, sa, sb, bias, C, C.clone()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for A, B, sa, sb, bias, C, _ in probs:
            dg.gemm_i8_tn(A, B, C.zero_(), sa, sb, bias=bias)
    side.synchronize()
    for *_, C, want in probs:
        assert torch.equal(C, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for A, B, sa, sb, bias, C, _ in probs:
            dg.gemm_i8_tn(A, B, C, sa, sb, bias=bias)
    for _ in range(2):
        for *_, C, _w in probs:
            C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for *_, C, want in probs:
            assert torch.equal(C, want)
    assert dg.device_status() == dg.OK


def test_fuzz():
    import random
    rng = random.Random(11)
    for i in range(60):
        M = int(2 ** rng.uniform(0, 10.5))
        N = int(2 ** rng.uniform(0, 12))
        K = int(2 ** rng.uniform(0, 12))
        pad = ((-K) % 16 + 16 * rng.randrange(3),) * 2 if i % 3 else (rng.randrange(5), rng.randrange(5))
        _check(M, N, K, rng.choice(list(ref.TYPES)), rng.random() < 0.5, rng.choice([0.0, 0.0, 1.0, -0.25]), pad=pad,
               c_pad=rng.choice([0, 0, 1, 8]), seed=1000 + i)


def test_refusals():
    import dense_gemm_09_gb300 as dg
    A, B, sa, sb, bias, _ = _operands(4, 6, 32, 1)
    C = torch.empty((4, 6), device="cuda")
    with pytest.raises(TypeError):
        dg.gemm_i8_tn(A.to(torch.uint8), B, C, sa, sb)
    with pytest.raises(TypeError):
        dg.gemm_i8_tn(A, B, C.double(), sa, sb)
    with pytest.raises(TypeError):
        dg.gemm_i8_tn(A, B, C, sa.half(), sb)
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A, B[:, :31], C, sa, sb)
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A, B, C[:, :5], sa, sb)
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A, B, C, sa[:3], sb)
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A, B, C, sa, sb, bias=bias[:5])
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A.cpu(), B, C, sa, sb)
    with pytest.raises(ValueError):
        dg.gemm_i8_tn(A, B, torch.empty((6, 4), device="cuda").t(), sa, sb)


@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("M", [12, 16, 31])
def test_more_channels_than_one_wave(M, ty):
    # a CTA an SM holds 128 channels: several tiles a CTA, the last wave ragged
    import dense_gemm_09_gb300 as dg
    for N in (19456, 19457, 20481, 24576, 29312, 39001):
        _check(M, N, 1024, ty, True, 0.5)
    assert dg.device_status() == dg.OK
