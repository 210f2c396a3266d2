"""The 8-bit row operators on the GPU against their formulas in float64."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu

# row lengths around every switch of the kernels: one element, one vector of
# 8, a warp's registers (256, 1024), a block's (4096, 8192, 16384, 32768), past it
LENGTHS = [1, 3, 7, 8, 9, 64, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 8191, 8200, 16384, 16391, 32768,
           32776, 40001]
LAYOUTS = {"tight": (0, 0), "pitched": (24, 0), "odd": (5, 1), "offset": (8, 3)}


def _x(rows, cols, dtype, seed, scale=1.0, layout=(0, 0)):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * scale
    d, _ = ref.pitched(rows, cols, dtype, *layout)
    d.copy_(x)
    return d


def _out(rows, cols, layout=(0, 0)):
    q, qs = ref.pitched(rows, cols, torch.int8, layout[0], layout[1], fill=77)
    return q, qs, torch.full((rows,), -1.0, device="cuda")


def _untouched(q, storage, layout):
    """The bytes between and around q's rows still hold the fill."""
    rows, cols = q.shape
    pad, off = layout
    s = storage.clone()
    s[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = 77
    return bool((s == 77).all())


@pytest.mark.parametrize("layout", LAYOUTS, ids=list(LAYOUTS))
@pytest.mark.parametrize("ty", ref.TYPES)
def test_quantize(ty, layout):
    import dense_gemm_09_gb300 as dg
    lay = LAYOUTS[layout]
    for cols in LENGTHS:
        rows = 5 if cols < 5000 else 2
        x = _x(rows, cols, ref.TYPES[ty], cols, layout=lay)
        q, qs, s = _out(rows, cols, lay)
        assert dg.quantize_i8(x, q, s) == (q, s)
        torch.cuda.synchronize()
        ref.check_rows(x.cpu().double(), 0.0, q.cpu(), s.cpu())
        assert _untouched(q, qs, lay)


@pytest.mark.parametrize("layout", LAYOUTS, ids=list(LAYOUTS))
@pytest.mark.parametrize("ty", ref.TYPES)
@pytest.mark.parametrize("residual,f32_gamma", [(True, False), (False, False), (True, True)])
def test_rmsnorm(ty, layout, residual, f32_gamma):
    import dense_gemm_09_gb300 as dg
    lay, dt, eps = LAYOUTS[layout], ref.TYPES[ty], 1e-5
    for cols in LENGTHS:
        rows = 5 if cols < 5000 else 2
        x = _x(rows, cols, dt, cols, layout=lay)
        r = _x(rows, cols, dt, cols + 1, 3.0, layout=lay) if residual else None
        gamma = (1.0 + 0.3 * _x(1, cols, torch.float32, cols + 2)[0]).to(torch.float32 if f32_gamma else dt)
        q, qs, s = _out(rows, cols, lay)
        H = ref.pitched(rows, cols, dt, *lay)[0] if residual else None
        dg.rmsnorm_i8(x, gamma, q, s, residual=r, H=H, eps=eps)
        torch.cuda.synchronize()
        h, y, delta = ref.norm_rows(x.cpu(), gamma.cpu(), r.cpu() if residual else None, eps)
        ref.check_rows(y, delta, q.cpu(), s.cpu())
        assert _untouched(q, qs, lay)
        if residual:
            # one FP32 sum, one rounding to the type
            tol = (ref.U[dt] + 2 * ref.E) * h.abs() + ref.TINY[dt]
            assert bool(((H.cpu().double() - h).abs() <= tol).all())


@pytest.mark.parametrize("layout", LAYOUTS, ids=list(LAYOUTS))
@pytest.mark.parametrize("ty", ref.TYPES)
def test_swiglu(ty, layout):
    import dense_gemm_09_gb300 as dg
    lay, dt = LAYOUTS[layout], ref.TYPES[ty]
    for cols in LENGTHS:
        rows = 5 if cols < 5000 else 2
        g, u = _x(rows, cols, dt, cols, 2.0, lay), _x(rows, cols, dt, cols + 9, layout=lay)
        q, qs, s = _out(rows, cols, lay)
        dg.swiglu_i8(g, u, q, s)
        torch.cuda.synchronize()
        y, delta = ref.swiglu_rows(g.cpu(), u.cpu())
        ref.check_rows(y, delta, q.cpu(), s.cpu())
        assert _untouched(q, qs, lay)


def test_swiglu_of_the_two_halves_of_one_matrix():
    import dense_gemm_09_gb300 as dg
    gu = _x(33, 2 * 520, torch.bfloat16, 4)
    q, _, s = _out(33, 520)
    dg.swiglu_i8(gu[:, :520], gu[:, 520:], q, s)
    y, delta = ref.swiglu_rows(gu[:, :520].cpu(), gu[:, 520:].cpu())
    ref.check_rows(y, delta, q.cpu(), s.cpu())


def test_swiglu_large_gates():
    # sigmoid's ends: the gate passes, or the product vanishes without a NaN
    import dense_gemm_09_gb300 as dg
    g = torch.tensor([[100.0, -100.0, 88.5, -88.5, -1e30, 1e30, 0.0, -0.0]], device="cuda")
    u = torch.tensor([[1e28, 1.0, 1.0, 1.0, 1.0, 0.0, 5.0, 5.0]], device="cuda")
    q, _, s = _out(1, 8)
    dg.swiglu_i8(g, u, q, s)
    assert q.cpu().tolist() == [[127, 0, 0, 0, 0, 0, 0, 0]]
    assert float(s[0]) == pytest.approx(1e30 / 127, rel=1e-6)


@pytest.mark.parametrize("layout", LAYOUTS, ids=list(LAYOUTS))
@pytest.mark.parametrize("ty", ref.TYPES)
def test_dequantize(ty, layout):
    import dense_gemm_09_gb300 as dg
    lay, dt = LAYOUTS[layout], ref.TYPES[ty]
    for cols in LENGTHS:
        rows = 5
        gen = torch.Generator().manual_seed(cols)
        q, _ = ref.pitched(rows, cols, torch.int8, *lay)
        q.copy_(torch.randint(-128, 128, (rows, cols), generator=gen, dtype=torch.int8))
        s = (torch.rand(rows, generator=gen) + 0.01).cuda()
        x, xs = ref.pitched(rows, cols, dt, *lay, fill=77)
        assert dg.dequantize_i8(q, s, x) is x
        want = (q.cpu().float() * s.cpu()[:, None]).to(dt)  # one FP32 product, one rounding
        assert torch.equal(x.cpu(), want)
        assert _untouched(x, xs, lay)


@pytest.mark.parametrize("cols", [5, 8, 700, 5000, 33000])
def test_rows_of_zeros_and_rows_that_are_not_finite(cols):
    import dense_gemm_09_gb300 as dg
    for dt in ref.TYPES.values():
        x = _x(6, cols, dt, 3)
        x[1] = 0.0
        x[2, cols - 1] = float("nan")
        x[3, 0] = float("inf")
        x[4, cols // 2] = float("-inf")
        for call in ("quantize", "norm", "swiglu"):
            q, _, s = _out(6, cols)
            if call == "quantize":
                dg.quantize_i8(x, q, s)
            elif call == "norm":
                dg.rmsnorm_i8(x, torch.ones(cols, dtype=dt, device="cuda"), q, s)
            else:
                dg.swiglu_i8(torch.ones_like(x), x, q, s)
            s, q = s.cpu(), q.cpu()
            assert torch.isnan(s).tolist() == [False, False, True, True, True, False], (call, dt)
            assert float(s[1]) == 0.0 and bool((q[1:5] == 0).all())
            assert bool((q[[0, 5]].abs().amax(1) == 127).all())
            v = torch.empty((6, cols), device="cuda")
            dg.dequantize_i8(q.cuda(), s.cuda(), v)
            assert torch.isnan(v).all(1).tolist() == [False, False, True, True, True, False]


def test_a_sum_of_squares_past_fp32_marks_its_row():
    import dense_gemm_09_gb300 as dg
    x = torch.full((2, 64), 1e20, device="cuda")
    x[1] = 1e10
    q, _, s = _out(2, 64)
    dg.rmsnorm_i8(x, torch.ones(64, device="cuda"), q, s)
    assert torch.isnan(s).tolist() == [True, False]
    assert bool((q[0] == 0).all()) and bool((q[1] == 127).all())


def test_rows_of_the_smallest_numbers_keep_their_steps():
    # 127 / a is past FP32's range here; subnormal rows too
    import dense_gemm_09_gb300 as dg
    steps = torch.arange(-127, 128, dtype=torch.float32)
    for e in (-120, -126, -130, -140):
        x = (steps.double() * 2.0 ** e).float().cuda()[None, :]
        q, _, s = _out(1, 255)
        dg.quantize_i8(x, q, s)
        assert torch.equal(q.cpu()[0], steps.to(torch.int8)), e
        assert float(s[0]) == pytest.approx(2.0 ** e, rel=1e-3, abs=2.0 ** -149)


def test_ties_go_to_the_even_step():
    import dense_gemm_09_gb300 as dg
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]], device="cuda")
    q, _, s = _out(1, 8)
    dg.quantize_i8(x, q, s)
    assert q.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -2, 126]] and float(s[0]) == 1.0


@pytest.mark.parametrize("cols", [100, 4096, 33001])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_rmsnorm_writes_h_over_an_input(cols, into):
    import dense_gemm_09_gb300 as dg
    x, r = _x(3, cols, torch.bfloat16, 1), _x(3, cols, torch.bfloat16, 2, 2.0)
    gamma = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    q0, _, s0 = _out(3, cols)
    H = torch.empty_like(x)
    dg.rmsnorm_i8(x, gamma, q0, s0, residual=r, H=H)
    q1, _, s1 = _out(3, cols)
    x1, r1 = x.clone(), r.clone()
    target = x1 if into == "x" else r1
    dg.rmsnorm_i8(x1, gamma, q1, s1, residual=r1, H=target)
    assert torch.equal(target, H) and torch.equal(q0, q1) and torch.equal(s0, s1)


def test_many_rows_and_empty_ones():
    import dense_gemm_09_gb300 as dg
    x = _x(70001, 16, torch.float16, 8)  # more rows than a grid dimension of 65535
    q, _, s = _out(70001, 16)
    dg.quantize_i8(x, q, s)
    ref.check_rows(x.cpu().double(), 0.0, q.cpu(), s.cpu())
    for shape in ((0, 16), (4, 0)):
        x = torch.empty(shape, device="cuda")
        q, s = torch.empty(shape, dtype=torch.int8, device="cuda"), torch.full((shape[0],), 3.0, device="cuda")
        dg.quantize_i8(x, q, s)
        dg.swiglu_i8(x, x, q, s)
        dg.rmsnorm_i8(x, torch.empty(shape[1], device="cuda"), q, s)
        dg.dequantize_i8(q, s, x)
        assert bool((s == 3.0).all())


def test_offsets_past_2_31_elements():
    # the last rows of a matrix of more than 2^31 elements (rows far apart)
    import dense_gemm_09_gb300 as dg
    pitch, rows = 1 << 27, 18
    x = torch.empty(rows * pitch, dtype=torch.float16, device="cuda").view(rows, pitch)[:, :300]
    q = torch.empty(rows * pitch, dtype=torch.int8, device="cuda").view(rows, pitch)[:, :300]
    x.copy_(_x(rows, 300, torch.float16, 6))
    s = torch.empty(rows, device="cuda")
    dg.quantize_i8(x, q, s)
    ref.check_rows(x.cpu().double(), 0.0, q.cpu(), s.cpu())
    v = x
    dg.dequantize_i8(q, s, v)
    assert torch.equal(v.cpu(), (q.cpu().float() * s.cpu()[:, None]).half())


def test_another_stream():
    import dense_gemm_09_gb300 as dg
    side = torch.cuda.Stream()
    x = _x(64, 4096, torch.bfloat16, 2)
    q, _, s = _out(64, 4096)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        dg.quantize_i8(x, q, s)
    q2, _, s2 = _out(64, 4096)
    dg.quantize_i8(x, q2, s2, stream=side)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
    ref.check_rows(x.cpu().double(), 0.0, q.cpu(), s.cpu())


def test_refusals():
    import dense_gemm_09_gb300 as dg
    x = torch.ones((4, 8), device="cuda")
    q, s = torch.empty((4, 8), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    g = torch.ones(8, device="cuda")
    with pytest.raises(TypeError):
        dg.quantize_i8(x.double(), q, s)
    with pytest.raises(TypeError):
        dg.quantize_i8(x, q.to(torch.uint8), s)
    with pytest.raises(ValueError):
        dg.quantize_i8(x, q[:, :7], s)
    with pytest.raises(ValueError):
        dg.quantize_i8(x, q, s[:3])
    with pytest.raises(ValueError):
        dg.quantize_i8(x.cpu(), q, s)
    with pytest.raises(ValueError):
        dg.quantize_i8(x.t(), torch.empty((8, 4), dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda"))
    with pytest.raises(TypeError):
        dg.rmsnorm_i8(x.half(), g.bfloat16(), q, s)
    with pytest.raises(ValueError):
        dg.rmsnorm_i8(x, g[:7], q, s)
    with pytest.raises(TypeError):
        dg.rmsnorm_i8(x, g, q, s, residual=x.half())
    with pytest.raises(ValueError):
        dg.rmsnorm_i8(x, g, q, s, H=x[:3])
    with pytest.raises(dg.DgemmError):
        dg.rmsnorm_i8(x, g, q, s, eps=-1.0)
    with pytest.raises(dg.DgemmError):
        dg.rmsnorm_i8(x, g, q, s, eps=float("nan"))
    with pytest.raises(TypeError):
        dg.swiglu_i8(x, x.half(), q, s)
    with pytest.raises(ValueError):
        dg.dequantize_i8(q, s, x[:, :4])
    with pytest.raises(ValueError, match="overlapping"):
        dg.quantize_i8(x[:1].expand(4, 8), q, s)
    with pytest.raises(ValueError):
        dg.quantize_i8(x[0], q[0], s)
    with pytest.raises(TypeError):
        dg.quantize_i8(None, q, s)
    with pytest.raises(ValueError):
        dg.quantize_i8(x, None, s)
