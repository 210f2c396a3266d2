"""The 8-bit floating-point kernels' failure detection and bounds checks on a GPU: a stalled
tensor-core launch ends by itself with DGEMM_ERR_TIMEOUT and leaves the context usable, also
where its waits run out with loads in flight; in the checked build no index that a kernel
computes leaves its extent; operands past 2^31 elements and bytes."""
import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu

# (variant, bn, split), M, N: pairs of either kind, single CTAs, clusters that share a tile;
# several tiles a CTA
KINDS = [((2, 128, 1), 300, 700), ((2, 256, 1), 300, 700), ((2, 256, 1), 4096, 8192), ((3, 16, 1), 12, 1000), ((3, 16, 1), 12, 32768),
         ((3, 16, 8), 16, 400), ((3, 32, 4), 30, 700), ((3, 64, 1), 60, 1000), ((3, 64, 3), 60, 1000)]


def operands(m, n, k, rb=128):
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa = ref.operand(m, k, 1, torch.float8_e4m3fn, g)
    b, sb = ref.operand(n, k, rb, torch.float8_e4m3fn, g)
    return a, b, sa, sb


@pytest.mark.parametrize("k", [128, 384, 2048])
@pytest.mark.parametrize("tune,m,n", KINDS, ids=["%d-%d-%d_%dx%d" % (t + (m, n)) for t, m, n in KINDS])
def test_waits_that_run_out_at_once(tune, m, n, k):
    import dense_gemm_09_gb300 as dg
    a, b, sa, sb = operands(m, n, k)
    c, want = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    dg.tune_f8_next(*tune)
    dg.gemm_f8_tn(a, b, want, sa, sb)
    assert dg.device_status(clear=True) == dg.OK
    name = dg.last_kernel()
    for limit in (0, 1, 1000, 3000, 20000, 2_000_000):
        dg.tune_f8_next(*tune)
        dg.test_inject_stall(limit)
        dg.gemm_f8_tn(a, b, c, sa, sb)
        assert dg.last_kernel() == name
        st = dg.device_status(clear=True)  # synchronises
        assert st == dg.ERR_TIMEOUT, dg.status_string(st)
        dg.tune_f8_next(*tune)
        dg.gemm_f8_tn(a, b, c.zero_(), sa, sb)
        assert dg.device_status(clear=True) == dg.OK
        assert torch.equal(c, want)


@pytest.mark.parametrize("m,n", [(300, 700), (2048, 8192)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_waits_that_run_out_with_the_old_c_on_its_way(m, n, out):
    import dense_gemm_09_gb300 as dg
    a, b, sa, sb = operands(m, n, 384)
    c0 = torch.randn(m, n, device="cuda").to(out)
    want = c0.clone()
    dg.tune_f8_next(2, 128, 1)
    dg.gemm_f8_tn(a, b, want, sa, sb, beta=-1.5)
    assert dg.device_status(clear=True) == dg.OK
    for limit in (0, 1, 1000, 3000, 20000):
        dg.tune_f8_next(2, 128, 1)
        dg.test_inject_stall(limit)
        dg.gemm_f8_tn(a, b, c0.clone(), sa, sb, beta=-1.5)
        assert dg.device_status(clear=True) == dg.ERR_TIMEOUT
        c = c0.clone()
        dg.tune_f8_next(2, 128, 1)
        dg.gemm_f8_tn(a, b, c, sa, sb, beta=-1.5)
        assert dg.device_status(clear=True) == dg.OK and torch.equal(c, want)


def test_a_stalled_launch_by_expert():
    import dense_gemm_09_gb300 as dg
    a, _, sa, _ = operands(600, 1, 512)
    b = torch.randn(5, 300, 512, device="cuda").to(torch.float8_e4m3fn)
    sb = torch.rand(5, 3, 4, device="cuda")
    off = torch.tensor([0, 100, 100, 411, 500, 600], dtype=torch.int32, device="cuda")
    for tune in ((2, 256, 1), (2, 128, 1), (3, 64, 1)):
        c, want = torch.empty(600, 300, device="cuda"), torch.empty(600, 300, device="cuda")
        dg.tune_f8_next(*tune)
        dg.gemm_f8_tn_experts(a, b, want, sa, sb, off)
        for limit in (1, 20000):
            dg.tune_f8_next(*tune)
            dg.test_inject_stall(limit)
            dg.gemm_f8_tn_experts(a, b, c, sa, sb, off)
            assert dg.device_status(clear=True) == dg.ERR_TIMEOUT
        dg.tune_f8_next(*tune)
        dg.gemm_f8_tn_experts(a, b, c.zero_(), sa, sb, off)
        assert dg.device_status(clear=True) == dg.OK and torch.equal(c, want)


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


def passed(dg):
    lib = dg.lib()
    st, site = lib.dgemm_device_status(0), lib.dgemm_check_site()
    lib.dgemm_device_status(1)
    assert st == dg.OK and site == 0, "%s at site %d" % (dg.status_string(st), site)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (7, 129, 130), (16, 300, 1000), (64, 640, 256), (300, 257, 520), (513, 1030, 384)])
def test_checked_products(checked, m, n, k):
    from tests.test_gpu_f8_gemm import KERNELS, check
    for kernel in KERNELS:
        check(checked, m, n, k, kernel, out="f32")
        check(checked, m, n, k, kernel, rb=1, out="bf16", bias=True, beta=0.5, cpad=1)
    check(checked, m, n, k, pad=1)
    passed(checked)


def test_checked_products_by_expert(checked):
    from tests.test_gpu_f8_gemm import KERNELS, OFFSETS, check_experts
    for kernel in KERNELS:
        for o in OFFSETS.values():
            check_experts(checked, o, 300, 400, kernel, rows=max(o) + 7)
            check_experts(checked, o, 130, 256, kernel, 1, "f32", cpad=1)
    passed(checked)


def test_checked_rows_and_experts(checked):
    from tests import test_gpu_experts as te
    from tests import test_gpu_f8_rows as tr
    for form in ("rows", "blocks", "transposed"):
        for t in ref.TYPES.values():
            for m, k in tr.SHAPES[:9]:
                tr.check_quantize(checked, tr.values(m, k, t), form, torch.float8_e4m3fn)
            x, _ = ref.pitched(200, 333, t, 1, 1)
            x.copy_(tr.values(200, 333, t))
            tr.check_quantize(checked, x, form, torch.float8_e5m2, 3, 1)
    for args in te.MOVES[:6]:
        te.test_gather(checked, *args, "bf16", 0, 0)
        te.test_gather_f8(checked, *args, "f32", "e4m3")
        te.test_combine(checked, *args, "f16", 1, 3)
        te.test_combine_grad(checked, *args, "bf16", False)
    te.test_sort(checked, 4099, 6, 256, 0.01, torch.int32)
    passed(checked)


# ---- past 2^31

def test_rows_past_2_31():
    """Offsets past 2^31 elements, and 2^32 bytes, of the tokens, the sorted rows and the scales."""
    import dense_gemm_09_gb300 as dg
    k, tokens, top = 65536, 20000, 2  # 40000 sorted rows: 2.6e9 elements
    x = torch.empty(tokens, k, dtype=torch.bfloat16, device="cuda").normal_()
    position = torch.randperm(tokens * top, device="cuda").to(torch.int32).view(tokens, top)
    y = torch.empty(tokens * top, k, dtype=torch.bfloat16, device="cuda")
    dg.gather_by_expert(x, position, y)
    look = torch.cat([torch.arange(4), torch.arange(tokens - 4, tokens), torch.randint(0, tokens, (40,))])
    for t in look.tolist():
        for j in range(top):
            assert torch.equal(y[position[t, j].item()], x[t])
    w = torch.rand(tokens, top, device="cuda")
    dw, out = torch.empty(tokens, top, device="cuda"), torch.empty_like(x)
    dg.combine_experts(y, position, w, out)
    for t in look.tolist():
        # (one rounding of each product and sum: float64 holds a product of FP32 numbers exactly)
        first = (w[t, 0] * x[t].float()).double()
        assert torch.equal(out[t], (w[t, 1].double() * x[t].double() + first).float().bfloat16())
    del out
    q = torch.empty(tokens * top, k, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(tokens * top, k // 128, device="cuda")
    dg.gather_by_expert_f8(x, position, q, s)
    want, ws = ref.quantized(x[look.cuda()].float(), 1, torch.float8_e4m3fn)
    at = position[look.cuda(), 1].long()
    assert torch.equal(q.view(torch.uint8)[at], want.view(torch.uint8)) and torch.equal(s[at], ws)
    dg.combine_experts_grad(x, y, position, w, y, dw)  # in place
    for t in look.tolist():
        assert torch.equal(y[position[t, 1].item()], (w[t, 1] * x[t].float()).bfloat16())
    dg.dequantize_f8(q, s, y)
    assert torch.equal(y[at], (want.float() * ref.spread(ws, 1, *want.shape)).bfloat16())


def test_products_past_2_31():
    import dense_gemm_09_gb300 as dg
    m, n, k = 70000, 256, 32768  # A: 2.3e9 bytes
    a = torch.randint(0, 120, (m, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sa = torch.rand(m, k // 128, device="cuda")
    b, sb = ref.operand(n, k, 128, torch.float8_e4m3fn, torch.Generator(device="cuda").manual_seed(0))
    look = torch.tensor([0, 1, 40000, 65535, 65536, 69998, 69999], device="cuda")
    want, mag = ref.product(a.view(torch.uint8)[look].view(torch.float8_e4m3fn), sa[look], 1, b, sb, 128)
    for tune in ((0, 0, 1), (2, 128, 1), (3, 64, 1)):
        c = torch.empty(m, n, device="cuda")
        dg.tune_f8_next(*tune)
        dg.gemm_f8_tn(a, b, c, sa, sb)
        assert bool(((c[look].double() - want).abs() <= (ref.product_error(k) + ref.E) * mag).all())
    # channels past 2^31 bytes of weights, as experts
    w = a.view(7, 10000, k)
    sw = torch.rand(7, ref.blocks(10000), k // 128, device="cuda")
    off = torch.tensor([0, 10, 20, 30, 40, 50, 60, 256], dtype=torch.int32, device="cuda")
    c = torch.empty(n, 10000, device="cuda")
    sbr = sb.repeat_interleave(128, 0)[:n].contiguous()
    dg.gemm_f8_tn_experts(b, w, c, sbr, sw, off)
    want, mag = ref.product(b[60:], sbr[60:], 1, w[6], sw[6], 128)
    assert bool(((c[60:].double() - want).abs() <= (ref.product_error(k) + ref.E) * mag).all())
    # C past 2^31 elements
    m, n, k = 50000, 50000, 256
    a, sa = ref.operand(m, k, 1, torch.float8_e4m3fn, torch.Generator(device="cuda").manual_seed(1))
    b, sb = ref.operand(n, k, 128, torch.float8_e4m3fn, torch.Generator(device="cuda").manual_seed(2))
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    dg.gemm_f8_tn(a, b, c, sa, sb)
    want, mag = ref.product(a[-300:], sa[-300:], 1, b, sb, 128)
    tol = ref.product_error(k) * mag
    assert bool(((c[-300:].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
