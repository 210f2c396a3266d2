"""gemm_f8_tn and gemm_f8_tn_experts on a GPU, against float64."""
import itertools

import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


# (variant, bn, split) of tune_f8_next; None: the library's choice
KERNELS = [None, (1, 0, 1), (2, 128, 1), (2, 256, 1), (3, 16, 1), (3, 16, 4), (3, 32, 2), (3, 64, 1), (3, 64, 8), (3, 64, 3),
           (4, 0, 4), (4, 0, 8)]


def tune(dg, kernel):
    if kernel is not None:
        dg.tune_f8_next(*kernel)


def held(q, pad=0, offset=0):
    """An 8-bit matrix at a pitch on 16-byte boundaries, or `pad` past it."""
    m, k = q.shape
    y, _ = ref.pitched(m, k, torch.uint8, -k % 16 + pad, offset)
    y.copy_(q.view(torch.uint8))
    return y.view(q.dtype)


def check(dg, m, n, k, kernel=None, ra=1, rb=128, fa="e4m3", fb="e4m3", out="bf16", bias=False, beta=0.0, pad=0, offset=0,
          cpad=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, sa = ref.operand(m, k, ra, ref.F8[fa], g)
    b, sb = ref.operand(n, k, rb, ref.F8[fb], g)
    t = ref.TYPES[out]
    c, store = ref.pitched(m, n, t, cpad, fill=5)
    c0 = torch.randn(m, n, generator=g, device="cuda").to(t)
    c.copy_(c0 if beta else torch.full_like(c0, float("nan")))  # (not read without beta)
    bi = torch.randn(n, generator=g, device="cuda") if bias else None
    tune(dg, kernel)
    assert dg.gemm_f8_tn(held(a, pad, offset), held(b, pad, offset), c, sa, sb, bias=bi, beta=beta) is c
    name = dg.last_kernel()
    want, mag = ref.product(a, sa, ra, b, sb, rb)
    tol = ref.product_error(k) * mag
    if bias:
        want, tol = want + bi.double(), tol + ref.E * (want.abs() + bi.double().abs() + tol)
    if beta:
        want, tol = want + beta * c0.double(), tol + ref.E * (want.abs() + (beta * c0.double()).abs() + tol)
    tol = tol + ref.U[t] * (want.abs() + tol) + ref.TINY[t]
    top = torch.finfo(t).max  # (what is past it becomes infinite)
    err = (c.double().clamp(-top, top) - want.clamp(-top, top)).abs()
    assert bool((err <= tol).all()), (name, (err / tol).max().item())
    c.fill_(5)
    assert bool((store == 5).all())
    assert dg.device_status() == dg.OK
    return name


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("k", [1, 16, 127, 128, 129, 400, 1024])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 128), (3, 129), (16, 256), (17, 100), (64, 64), (100, 384), (129, 127), (300, 513)])
def test_sizes(dg, m, n, k, kernel):
    check(dg, m, n, k, kernel, out="f32")
    check(dg, m, n, k, kernel, out="bf16", rb=1)


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("out", ref.TYPES)
@pytest.mark.parametrize("ra,rb", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_forms(dg, ra, rb, out, kernel):
    for (fa, fb), bias, beta in zip(itertools.product(ref.F8, ref.F8), (False, True, False, True), (0.0, 1.0, -0.5, 0.0)):
        check(dg, 150, 270, 333, kernel, ra, rb, fa, fb, out, bias, beta)
        check(dg, 7, 600, 640, kernel, ra, rb, fa, fb, out, bias, beta, cpad=3)


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (8, 8), (4, 4), (16, 0)])
@pytest.mark.parametrize("m,n,k", [(5, 70, 200), (130, 140, 384)])
def test_operands_off_16_bytes(dg, m, n, k, pad, offset):
    name = check(dg, m, n, k, pad=pad, offset=offset, bias=True, beta=0.5)
    if pad % 16 or offset % 16:
        assert "any" in name


@pytest.mark.parametrize("m,n,k", [(1, 8192, 4096), (33, 4096, 7168), (512, 1536, 2048), (1000, 1111, 4104), (2048, 2304, 512)])
def test_larger(dg, m, n, k):
    for out, rb in (("bf16", 128), ("f32", 1)):
        check(dg, m, n, k, out=out, rb=rb)


@pytest.mark.parametrize("kernel", [(2, 128, 1), (2, 256, 1), (3, 16, 4), (3, 64, 1)], ids=str)
@pytest.mark.parametrize("out", ref.TYPES)
@pytest.mark.parametrize("m,n,k,cpad", [(1, 33, 128, 7), (257, 1000, 200, 0), (130, 132, 640, 0), (1100, 2100, 300, 12), (2100, 4160, 400, 0),
                                        (300, 513, 256, 0)])
def test_the_old_c(dg, m, n, k, cpad, out, kernel):
    """Several tiles a CTA, edges inside a box, rows of C on 16 bytes and off them."""
    check(dg, m, n, k, kernel, 1, 1, "e5m2", "e4m3", out, True, 0.75, cpad=cpad)


# (clusters of eight, of as many tiles as there are groups of eight SMs, don't all fit the GPU)
@pytest.mark.parametrize("m,n,k", [(3, 2176, 7040), (9, 2304, 7040), (17, 2432, 4096), (20, 2304, 16384), (40, 1152, 4096)])
def test_few_rows_and_a_long_k_run_on_the_tensor_cores(dg, m, n, k):
    assert "any" not in check(dg, m, n, k)
    assert "any" not in check(dg, m, n, k, kernel=(3, 32, 8))


def test_no_k(dg):
    a, b = (torch.empty(r, 0, dtype=torch.float8_e4m3fn, device="cuda") for r in (5, 9))
    sa, sb = torch.empty(5, 0, device="cuda"), torch.empty(9, 0, device="cuda")
    bias, c = torch.randn(9, device="cuda"), torch.randn(5, 9, device="cuda")
    want = bias + 0.5 * c
    dg.gemm_f8_tn(a, b, c, sa, sb, bias=bias, beta=0.5)
    assert torch.equal(c, want)


def test_nothing_to_do(dg):
    for m, n in ((0, 5), (5, 0)):
        a, b = (torch.empty(r, 256, dtype=torch.float8_e4m3fn, device="cuda") for r in (m, n))
        c = torch.empty(m, n, device="cuda")
        assert dg.gemm_f8_tn(a, b, c, torch.empty(m, 2, device="cuda"), torch.empty(n, 2, device="cuda")) is c


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("m", [4, 200])
def test_a_block_that_is_not_finite_stays_in_its_row(dg, m, kernel):
    """A scale of NaN (what the quantisation leaves of such a block) reaches the row's
    products and no others; so does a NaN or an infinity held in 8 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    a, sa = ref.operand(m, 512, 1, torch.float8_e5m2, g)
    b, sb = ref.operand(300, 512, 128, torch.float8_e4m3fn, g)
    sa[1, 2] = float("nan")
    a.view(torch.uint8)[2, 5] = 0x7F  # NaN
    a.view(torch.uint8)[3, 7] = 0x7C  # infinity
    b.view(torch.uint8)[:, 7] = b.view(torch.uint8)[:, 7] & 0x80 | 0x38  # +-1
    c = torch.empty(m, 300, device="cuda")
    tune(dg, kernel)
    dg.gemm_f8_tn(a, b, c, sa, sb)
    fine = torch.isfinite(c)
    assert not bool(fine[1:4].any()) and bool(fine[0].all()) and bool(fine[4:].all())
    assert bool(c[1:3].isnan().all()) and bool(c[3].isinf().all())


# ---- rows sorted by expert

def check_experts(dg, offsets, n, k, kernel=None, rb=128, out="bf16", fa="e4m3", rows=None, pad=0, seed=0, cpad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    e = len(offsets) - 1
    m = max(offsets) if rows is None else rows
    a, sa = ref.operand(m, k, 1, ref.F8[fa], g)
    both = [ref.operand(n, k, rb, torch.float8_e4m3fn, g) for _ in range(e)]
    step = k + (-k % 16) + pad
    b = torch.zeros(e, n + 1, step, dtype=torch.uint8, device="cuda")[:, :n, :k]
    sb = torch.full((e, both[0][1].shape[0] + 1, ref.blocks(k)), float("nan"), device="cuda")[:, :-1]
    for i, (q, s) in enumerate(both):
        b[i].copy_(q.view(torch.uint8))
        sb[i].copy_(s)
    t = ref.TYPES[out]
    c, store = ref.pitched(m, n, t, cpad, fill=5)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    tune(dg, kernel)
    assert dg.gemm_f8_tn_experts(held(a), b.view(torch.float8_e4m3fn), c, sa, sb, off) is c
    name, at = dg.last_kernel(), 0
    for i in range(e):
        lo = at = max(at, min(max(offsets[i], 0), m))
        hi = max(lo, min(max(offsets[i + 1], 0), m))
        if hi > lo:
            want, mag = ref.product(a[lo:hi], sa[lo:hi], 1, *both[i], rb)
            tol = ref.product_error(k) * mag
            tol = tol + ref.U[t] * (want.abs() + tol) + ref.TINY[t]
            top = torch.finfo(t).max
            err = (c[lo:hi].double().clamp(-top, top) - want.clamp(-top, top)).abs()
            assert bool((err <= tol).all()), (name, i, (err / tol).max().item())
            c[lo:hi] = 5
    # rows of no expert, and what lies beside the rows
    assert bool((store == 5).all())
    assert dg.device_status() == dg.OK
    return name


OFFSETS = {"one": [0, 1], "empty": [0, 0, 0, 0], "some empty": [0, 0, 5, 5, 70, 71, 71], "ragged": [0, 130, 131, 400, 528, 529, 800],
           "gaps": [3, 10, 10, 260], "64 of one": list(range(65)), "tail": [0, 20, 50]}


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
@pytest.mark.parametrize("name", OFFSETS)
def test_experts(dg, name, kernel):
    o = OFFSETS[name]
    for n, k, rb, out in ((128, 128, 128, "f32"), (300, 520, 1, "bf16"), (520, 400, 128, "f16")):
        check_experts(dg, o, n, k, kernel, rb, out, rows=max(o) + 37)
        check_experts(dg, o, n, k, kernel, rb, out, "e5m2", rows=max(o) + 1, cpad=1)


def test_experts_off_16_bytes(dg):
    assert "any" in check_experts(dg, OFFSETS["ragged"], 100, 200, pad=1)


def test_bad_offsets_touch_nothing_else(dg):
    """Offsets out of order or out of range (no program means them) stay within the
    operands."""
    for o in ([0, 50, 20, 90], [-5, 10, 1000, 30], [2 ** 30, 0, 7], [200, 100, 0]):
        check_experts(dg, o, 130, 256, rows=120)


@pytest.mark.parametrize("kernel", KERNELS, ids=str)
def test_many_experts(dg, kernel):
    g = torch.Generator().manual_seed(2)
    counts = torch.randint(0, 4, (1024,), generator=g)
    check_experts(dg, [0] + counts.cumsum(0).tolist(), 140, 128, kernel)
