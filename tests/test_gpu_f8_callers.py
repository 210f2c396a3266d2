"""gemm_f8_tn and gemm_f8_tn_experts as several callers use them at once, and on operands
that share their memory."""
import threading

import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def operands(m, n, k, rb, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ref.operand(m, k, 1, torch.float8_e4m3fn, g) + ref.operand(n, k, rb, torch.float8_e4m3fn, g)


def test_kernels_side_by_side(dg):
    """CTA pairs, clusters that split K and dot products on streams of their own, from threads, give
    the bits that they give alone."""
    cases = []
    for m, n, k, rb, kernel in ((600, 2048, 1024, 128, (2, 256, 1)), (300, 1024, 2048, 1, (2, 128, 1)),
                                (20, 512, 4096, 128, (3, 32, 8)), (5, 4096, 1024, 1, (4, 0, 8))):
        a, sa, b, sb = operands(m, n, k, rb)
        dg.tune_f8_next(*kernel)
        want = dg.gemm_f8_tn(a, b, torch.empty(m, n, device="cuda"), sa, sb)
        cases.append((a, sa, b, sb, kernel, want))
    torch.cuda.synchronize()
    errors = []

    def work(a, sa, b, sb, kernel, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                c = torch.empty_like(want)
                wrong = torch.zeros((), dtype=torch.int64, device="cuda")
                for _ in range(50):
                    c.zero_()
                    dg.tune_f8_next(*kernel)
                    dg.gemm_f8_tn(a, b, c, sa, sb)
                    wrong += (c != want).sum()
                assert wrong.item() == 0
        except BaseException as e:  # noqa: BLE001
            errors.append((kernel, e))

    threads = [threading.Thread(target=work, args=case) for case in cases]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and dg.device_status() == dg.OK


def test_two_graphs_in_turn(dg):
    """Two captures of products that split K, replayed on two streams at once."""
    a, sa, b, sb = operands(9, 640, 4096, 128)
    want = dg.gemm_f8_tn(a, b, torch.empty(9, 640, device="cuda"), sa, sb)
    pairs = []
    for _ in range(2):
        c, graph = torch.zeros_like(want), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                dg.gemm_f8_tn(a, b, c, sa, sb, beta=-1.0)
                dg.gemm_f8_tn(a, b, c, sa, sb)
        pairs.append((graph, c, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, c, stream in pairs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for _, c, _ in pairs)


@pytest.mark.parametrize("m", [3, 200])
def test_a_matrix_times_itself(dg, m):
    a, sa, _, _ = operands(m, 1, 640, 1)
    c = dg.gemm_f8_tn(a, a, torch.empty(m, m, device="cuda"), sa, sa)
    want, mag = ref.product(a, sa, 1, a, sa, 1)
    assert bool(((c.double() - want).abs() <= (ref.product_error(640) + ref.E) * mag).all())


@pytest.mark.parametrize("n", [100, 384])
def test_experts_that_share_their_weights(dg, n):
    """A broadcast dimension of experts (strides of 0) is each expert's own copy."""
    a, sa, b, sb = operands(90, n, 256, 128)
    off = torch.tensor([0, 10, 10, 64, 90], dtype=torch.int32, device="cuda")
    c = torch.empty(90, n, device="cuda")
    dg.gemm_f8_tn_experts(a, b.expand(4, n, 256), c, sa, sb.expand(4, *sb.shape), off)
    want, mag = ref.product(a, sa, 1, b, sb, 128)
    assert bool(((c.double() - want).abs() <= (ref.product_error(256) + ref.E) * mag).all())


def test_experts_without_k(dg):
    """Sums of nothing: the experts' rows are 0, the others as they were."""
    a, sa = torch.empty(9, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(9, 0, device="cuda")
    b, sb = torch.empty(2, 5, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(2, 5, 0, device="cuda")
    c = torch.full((9, 5), 7.0, device="cuda")
    dg.gemm_f8_tn_experts(a, b, c, sa, sb, torch.tensor([1, 3, 6], dtype=torch.int32, device="cuda"))
    assert c[:, 0].tolist() == [7, 0, 0, 0, 0, 0, 7, 7, 7] and bool((c == c[:, :1]).all())


def test_a_layer_without_tokens(dg):
    from dense_gemm_09_gb300.moe import ExpertMlp
    w = [torch.randn(3, *s, device="cuda") for s in ((128, 256), (128, 256), (256, 128))]
    h = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    ids, weights = torch.empty(0, 2, dtype=torch.int64, device="cuda"), torch.empty(0, 2, device="cuda")
    assert ExpertMlp(*w)(h.clone(), ids, weights, h) is h
