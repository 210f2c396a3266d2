"""The 8-bit floating-point calls and the calls on tokens by expert together, as programs use
them: a mixture-of-experts layer, a linear layer's training step; on other streams, in graphs,
and from threads."""
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


def moe_inputs(tokens, top=3, e=6, hidden=384, ffn=256, seed=0, padded=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [torch.randn(e, ffn, hidden, generator=g, device="cuda") / hidden ** 0.5 for _ in range(2)]
    w.append(torch.randn(e, hidden, ffn, generator=g, device="cuda") / ffn ** 0.5)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    best, ids = torch.topk(torch.randn(tokens, e, generator=g, device="cuda"), top, dim=1)
    if padded:
        ids[-padded:] = -1
    return w, x, ids.contiguous(), torch.softmax(best, 1)


def moe_exact(layer, x, ids, weights, h):
    """The layer step by step on the quantised values that it holds, in float64 (and the sum of
    magnitudes of what is added up last)."""
    q, s = ref.quantized(x.float(), 1, torch.float8_e4m3fn)
    xq = q.double() * ref.spread(s.double(), 1, *q.shape)
    out, mag = h.double(), h.double().abs()
    e, n1, k1 = layer.w1.shape
    _, n2, k2 = layer.w2.shape
    for i in range(e):
        token, choice = torch.nonzero(ids == i, as_tuple=True)
        w1 = layer.w1[i].double() * ref.spread(layer.s1[i].double(), 128, n1, k1)
        w2 = layer.w2[i].double() * ref.spread(layer.s2[i].double(), 128, n2, k2)
        gu = (xq[token] @ w1.t()).to(torch.bfloat16).float()
        g, u = gu[:, :n1 // 2], gu[:, n1 // 2:]
        q, s = ref.quantized(g / (1 + torch.exp(-g)) * u, 1, torch.float8_e4m3fn)
        y = (q.double() * ref.spread(s.double(), 1, *q.shape)) @ w2.t()
        y = y * weights[token, choice].double()[:, None]
        out.index_add_(0, token, y)
        mag.index_add_(0, token, y.abs())
    return out, mag


# A step of the layer rounds twice where the exact form may round the other way: gu to bfloat16
# (2^-8) and the gated values to 8 bits (a half step is 2^-4; a flip moves one by a step, 2^-3).
# Both happen for the few values whose FP32 sums lie next to a border; the norm of the
# difference stays below one step of bfloat16 of the output and what 1 value in 100 that flips
# by 2^-3 adds: sqrt(1/100) 2^-3 = 2^-6.3, with 2^-8 below 2^-5.
LAYER_TOL = 2.0 ** -5


def near(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("tokens,padded", [(1, 0), (7, 2), (64, 0), (500, 100)])
def test_moe_layer(dg, tokens, padded):
    from dense_gemm_09_gb300.moe import ExpertMlp
    w, x, ids, weights = moe_inputs(tokens, padded=padded)
    layer = ExpertMlp(*w)
    h0 = torch.randn(x.shape, device="cuda").bfloat16()
    h = layer(x, ids, weights, h0.clone())
    want, _ = moe_exact(layer, x, ids, weights, h0)
    assert near(h.double() - h0.double(), want - h0.double()) < LAYER_TOL + 2.0 ** -8 * (h0.double().norm() / (want - h0.double()).norm()).item()
    if padded:
        assert torch.equal(h[-padded:], h0[-padded:])
    assert dg.device_status() == dg.OK


def test_moe_layer_all_padding(dg):
    from dense_gemm_09_gb300.moe import ExpertMlp
    w, x, ids, weights = moe_inputs(9, padded=9)
    h0 = torch.randn(x.shape, device="cuda").bfloat16()
    assert torch.equal(ExpertMlp(*w)(x, ids, weights, h0.clone()), h0)


def test_moe_layer_in_a_graph_streams_and_threads(dg):
    """The same layer captured (and replayed with new inputs), on side streams and from threads at
    once gives what it gives alone, to the bit."""
    from dense_gemm_09_gb300.moe import ExpertMlp
    w, x, ids, weights = moe_inputs(40)
    layer = ExpertMlp(*w)
    cases = []
    for seed in range(4):
        _, x, ids, weights = moe_inputs(40, seed=seed)
        cases.append((x, ids, weights, layer(x, ids, weights, torch.zeros_like(x))))
    torch.cuda.synchronize()
    # captured on its own buffers
    sx, si, sw, sh = (t.clone() for t in cases[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(sx, si, sw, sh)
    for x, ids, weights, want in cases:
        sx.copy_(x), si.copy_(ids), sw.copy_(weights), sh.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sh, want)
    # on streams of their own, from threads, beside replays
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                x, ids, weights, _ = cases[i]
                for _ in range(20):
                    got[i] = layer(x, ids, weights, torch.zeros_like(x))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    for _ in range(20):
        sh.zero_()
        graph.replay()
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(g, c[3]) for g, c in zip(got, cases))
    assert torch.equal(sh, cases[3][3])
    assert dg.device_status() == dg.OK


def test_the_command_runs(dg, monkeypatch, capsys):
    from dense_gemm_09_gb300 import moe
    monkeypatch.setattr("sys.argv", ["moe", "--hidden", "512", "--ffn", "256", "--experts", "8", "--top", "2", "--tokens", "1", "33"])
    moe.main()
    lines = [line for line in capsys.readouterr().out.splitlines() if "tokens:" in line]
    assert len(lines) == 2


@pytest.mark.parametrize("tokens,k,n", [(1, 128, 128), (100, 256, 384), (777, 520, 650)])
def test_a_linear_layers_training_step(dg, tokens, k, n):
    """y = x W^T, dx = dy W, dW += dy^T x, from one quantisation of W and the transposed ones of x
    and dy, each against float64 on the quantised values, and the whole against FP32."""
    g = torch.Generator(device="cuda").manual_seed(1)
    f8, f5 = torch.float8_e4m3fn, torch.float8_e5m2
    x, dy = torch.randn(tokens, k, generator=g, device="cuda"), torch.randn(tokens, n, generator=g, device="cuda")
    w, grad0 = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5, torch.randn(n, k, generator=g, device="cuda")

    def quant(t, rows, dtype, transposed=False):
        m, c = (t.shape[1], t.shape[0]) if transposed else t.shape
        q = torch.empty(m, -(-c // 16) * 16, dtype=dtype, device="cuda")[:, :c]
        return dg.quantize_f8(t, q, torch.empty(-(-m // rows), ref.blocks(c), device="cuda"), transposed=transposed)

    def held(q, s, rows):
        return q.double() * ref.spread(s.double(), rows, *q.shape)

    (qx, sx), (qw, sw), (qd, sd) = quant(x, 1, f8), quant(w, 128, f8), quant(dy, 1, f5)
    (qxt, sxt), (qdt, sdt) = quant(x, 1, f8, True), quant(dy, 1, f5, True)
    y, dx = torch.empty(tokens, n, device="cuda"), torch.empty(tokens, k, device="cuda")
    dw = grad0.clone()
    dg.gemm_f8_tn(qx, qw, y, sx, sw)
    wt = torch.empty(k, -(-n // 16) * 16, dtype=f8, device="cuda")[:, :n]
    wt.copy_(qw.t())  # W's blocks transpose with their scales
    dg.gemm_f8_tn(qd, wt, dx, sd, sw.t())
    dg.gemm_f8_tn(qdt, qxt, dw, sdt, sxt, beta=1.0)
    X, W, D = held(qx, sx, 1), held(qw, sw, 128), held(qd, sd, 1)
    Xt, Dt = held(qxt, sxt, 1), held(qdt, sdt, 1)
    for got, a, b, add, depth in ((y, X, W.t(), 0.0, k), (dx, D, W, 0.0, n), (dw, Dt, Xt.t(), grad0.double(), tokens)):
        want = a @ b + add
        tol = (ref.product_error(depth) + 2 * ref.E) * (a.abs() @ b.abs() + (add.abs() if torch.is_tensor(add) else 0.0))
        assert bool(((got.double() - want).abs() <= tol + ref.U[torch.float32] * want.abs()).all())
    # the whole: a half step of e4m3 is 2^-4 of a value, of e5m2 2^-3; in norm, independent errors
    # of at most that size on either factor: below sqrt(2) 2^-3
    for got, want in ((y, x @ w.t()), (dx, dy @ w), (dw - grad0, dy.t() @ x)):
        assert near(got, want.double()) < 2.0 ** -2.5


def test_side_stream_argument(dg):
    """stream= takes a Stream or a handle; the work is ordered there."""
    s = torch.cuda.Stream()
    x = torch.randn(300, 512, device="cuda").bfloat16()
    q, sc, v = torch.empty(300, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(300, 4, device="cuda"), torch.empty_like(x)
    torch.cuda.synchronize()
    dg.quantize_f8(x, q, sc, stream=s)
    dg.dequantize_f8(q, sc, v, stream=s.cuda_stream)
    s.synchronize()
    want, ws = ref.quantized(x.float(), 1, torch.float8_e4m3fn)
    assert torch.equal(v, (want.float() * ref.spread(ws, 1, 300, 512)).bfloat16())


def test_a_chain_of_launches_sees_the_last_ones_writes(dg):
    """Each call of a long chain on one stream reads what the call before it wrote."""
    t, k = 64, 512
    w = torch.eye(k, device="cuda")
    qw, sw = dg.quantize_f8(w, torch.empty(k, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, 4, device="cuda"))
    x = torch.randn(t, k, device="cuda").bfloat16()
    q, s = torch.empty(t, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(t, 4, device="cuda")
    dg.quantize_f8(x, q, s)
    v0 = dg.dequantize_f8(q, s, torch.empty_like(x, dtype=torch.float32)).clone()
    c, c2 = torch.empty(t, k, device="cuda"), torch.empty(t, k, device="cuda")
    for _ in range(50):  # identity, again and again: values of an 8-bit block keep their largest and so their steps
        dg.gemm_f8_tn(q, qw, c, s, sw)
        q.zero_()
        dg.quantize_f8(c, q, s)
        dg.gemm_f8_tn(q, qw, c2, s, sw)
    # the scale 448/448 ... of the identity is 1/448 with Q = 448: two roundings a pass
    assert near(c2, v0.double()) < 100 * 3 * 2.0 ** -23 + 1e-12
