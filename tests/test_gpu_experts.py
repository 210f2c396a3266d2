"""Tokens sorted by expert and back, on a GPU."""
import pytest
import torch

from tests import f8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg


def choices(tokens, top, e, seed=0, bad=0.0, dtype=torch.int32):
    """Expert numbers, of each token's choices mostly different ones; some out of range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    like = torch.rand(tokens, e, generator=g, device="cuda") + 0.5 * torch.rand(e, generator=g, device="cuda")
    ids = torch.topk(like, min(top, e), dim=1).indices
    if top > e:  # the same expert twice
        ids = torch.cat([ids, torch.randint(0, e, (tokens, top - e), generator=g, device="cuda")], 1)
    wrong = torch.tensor([-1, e, -2 ** 31, 2 ** 31 - 1], device="cuda")[torch.randint(0, 4, ids.shape, generator=g, device="cuda")]
    return torch.where(torch.rand(ids.shape, generator=g, device="cuda") < bad, wrong, ids).to(dtype).contiguous()


def sorted_plain(ids, e):
    """(offsets, position), pair by pair."""
    lists = [[] for _ in range(e)]
    flat = ids.reshape(-1).tolist()
    for i, x in enumerate(flat):
        if 0 <= x < e:
            lists[x].append(i)
    position, offsets = [-1] * len(flat), [0]
    for rows in lists:
        for r, i in enumerate(rows):
            position[i] = offsets[-1] + r
        offsets.append(offsets[-1] + len(rows))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(position, dtype=torch.int32).view(ids.shape)


def sort(dg, ids, e):
    offsets = torch.full((e + 1,), -7, dtype=torch.int32, device="cuda")
    position = torch.full(ids.shape, -7, dtype=torch.int32, device="cuda")
    dg.sort_by_expert(ids, offsets, position)
    return offsets, position


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top,e,bad", [(1, 1, 1, 0), (1, 8, 64, 0), (16, 8, 64, 0.25), (33, 3, 5, 0), (100, 6, 4, 0.1),
                                              (7, 1, 1024, 0), (1024, 8, 128, 0), (1025, 8, 60, 0.3), (4099, 6, 256, 0.01),
                                              (20000, 8, 1024, 0), (70000, 4, 8, 0.5), (300, 2, 16, 1.0)])
def test_sort(dg, tokens, top, e, bad, dtype):
    ids = choices(tokens, top, e, bad=bad, dtype=dtype)
    if dtype == torch.int64 and bad:
        ids[0, 0] = 2 ** 32 + 1  # not expert 1
    offsets, position = sort(dg, ids, e)
    wo, wp = sorted_plain(ids, e)
    assert torch.equal(offsets.cpu(), wo) and torch.equal(position.cpu(), wp)


def test_sort_of_nothing(dg):
    for shape in ((0, 4), (4, 0)):
        offsets, _ = sort(dg, torch.empty(shape, dtype=torch.int32, device="cuda"), 5)
        assert offsets.tolist() == [0] * 6


@pytest.mark.parametrize("tokens", [20, 257])
@pytest.mark.parametrize("e", [1, 2, 3, 31, 32, 127, 128, 129, 1023])
def test_padding_is_no_expert(dg, tokens, e):
    """Numbers next to the range, and of every bit, among those of each expert."""
    g = torch.Generator().manual_seed(e)
    ids = torch.randint(0, e, (tokens, 8), generator=g, dtype=torch.int32)
    ids[:, ::3] = torch.tensor([-1, e, 2 * e, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)[
        torch.randint(0, 5, ids[:, ::3].shape, generator=g)].to(torch.int32)
    wo, wp = sorted_plain(ids.cuda(), e)
    offsets, position = sort(dg, ids.cuda(), e)
    assert torch.equal(offsets.cpu(), wo) and torch.equal(position.cpu(), wp)


def test_sort_of_one_expert(dg):
    """Every pair goes to the last expert: the longest run of equal numbers."""
    ids = torch.full((5000, 4), 63, dtype=torch.int32, device="cuda")
    offsets, position = sort(dg, ids, 64)
    assert torch.equal(position.view(-1), torch.arange(20000, dtype=torch.int32, device="cuda"))
    assert offsets.tolist() == [0] * 64 + [20000]


MOVES = [(1, 1, 1, 1), (1, 8, 64, 4096), (16, 8, 64, 129), (33, 3, 5, 1000), (100, 6, 4, 2056), (257, 2, 16, 520), (40, 20, 32, 136),
         (3000, 4, 8, 256), (5, 4, 8, 40000)]


def setup(dg, tokens, top, e, k, t, pad, offset, extra=3, bad=0.2):
    ids = choices(tokens, top, e, bad=bad)
    _, position = sort(dg, ids, e)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, xs = ref.pitched(tokens, k, t, pad, offset)
    x.copy_(torch.randn(tokens, k, generator=g, device="cuda"))
    y, ys = ref.pitched(tokens * top + extra, k, t, pad, offset, fill=5)
    return ids, position, x, xs, y, ys, g


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (1, 0), (0, 3)])
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("tokens,top,e,k", MOVES)
def test_gather(dg, tokens, top, e, k, dtype, pad, offset):
    ids, position, x, _, y, ys, _ = setup(dg, tokens, top, e, k, ref.TYPES[dtype], pad, offset)
    x.view(-1, k)[0, 0] = float("nan")
    assert dg.gather_by_expert(x, position, y) is y
    kept = position.view(-1) >= 0
    rows, src = position.view(-1)[kept].long(), torch.arange(tokens, device="cuda").repeat_interleave(top)[kept]
    assert torch.equal(y[rows].nan_to_num(77.0), x[src].nan_to_num(77.0))
    y[rows] = 5
    assert bool((ys == 5).all())


@pytest.mark.parametrize("f8", ref.F8)
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("tokens,top,e,k", MOVES)
def test_gather_f8(dg, tokens, top, e, k, dtype, f8):
    for pad, offset in ((0, 0), (1, 3)):
        ids, position, x, _, _, _, _ = setup(dg, tokens, top, e, k, ref.TYPES[dtype], pad, offset)
        q, store = ref.pitched(tokens * top + 3, k, torch.uint8, pad, offset, fill=99)
        s = torch.full((tokens * top + 3, ref.blocks(k)), 7.0, device="cuda")
        dg.gather_by_expert_f8(x, position, q.view(ref.F8[f8]), s)
        want, ws = ref.quantized(x.float(), 1, ref.F8[f8])
        kept = position.view(-1) >= 0
        rows, src = position.view(-1)[kept].long(), torch.arange(tokens, device="cuda").repeat_interleave(top)[kept]
        assert torch.equal(q[rows], want.view(torch.uint8)[src]) and torch.equal(s[rows], ws[src])
        q[rows] = 99
        s[rows] = 7.0
        assert bool((store == 99).all()) and bool((s == 7.0).all())


def sums(y, position, weights, tokens, top):
    """(sum, sum of magnitudes) over each token's rows in float64."""
    at = position.long().clamp(min=0)
    part = torch.where(position[..., None] >= 0, y.double()[at] * (1.0 if weights is None else weights.double()[..., None]), 0.0)
    return part.sum(1), part.abs().sum(1)


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 3)])
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("tokens,top,e,k", MOVES)
def test_combine(dg, tokens, top, e, k, dtype, pad, offset):
    t = ref.TYPES[dtype]
    ids, position, x, xs, y, _, g = setup(dg, tokens, top, e, k, t, pad, offset)
    y.copy_(torch.randn(y.shape, generator=g, device="cuda"))
    weights = torch.rand(tokens, top, generator=g, device="cuda")
    weights[position < 0] = float("nan")  # (of pairs without a row)
    for w, beta in ((weights, 0.0), (weights, 1.0), (None, -0.5)):
        x0 = x.clone()
        if not beta:
            x.fill_(float("nan"))  # (not read)
        assert dg.combine_experts(y, position, w, x, beta=beta) is x
        want, mag = sums(y, position, w, tokens, top)
        if beta:
            want, mag = want + beta * x0.double(), mag + (beta * x0.double()).abs()
        # a rounding for each row's addition
        tol = (top + 1) * ref.E * mag
        tol = tol + ref.U[t] * (want.abs() + tol) + ref.TINY[t]
        assert bool(((x.double() - want).abs() <= tol).all())
        x.copy_(x0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("tokens,top,e,k", MOVES)
def test_combine_grad(dg, tokens, top, e, k, dtype, in_place):
    t = ref.TYPES[dtype]
    for pad, offset in ((0, 0), (1, 3)):
        ids, position, dx, _, y, ys, g = setup(dg, tokens, top, e, k, t, pad, offset)
        kept = position >= 0
        rows, src = position[kept].long(), torch.arange(tokens, device="cuda")[:, None].expand(-1, top)[kept]
        y[rows] = torch.randn(rows.numel(), k, generator=g, device="cuda").to(t)
        y0 = y.clone()
        weights, dw = torch.rand(tokens, top, generator=g, device="cuda"), torch.full((tokens, top), 9.0, device="cuda")
        dy, dys = (y, ys) if in_place else ref.pitched(y.shape[0], k, t, pad + 8, offset, fill=5)
        dg.combine_experts_grad(dx, y, position, weights, dy, dw)
        assert not bool(dw[~kept].any())
        want, mag = ((f(dx.double()[src]) * f(y0.double()[rows])).sum(1) for f in (lambda v: v, torch.abs))
        # each thread adds up at most k / 256 + 8 products in order, then 5 + 8 levels
        assert bool(((dw[kept].double() - want).abs() <= (k / 256 + 8 + 14) * ref.E * mag).all())
        # the product in FP32, then the type: torch rounds twice alike
        assert torch.equal(dy[rows], (weights[kept][:, None] * dx.float()[src]).to(t))
        dy[rows] = 5
        assert bool((dys == 5).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_positions_are_skipped(dg, dtype):
    """Rows past the sorted rows (of a caller with fewer of them) move nothing."""
    t = ref.TYPES[dtype]
    position = torch.tensor([[0, 7], [5, -3], [6, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    x, y = torch.randn(3, 264, device="cuda").to(t), torch.full((6, 264), 5.0, device="cuda", dtype=t)
    dg.gather_by_expert(x, position, y)
    assert torch.equal(y[0], x[0]) and torch.equal(y[5], x[1]) and bool((y[1:5] == 5).all())
    q, s = torch.zeros(6, 264, dtype=torch.float8_e4m3fn, device="cuda"), torch.full((6, 3), 7.0, device="cuda")
    dg.gather_by_expert_f8(x, position, q, s)
    assert bool((s[1:5] == 7).all()) and bool((s[0] < 7).all())
    w, dw = torch.rand(3, 2, device="cuda"), torch.empty(3, 2, device="cuda")
    out = torch.empty_like(x)
    dg.combine_experts(y, position, w, out)
    assert torch.equal(out[0], (w[0, 0] * y[0].float()).to(t)) and not bool(out[2].any())
    dy = torch.full_like(y, 5.0)
    dg.combine_experts_grad(x, y, position, w, dy, dw)
    assert bool((dy[1:5] == 5).all()) and dw[0, 1] == 0 and not bool(dw[2].any())


def test_gradients_against_differences(dg):
    """d/dy and d/dw of <g, combine(y, w)> and d/dx of <h, gather(x)>, by differences
    (both are linear in each of their inputs, so a difference is the derivative)."""
    tokens, top, e, k = 12, 4, 8, 136
    ids, position, x, _, y, _, g = setup(dg, tokens, top, e, k, torch.float32, 0, 0)
    w = torch.rand(tokens, top, generator=g, device="cuda")
    y.copy_(torch.randn(y.shape, generator=g, device="cuda"))
    up = torch.randn(tokens, k, generator=g, device="cuda")
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    dg.combine_experts_grad(up, y, position, w, dy, dw)

    def loss(y, w):
        return (dg.combine_experts(y, position, w, torch.empty_like(up)).double() * up.double()).sum()

    for _ in range(4):
        ty, tw = torch.randn(y.shape, generator=g, device="cuda"), torch.randn(w.shape, generator=g, device="cuda")
        size = ((y.abs() + ty.abs()).double().sum() * up.abs().double().max()).item()
        tol = 2 * (top + 20) * ref.E * size
        assert abs((loss(y + ty, w) - loss(y, w)) - (dy.double() * ((y + ty) - y).double()).sum()) <= tol
        assert abs((loss(y, w + tw) - loss(y, w)) - (dw.double() * ((w + tw) - w).double()).sum()) <= 4 * tol
    h = torch.randn(y.shape, generator=g, device="cuda")
    dx = dg.combine_experts(h, position, None, torch.empty_like(x))
    moved = dg.gather_by_expert(x, position, torch.zeros_like(y))
    left, right = (moved.double() * h.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(left - right) <= (top + 1) * ref.E * (moved.abs() * h.abs()).double().sum()
