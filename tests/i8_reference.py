"""Plain 64-bit forms of the 8-bit operators, and how far FP32 may be off them.

The formulas (include/dgemm.h), in float64 on the stored inputs.  Tolerances
are derived from the roundings each call may make:
  * unit roundoffs U of the output types (2^-24, 2^-11, 2^-8);
  * a row value y: up to `delta` relative, from the FP32 operations before it;
  * an int8 step may differ from the exact quotient y / scale by half a step
    plus 127 * (delta + the scale's and the quotient's own roundings).
"""
from __future__ import annotations

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# the smallest spacing of a type: what a subnormal result may be off by
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
E = 2.0 ** -24


def pitched(rows, cols, dtype, pad=0, offset=0, fill=0, device="cuda"):
    """(matrix, storage): rows x cols at a pitch of cols + pad, `offset`
    elements into a storage filled with `fill`."""
    s = torch.full((offset + max(rows, 1) * (cols + pad),), fill, dtype=dtype, device=device)
    return s[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], s


def norm_rows(x, gamma, residual, eps):
    """(h, y, delta): the norm in float64.  delta: each thread adds at most 64
    squares in order, then 10 levels of pairs, each step within E of a sum of
    positive terms; half of that goes through the square root.  rsqrt 2 ulp,
    the mean, the residual's sum (twice: it is squared) and the two products
    one rounding each."""
    h = x.double() + (residual.double() if residual is not None else 0.0)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * gamma.double()
    return h, y, (0.5 * (64 + 10 + 2) + 4 + 5) * E


def swiglu_rows(g, u):
    """(y, delta).  The device's fast exponential is within 2 + 1.173 |g| ulp
    (CUDA's documented bound), its fast division within 2 ulp; an ulp is at
    most 2 E."""
    g, u = g.double(), u.double()
    y = g / (1.0 + torch.exp(-g)) * u
    return y, (2.0 * (2 + 1.173 * float(g.abs().max() if g.numel() else 0.0) + 2) + 3) * E


def check_rows(y, delta, q, scale):
    """q and scale (from the device, moved to the CPU) against the rows y."""
    q, scale = q.double(), scale.double()
    amax = y.abs().amax(1)
    want = amax / 127.0
    assert bool(((scale - want).abs() <= (delta + 2 * E) * want + 2.0 ** -149).all())
    pos = want > 0
    assert bool((q[~pos] == 0).all())
    step = (q[pos] - y[pos] / want[pos][:, None]).abs()
    assert float(step.max() if step.numel() else 0.0) <= 0.5 + 127.0 * (2 * delta + 4 * E), float(step.max())
    # the largest value of every row stands at +-127
    if pos.any():
        assert bool((q[pos].abs().amax(1) == 127).all())


def product(a, b, sa, sb, bias=None, beta=0.0, c=None):
    """(y, |terms|) of the product in float64; the integer sums are exact."""
    s = a.double() @ b.double().t()
    y = s * sa.double()[:, None] * sb.double()[None, :]
    mag = y.abs()
    if bias is not None:
        y = y + bias.double()[None, :]
        mag = mag + bias.double().abs()[None, :]
    if beta != 0.0:
        y = y + beta * c.double()
        mag = mag + (beta * c.double()).abs()
    return y, mag


def partial_error(a, b):
    """Relative error the sum itself may have: none while partial sums stay
    below 2^24 whatever their order (K <= 1024), else one FP32 rounding (an ulp,
    if it truncates) for each 16-deep step, of at most the sum of |products|."""
    K = a.shape[1]
    return 0.0 if K <= 1024 else (K / 16 + 16) * 2 * E


def check_product(got, y, mag, sum_mag=None, sum_err=0.0):
    """got (device type, on the CPU) within the roundings of y: up to four FP32
    operations on terms of size mag, the sum's own error, one rounding to
    the output type."""
    tol = U[got.dtype] * (y.abs() + 4 * E * mag) + 4 * E * mag + TINY[got.dtype]
    if sum_mag is not None:
        tol = tol + sum_err * sum_mag
    off = ((got.double() - y).abs() / tol).max() if got.numel() else torch.tensor(0.0)
    assert bool(off <= 1.0), "worst error / tolerance = %g" % float(off)
