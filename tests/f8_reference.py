"""Plain forms of the 8-bit floating-point operators and of tokens by expert, and
how far FP32 may be off them.

Quantised values of given inputs are defined to the bit by FP32 operations, which
torch repeats; products and sums are formed in float64 on the stored inputs.  E is
FP32's unit roundoff, U the output types'.
"""
from __future__ import annotations

import torch

from tests.i8_reference import E, TINY, TYPES, U, pitched  # noqa: F401

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def quantized(y, rows, f8):
    """(Q, scale) of FP32 values with a scale for each rows x 128 of them."""
    m, k = y.shape
    z = torch.nn.functional.pad(y, (0, -k % BLOCK, 0, -m % rows))
    z = z.reshape(z.shape[0] // rows, rows, z.shape[1] // BLOCK, BLOCK)
    a = z.abs().amax((1, 3))  # (NaN where there is one)
    fine = torch.isfinite(a)
    factor = torch.where(a < 2.0 ** -100, 2.0 ** 100, 1.0)
    # (quotients rounded once: torch divides FP32 by a number, or a number by FP32,
    # through a rounded reciprocal; float64's quotient rounds to FP32's)
    inv = torch.where(fine & (a > 0), (TOP[f8] / (a * factor).double()).float(), 0.0)
    q = (z * factor[:, None, :, None]) * inv[:, None, :, None]
    q = torch.where((inv > 0)[:, None, :, None], q, 0.0).clamp(-TOP[f8], TOP[f8])
    q = q.reshape(-1, z.shape[2] * BLOCK)[:m, :k].to(f8)
    return q, torch.where(fine, (a.double() / TOP[f8]).float(), float("nan"))


def spread(scale, rows, m, k):
    """A scale for each value."""
    s = scale.repeat_interleave(BLOCK, -1)[..., :k]
    return s.repeat_interleave(rows, -2)[..., :m, :] if rows > 1 else s


def operand(m, k, rows, f8, g, loud=True):
    """(Q, scale): random 8-bit values of every size, and scales over some octaves."""
    q = torch.randn(m, k, generator=g, device="cuda") * 2.0 ** torch.randint(-6, 7, (m, 1), generator=g, device="cuda")
    scale = torch.exp2(6 * torch.rand(-(-m // rows), blocks(k), generator=g, device="cuda") - 3)
    return q.to(f8), scale


def product(a, sa, ra, b, sb, rb):
    """(C, |C|): the product in float64 and the sum of the terms' magnitudes."""
    m, k = a.shape
    x = a.double() * spread(sa.double(), ra, m, k)
    y = b.double() * spread(sb.double(), rb, b.shape[0], k)
    return x @ y.t(), x.abs() @ y.abs().t()


def product_error(k):
    """How far FP32 may be off, relative to the sum of the magnitudes: products are exact;
    a block's 128 are added in steps of 16 or more, each of which may truncate (2 E) at
    either operand of its addition; the two scales one rounding each; the sum over blocks
    one each."""
    return (2 * 2 * 8 + 2 + blocks(k)) * E
