"""swiglu_i8 where 1 + exp(-g) is next to FP32's largest number: the quotient is
small but not zero, and a large u makes an ordinary value of it."""
import pytest
import torch

from tests import i8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(4, 100, 4, 0), (4, 100, 3, 1), (40, 4096, 0, 0), (3, 33000, 0, 0),
                                                  (8003, 1000, 0, 0), (700, 12304, 0, 0)])
def test_gates_far_below_zero(rows, cols, pad, offset, ty):
    import dense_gemm_09_gb300 as dg
    gen = torch.Generator().manual_seed(cols)
    dt = ref.TYPES[ty]
    g, _ = ref.pitched(rows, cols, dt, pad, offset)
    u, _ = ref.pitched(rows, cols, dt, pad, offset)
    # 1 + exp(-g) from 2^123 to 2^128 (its FP32 form is finite up to g = -88.72)
    g.copy_((-85.3 - 3.4 * torch.rand((rows, cols), generator=gen)).clamp(min=-88.5))
    u.copy_(torch.randn((rows, cols), generator=gen) * 1e36)
    q, _ = ref.pitched(rows, cols, torch.int8, pad, offset)
    s = torch.empty(rows, device="cuda")
    dg.swiglu_i8(g, u, q, s)
    y, delta = ref.swiglu_rows(g, u)
    ref.check_rows(y, delta, q, s)
    # one such value in a row of zeros
    u[:, 1:] = 0.0
    dg.swiglu_i8(g, u, q, s)
    y, delta = ref.swiglu_rows(g, u)
    ref.check_rows(y, delta, q, s)
