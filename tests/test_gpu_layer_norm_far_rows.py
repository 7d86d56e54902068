"""The layer norm's backward of rows so far from 0 that their mean times rstd is beyond float's
range: channels that a thread has no element for, and rows that a block's last step has none
for, leave the sums alone."""
import pytest
import torch

import token_layer_reference as ref
from test_gpu_layer_norm import BF16, F32, ctx, gsr  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = 2.0 ** 121          # rstd is 1 / sqrt(1e-5) for a constant row: together 8e38


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dtotal", [False, True])
@pytest.mark.parametrize("rows,c", [(3, 24), (300, 33), (5, 77), (200, 1000), (40, 2050), (90, 9000), (20000, 32), (1300, 1024)])
def test_constant_rows(gsr, ctx, dtype, dtotal, rows, c):  # noqa: F811
    """xh is exactly 0, so dx = rstd (g - mean(g)) + dtotal, dw = 0, db = sum dout."""
    g = torch.Generator().manual_seed(rows + c)
    dout, more = (torch.randn(rows, c, generator=g).to(dtype) for _ in range(2))
    w = 1 + 0.3 * torch.randn(c, generator=g)
    total = torch.full((rows, c), FAR, dtype=dtype)
    mean, rstd = torch.full((rows,), FAR), torch.full((rows,), 1e-5).rsqrt()
    dx, dw, db = gsr.layer_norm_backward(ctx, dout.cuda(), total.cuda(), w.cuda(), mean.cuda(), rstd.cuda(),
                                         dl_dtotal=more.cuda() if dtotal else None)
    grad = dout.double() * w.double()
    m = grad.mean(1, keepdim=True)
    scale = rstd.double()[:, None]
    want = scale * (grad - m)
    # As token_layer_reference's with xh = 0 and rstd given.
    bound = scale * (ref.F * grad.abs() + (ref.DEPTH + 2) * ref.F * grad.abs().mean(1, keepdim=True)
                     + 4 * ref.F * (grad.abs() + m.abs())) + 2 * ref.F * want.abs()
    if dtotal:
        bound = bound + ref.F * (want.abs() + more.double().abs())
        want = want + more.double()
    ref.check(dx, (want, bound + ref.rounding(want, dtype)), "dx")
    assert (dw == 0).all()
    # A chain of a thread's rows, fewer than all, and a tree.
    ref.check(db, (dout.double().sum(0), min(rows, ref.ROWS) * ref.F * dout.double().abs().sum(0) + ref.DEPTH * ref.F
                   * dout.double().abs().sum(0)), "dbias")
