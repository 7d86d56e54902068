"""Gradients where a valid key holds an infinity that makes its scores -inf."""
import pytest
import torch

import decoder_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gsr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_tile_bin_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(gsr):
    c = gsr.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lq", [5, 128, 300])
@pytest.mark.parametrize("lk", [100, 400])
@pytest.mark.parametrize("d", [64, 128])
def test_key_gradients_beside_scores_of_minus_infinity(gsr, ctx, dtype, lq, lk, d):
    """A key whose scores are -inf for every query has probability 0: its dk and dv are
    zero and the others' are those without it.  (dq is 0 times infinity there.)"""
    g = torch.Generator().manual_seed(lq + lk + d)
    q, dout = (torch.randn(2, lq, 2, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(2, lk, 1, d, generator=g).to(dtype) for _ in range(2))
    q[..., 0] = 1.0
    none = torch.zeros(2, lk, dtype=torch.bool)
    none[0, :20] = none[0, lk - 1] = none[1, 30:70] = True
    k[none] = 0.0
    want = ref.attention(q.double(), k.double(), v.double(), ~none, d ** -0.5, dtype, dout.double())
    k[..., 0] = torch.where(none[:, :, None], float("-inf"), k[..., 0])
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = gsr.cross_attention_forward(ctx, *dev)
    _, dk, dv = gsr.cross_attention_backward(ctx, *dev, out, lse, dout.cuda())
    ref.check(dk, want["dk"], "dk")
    ref.check(dv, want["dv"], "dv")
