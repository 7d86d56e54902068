"""Cross attention of few query rows over long rows of keys: the running sums hold
what they were given, however many tiles follow."""
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
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [2.0, 32.0])
def test_sums_do_not_drift(gsr, ctx, dtype, d, base):
    """More items than the SMs have blocks, so a block walks a whole row of keys, 510
    tiles, whose largest scores come first.  Every score is a sum of two products
    that float holds exactly; what is left to round is the argument of each
    exponential (its parts relative to the scores' size and to their difference), the
    exponential, a sum's step per tile of 64 keys, and the join of four warps."""
    b, lk, rows = 304, 32640, 4
    g = torch.Generator().manual_seed(int(base) + d)
    q = torch.zeros(rows, d)
    q[:, 0] = base - torch.tensor([0.0, 0.5, 0.25, 1.0])
    q[:, 1] = torch.tensor([1.0, 0.75, 1.25, 0.5])
    k = torch.zeros(lk, d)
    k[:, 0] = base
    k[:, 1] = torch.randint(-64, 65, (lk,), generator=g) / 64
    k[:64, 1] = 3.0
    v = torch.randn(lk, d, generator=g).to(dtype)
    s = 0.125 * (q.double() @ k.double().T)
    want = torch.logsumexp(s, dim=1)
    spread = 2 * (s.amax(dim=1) - s.amin(dim=1))
    bound = ref.F * (4 * want.abs() + 4 * spread + 8 + lk / 64 + 16)
    out, lse = gsr.cross_attention_forward(
        ctx, q.to(dtype).cuda().view(1, rows, 1, d).expand(b, rows, 1, d),
        *(t.to(dtype).cuda().view(1, lk, 1, d).expand(b, lk, 1, d) for t in (k, v)), scale=0.125)
    error = (lse.cpu().double().view(b, rows) - want).abs().amax(dim=0)
    assert (error <= bound).all(), (error, bound)
    o = torch.softmax(s, dim=1) @ v.double()
    # P rounded to the storage type for its product with v, and the output
    e_o = (bound[:, None] + ref.U[dtype]) * (torch.softmax(s, dim=1) @ v.double().abs()) + ref.rounding(o, dtype)
    if dtype == torch.float16:
        e_o = e_o + 2.0 ** -24 * v.double().abs().sum(dim=0) / lk
    assert ((out.cpu().double()[0, :, 0] - o).abs() <= e_o).all()
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
