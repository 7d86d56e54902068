"""Cross attention's outputs are averages of v: what its rounding may not do to them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


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


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq", [3, 300])
def test_a_single_key_returns_its_value(gsr, ctx, dtype, d, lq):
    g = torch.Generator().manual_seed(lq + d)
    q = (3 * torch.randn(2, lq, 4, d, generator=g)).to(dtype).cuda()
    k, v = (torch.randn(2, 40, 2, d, generator=g).to(dtype).cuda() for _ in range(2))
    lengths = torch.ones(2, dtype=torch.int32, device="cuda")
    want = v[:, :1].repeat_interleave(2, dim=2).expand(2, lq, 4, d)
    assert torch.equal(gsr.cross_attention_forward(ctx, q, k, v, kv_lengths=lengths)[0], want)
    assert torch.equal(gsr.cross_attention_forward(ctx, q, k[:, :1], v[:, :1])[0], want)
    mask = torch.zeros(2, 40, dtype=torch.bool, device="cuda")
    mask[:, 17] = True
    want = v[:, 17:18].repeat_interleave(2, dim=2).expand(2, lq, 4, d)
    assert torch.equal(gsr.cross_attention_forward(ctx, q, k, v, key_mask=mask)[0], want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk", [(1, 200), (3, 20000), (300, 70), (300, 3000)])
@pytest.mark.parametrize("size", [1.0, 20.0])
def test_the_largest_values_stay_finite(gsr, ctx, d, lq, lk, size):
    """An average of f16's largest value is that value, within P's rounding (2^-11) and its
    own: for rows that many keys share and for rows that one key takes."""
    g = torch.Generator().manual_seed(lk + d)
    q = (size * torch.randn(1, lq, 8, d, generator=g)).to(F16).cuda()
    k = torch.randn(1, lk, 8, d, generator=g).to(F16).cuda()
    sign = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0).cuda()
    v = (65504.0 * sign).to(F16).expand(1, lk, 8, d).contiguous()
    out, _ = gsr.cross_attention_forward(ctx, q, k, v)
    assert torch.isfinite(out).all()
    assert ((out.float() * sign - 65504.0).abs() <= 65504.0 * 2.0 ** -10).all()


def test_infinite_values_stay_infinite(gsr, ctx):
    for lq in (2, 200):
        q = torch.zeros(1, lq, 1, 64, dtype=F16, device="cuda")
        v = torch.zeros(1, 150, 1, 64, dtype=F16, device="cuda")
        v[0, 3, 0, 5], v[0, 90, 0, 6], v[0, 90, 0, 7] = float("inf"), float("-inf"), float("nan")
        out, _ = gsr.cross_attention_forward(ctx, q, torch.zeros_like(v), v)
        assert (out[..., 5] == float("inf")).all() and (out[..., 6] == float("-inf")).all()
        assert torch.isnan(out[..., 7]).all()
        assert (out[..., :5] == 0).all() and (out[..., 8:] == 0).all()
