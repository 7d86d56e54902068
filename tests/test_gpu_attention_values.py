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
