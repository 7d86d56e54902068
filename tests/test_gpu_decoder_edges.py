"""Decoder operators beyond a grid's limits, off their alignment, and over long rows."""
import pytest
import torch

import decoder_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


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


def _norm(gsr, ctx, x, dout, w, b, groups, act, place=lambda t: t.cuda()):
    xd, dd = place(x), place(dout)
    out, mean, rstd = gsr.group_norm_forward(ctx, xd, groups, w.cuda(), b.cuda(), activation=act,
                                             out=place(torch.zeros_like(x)))
    dx, dw, db = gsr.group_norm_backward(ctx, dd, xd, groups, w.cuda(), b.cuda(), mean, rstd, activation=act,
                                         dl_dx=place(torch.zeros_like(x)))
    want = ref.group_norm(x.double(), groups, w.double(), b.double(), 1e-5, act, dout.double(), x.dtype)
    for name, got in (("mean", mean), ("rstd", rstd), ("out", out), ("dx", dx), ("dweight", dw), ("dbias", db)):
        ref.check(got, want[name], name)


def _features(n, s, c, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, s, c, generator=g).to(dtype), torch.randn(n, s, c, generator=g).to(dtype),
            1 + 0.3 * torch.randn(c, generator=g), 0.3 * torch.randn(c, generator=g))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_norm_gradients_of_unaligned_arrays(gsr, ctx, dtype, shift):
    def place(t):
        base = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        return base[shift:].view(t.shape).copy_(t)

    for s in (33, 3000):
        _norm(gsr, ctx, *_features(2, s, 32, dtype, s), 8, "silu", place)


@pytest.mark.parametrize("c,groups", [(8, 2), (6, 3)])
def test_more_samples_than_a_grid_has_rows(gsr, ctx, c, groups):
    _norm(gsr, ctx, *_features(65535 + 4000, 3, c, F32, c), groups, "gelu")


def test_more_masked_items_than_a_grid_has_rows(gsr, ctx):
    g = torch.Generator().manual_seed(2)
    b, lq, lk = 65536, 17, 3
    q, dout = (torch.randn(b, lq, 1, 8, generator=g).to(BF16) for _ in range(2))
    k, v = (torch.randn(b, lk, 1, 8, generator=g).to(BF16) for _ in range(2))
    mask = torch.rand(b, lk, generator=g) < 0.6
    want = ref.attention(q.double(), k.double(), v.double(), mask, 8 ** -0.5, BF16, dout.double())
    k[~mask], v[~mask] = float("nan"), float("inf")
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = gsr.cross_attention_forward(ctx, *dev, key_mask=mask.cuda())
    grads = gsr.cross_attention_backward(ctx, *dev, out, lse, dout.cuda(), key_mask=mask.cuda())
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(got, want[name], name)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk", [(40, 2000), (300, 32640)])
def test_lse_of_long_rows(gsr, ctx, dtype, d, lq, lk):
    """Scores that float holds exactly, so that lse' bound is that of the sums alone: 64
    keys in chains of 16, two steps per tile of 128, the join, and each exponential's
    argument and value."""
    g = torch.Generator().manual_seed(lk + d)
    q, k = torch.zeros(lq, d), torch.zeros(lk, d)
    q[:, 0], q[:, 1] = 8.0, torch.randint(-8, 9, (lq,), generator=g) / 8
    k[:, 0] = torch.randint(-16, 17, (lk,), generator=g) / 16
    k[:, 1] = torch.randint(-64, 65, (lk,), generator=g) / 64
    v = torch.randn(lk, d, generator=g)
    s = q.double() @ k.double().T
    want = torch.logsumexp(s, dim=1)
    spread = s.amax(dim=1) - s.amin(dim=1)
    bound = ref.F * (4 * want.abs() + 4 * spread + 8 + 16 + 4 + 2 * (lk / 128 + 1) + 8)
    out, lse = gsr.cross_attention_forward(ctx, *(t.to(dtype).cuda()[None, :, None] for t in (q, k, v)), scale=1.0)
    error = (lse.cpu().double().view(lq) - want).abs()
    assert (error <= bound).all(), (error.max(), bound.min())


def test_offsets_beyond_32_bits(gsr, ctx):
    """Arrays whose elements lie more than 2^32 elements apart, in one allocation side by side."""
    g = torch.Generator().manual_seed(4)
    base = torch.empty((1 << 32) + (1 << 22), dtype=BF16, device="cuda")

    def spread(shape, slot, fill=None):
        """[batch, tokens, heads, dim] over the whole of it: rows of 2,048 elements, a slot each."""
        batch, tokens, heads, dim = shape
        token = (1 << 32) // (batch * tokens) // 2048 * 2048
        t = base.as_strided(shape, (tokens * token, token, dim, 1), slot * heads * dim)
        return t if fill is None else t.copy_(fill)

    for lq, lk in ((3, 400), (200, 400)):
        shapes = [(2, lq, 4, 64), (2, lk, 2, 64)]
        q, dout = (torch.randn(shapes[0], generator=g).to(BF16) for _ in range(2))
        k, v = (torch.randn(shapes[1], generator=g).to(BF16) for _ in range(2))
        want_out, want_lse = gsr.cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda())
        want = gsr.cross_attention_backward(ctx, q.cuda(), k.cuda(), v.cuda(), want_out, want_lse, dout.cuda())
        far = [spread(t.shape, i, t.cuda()) for i, t in ((0, q), (2, k), (3, v), (2, dout))]
        # (slots of 256 elements for the query's arrays and of 128 for the keys': 0-255, 256-383, 384-511, 512-767)
        out, lse = gsr.cross_attention_forward(ctx, *far[:3], out=spread(shapes[0], 3))
        assert torch.equal(out, want_out) and torch.equal(lse, want_lse)
        got = gsr.cross_attention_backward(ctx, *far[:3], out, lse, far[3], dl_dq=spread(shapes[0], 4),
                                           dl_dk=spread(shapes[1], 10), dl_dv=spread(shapes[1], 11))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        positions, freq = torch.rand(lq, 2, generator=g).cuda() * 9, gsr.rotary_frequencies([8, 8])
        turned = gsr.rotary_forward(ctx, far[0], positions, freq, [8, 8], out=spread(shapes[0], 5))
        assert torch.equal(turned, gsr.rotary_forward(ctx, q.cuda(), positions, freq, [8, 8]))


def test_norm_of_more_elements_than_32_bits_count(gsr, ctx):
    """3 samples of 2^22 x 384: the last one's statistics and some of its rows."""
    n, s, c, groups = 3, 1 << 22, 384, 8
    x = torch.empty((n, s, c), dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    x[2] += 0.5
    out, mean, rstd = gsr.group_norm_forward(ctx, x, groups, activation="none")
    last = x[2].view(s, groups, c // groups)
    for group in range(groups):
        var, mu = torch.var_mean(last[:, group].double(), correction=0)
        scale = 1 / torch.sqrt(var + 1e-5)
        assert abs(mean[2, group] - mu) <= 64 * ref.F * 8 and abs(rstd[2, group] - scale) <= 512 * ref.F
        rows = last[s - 1000:, group].double()
        want = (rows - mu) * scale
        got = out[2, s - 1000:].view(1000, groups, c // groups)[:, group].double()
        assert ((got - want).abs() <= ref.U[BF16] * want.abs() + 1024 * ref.F).all()
    dout = torch.ones_like(x)
    dx, dw, db = gsr.group_norm_backward(ctx, dout, x, groups, None, None, mean, rstd, activation="none", dl_dx=dout)
    # With dL/dout = 1 the gradient's mean and its part along x are all of it.
    assert (db == n * s).all() and (dx[2, s - 1000:].float().abs() <= 1e-3).all()
