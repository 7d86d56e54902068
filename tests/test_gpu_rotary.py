"""Rotary positions with several axes against their 64-bit form."""
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


def _check(gsr, ctx, x, positions, sections, interleaved, freq=None):
    freq = gsr.rotary_frequencies(sections, device="cpu") if freq is None else freq
    full = positions if positions.dim() == 3 else positions.expand(x.shape[0], *positions.shape)
    for call, backward in ((gsr.rotary_forward, False), (gsr.rotary_backward, True)):
        got = call(ctx, x.cuda(), positions.cuda(), freq.cuda(), sections, interleaved=interleaved)
        ref.check(got, ref.rotary(x.double(), full, freq, sections, interleaved, x.dtype, backward))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("b,t,h,d,sections", [
    (1, 1, 1, 2, [1]), (2, 9, 3, 64, [8, 12, 12]), (1, 37, 5, 72, [10, 11, 11]), (2, 5, 2, 128, [16, 24, 24]),
    (1, 300, 16, 96, [16, 16, 8, 8]), (3, 4, 1, 20, [3, 0, 5]), (1, 7, 2, 10, [0, 0]), (1, 3, 7, 44, [22])])
def test_parity(gsr, ctx, dtype, interleaved, b, t, h, d, sections):
    g = torch.Generator().manual_seed(b + t + d)
    x = torch.randn(b, t, h, d, generator=g).to(dtype)
    ints = torch.randint(-5, 50, (b, t, len(sections)), generator=g, dtype=torch.int32)
    _check(gsr, ctx, x, ints, sections, interleaved)
    _check(gsr, ctx, x, torch.rand(t, len(sections), generator=g) * 50, sections, interleaved)


def test_long_positions(gsr, ctx):
    """Positions up to 2^31 - 1: the float product alone would lose the angle."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 6, 2, 16, generator=g)
    pos = torch.tensor([[0], [12345], [1 << 20], [(1 << 24) + 1], [(1 << 31) - 1], [-(1 << 31)]], dtype=torch.int32)
    _check(gsr, ctx, x, pos, [8], False)


def test_strided_views_and_in_place(gsr, ctx):
    """Heads of a packed projection, a slice of a longer sequence, transposed heads, and out = x."""
    g = torch.Generator().manual_seed(2)
    sections, freq = [4, 8, 4], gsr.rotary_frequencies([4, 8, 4])
    packed = torch.randn(2, 30, 3, 4, 32, generator=g).to(BF16).cuda()
    pos = torch.randint(0, 50, (20, 3), generator=g, dtype=torch.int32).cuda()
    for view in (packed[:, 5:25, 1], packed[:, 5:25, 1].transpose(1, 2).contiguous().transpose(1, 2),
                 packed[0, 5:25, 0].expand(2, 20, 4, 32), packed[:, 5:25, 2, :1].expand(2, 20, 4, 32)):
        want = gsr.rotary_forward(ctx, view.contiguous(), pos, freq, sections)
        assert torch.equal(gsr.rotary_forward(ctx, view, pos, freq, sections), want)
    view = packed[:, 5:25, 1]
    want = gsr.rotary_forward(ctx, view.contiguous(), pos, freq, sections)
    keep = packed.clone()
    gsr.rotary_forward(ctx, view, pos, freq, sections, out=view)
    assert torch.equal(view, want)
    assert torch.equal(packed[:, :5], keep[:, :5]) and torch.equal(packed[:, :, 0], keep[:, :, 0])


def test_unaligned(gsr, ctx):
    g = torch.Generator().manual_seed(3)
    base = torch.randn(2 * 9 * 3 * 32 + 3, generator=g).to(F16).cuda()
    pos, freq = torch.rand(9, 2, generator=g).cuda() * 9, gsr.rotary_frequencies([8, 8])
    for shift in (1, 2, 3):
        x = base[shift:shift + 2 * 9 * 3 * 32].view(2, 9, 3, 32)
        for inter in (False, True):
            want = gsr.rotary_forward(ctx, x.clone(), pos, freq, [8, 8], interleaved=inter)
            assert torch.equal(gsr.rotary_forward(ctx, x, pos, freq, [8, 8], interleaved=inter), want)


def test_backward_undoes_forward_and_differences(gsr, ctx):
    g = torch.Generator().manual_seed(4)
    x, dout, d = (torch.randn(1, 12, 2, 24, generator=g).cuda() for _ in range(3))
    pos, freq, sections = torch.rand(12, 2, generator=g).cuda() * 20, gsr.rotary_frequencies([5, 6]), [5, 6]
    turned = gsr.rotary_forward(ctx, x, pos, freq, sections)
    back = gsr.rotary_backward(ctx, turned, pos, freq, sections)
    assert (back - x).abs().max() <= 40 * ref.F * x.abs().max()
    # The operator is linear in x: its difference quotient has no truncation error,
    # only each side's float roundings (8 F per value and term).
    grad = gsr.rotary_backward(ctx, dout, pos, freq, sections)
    h = 0.5
    ends = [gsr.rotary_forward(ctx, x + s * h * d, pos, freq, sections).double() for s in (1, -1)]
    slope = ((ends[0] - ends[1]) * dout.double()).sum() / (2 * h)
    size = (dout.abs().double() * (x.abs() + d.abs()).double()).sum() + (grad.abs() * d.abs()).double().sum()
    assert abs(slope - (grad.double() * d.double()).sum()) <= 64 * ref.F * size


def test_empty_and_other_stream(gsr, ctx):
    freq = gsr.rotary_frequencies([4])
    x = torch.empty(0, 5, 2, 8, device="cuda")
    assert gsr.rotary_forward(ctx, x, torch.zeros(5, 1, device="cuda"), freq, [4]).shape == x.shape
    x = torch.randn(1, 500, 4, 8, device="cuda")
    pos = torch.rand(500, 1, device="cuda")
    want = gsr.rotary_forward(ctx, x, pos, freq, [4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gsr.rotary_forward(ctx, x, pos, freq, [4], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals(gsr, ctx):
    x = torch.randn(2, 5, 3, 16, device="cuda")
    pos, freq = torch.zeros(5, 2, device="cuda"), gsr.rotary_frequencies([4, 4])
    with pytest.raises(gsr.GsrError):   # more pairs than the head holds
        gsr.rotary_forward(ctx, x, pos, gsr.rotary_frequencies([4, 5]), [4, 5])
    with pytest.raises(gsr.GsrError):   # a negative section
        gsr.rotary_forward(ctx, x, pos, freq, [9, -1])
    with pytest.raises(gsr.GsrError):   # an output whose items share memory
        gsr.rotary_forward(ctx, x, pos, freq, [4, 4], out=x[:1].expand(2, 5, 3, 16))
    with pytest.raises(gsr.GsrError):   # tokens that share memory
        gsr.rotary_forward(ctx, x[:, :1].expand(2, 5, 3, 16), pos, freq, [4, 4])
    for call in (lambda: gsr.rotary_forward(ctx, x[0], pos, freq, [4, 4]),
                 lambda: gsr.rotary_forward(ctx, x.double(), pos, freq, [4, 4]),
                 lambda: gsr.rotary_forward(ctx, x, pos[:4], freq, [4, 4]),
                 lambda: gsr.rotary_forward(ctx, x, pos.long(), freq, [4, 4]),
                 lambda: gsr.rotary_forward(ctx, x, pos, freq[:7], [4, 4]),
                 lambda: gsr.rotary_forward(ctx, x, pos, freq, [2, 2, 2, 1, 1]),
                 lambda: gsr.rotary_forward(ctx, x.transpose(2, 3), pos, freq, [1, 0]),
                 lambda: gsr.rotary_forward(ctx, x.cpu(), pos, freq, [4, 4])):
        with pytest.raises(ValueError):
            call()
