"""Group norm with an activation against its 64-bit form, forward and backward."""
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


def _inputs(n, s, c, dtype, seed, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, s, c, generator=g) * (0.5 + torch.rand(c, generator=g))
         + offset * torch.randn(c, generator=g)).to(dtype)
    dout = torch.randn(n, s, c, generator=g).to(dtype)
    w, b = 1 + 0.3 * torch.randn(c, generator=g), 0.3 * torch.randn(c, generator=g)
    return x, dout, w, b


def _compare(gsr, ctx, x, dout, w, b, groups, act, eps=1e-5):
    xd, dd = x.cuda(), dout.cuda()
    wd, bd = (None if t is None else t.cuda() for t in (w, b))
    out, mean, rstd = gsr.group_norm_forward(ctx, xd, groups, wd, bd, eps=eps, activation=act)
    dx, dw, db = gsr.group_norm_backward(ctx, dd, xd, groups, wd, bd, mean, rstd, activation=act)
    want = ref.group_norm(x.double(), groups, None if w is None else w.double(), None if b is None else b.double(),
                          eps, act, dout.double(), x.dtype)
    for name, got in (("mean", mean), ("rstd", rstd), ("out", out), ("dx", dx), ("dweight", dw), ("dbias", db)):
        ref.check(got, want[name], name)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("n,s,c,groups", [(1, 1, 8, 2), (2, 7, 24, 8), (1, 256, 64, 8), (3, 101, 96, 32),
                                          (2, 1031, 5, 5), (1, 33, 48, 1), (1, 3000, 320, 32)])
def test_parity(gsr, ctx, dtype, act, n, s, c, groups):
    _compare(gsr, ctx, *_inputs(n, s, c, dtype, 1000 * n + s + c), groups, act)


@pytest.mark.parametrize("n,s,c,groups", [(1, 70001, 32, 8), (5, 9001, 128, 32), (300, 5, 16, 4), (2, 40, 2056, 8),
                                          (1, 65, 4096, 1), (7, 20011, 64, 1), (2, 30001, 12, 4), (3, 9000, 6, 1),
                                          (1, 50003, 3, 3), (2, 7001, 20, 5)])
def test_parity_long_and_wide(gsr, ctx, n, s, c, groups):
    for dtype in (BF16, F32):
        _compare(gsr, ctx, *_inputs(n, s, c, dtype, 77 + s), groups, "silu")


def test_sizes_around_the_paths(gsr, ctx):
    """Sample sizes on either side of what one block holds, in both directions."""
    for s in (127, 128, 511, 512, 513, 1023, 1025, 2047, 2049, 4096, 4097):
        _compare(gsr, ctx, *_inputs(2, s, 32, F16, s), 4, "silu")


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_missing_parameters(gsr, ctx, weight, bias):
    x, dout, w, b = _inputs(2, 50, 16, F32, 5)
    _compare(gsr, ctx, x, dout, w if weight else None, b if bias else None, 4, "silu")


def test_mean_far_from_zero(gsr, ctx):
    """Features a thousand deviations from 0: a difference of squares would have nothing left."""
    x, dout, w, b = _inputs(2, 4000, 32, F32, 6)
    _compare(gsr, ctx, x + 1000.0, dout, w, b, 8, "silu")


def test_first_value_far_from_the_rest(gsr, ctx):
    x, dout, w, b = _inputs(1, 4000, 32, F32, 7)
    x[0, 0] = 3e3
    _compare(gsr, ctx, x, dout, w, b, 8, "none")


def test_constant_features(gsr, ctx):
    x, dout, w, b = _inputs(1, 40, 16, F32, 8)
    _compare(gsr, ctx, torch.full_like(x, 0.75), dout, w, b, 4, "silu")


def test_unaligned_arrays(gsr, ctx):
    """Arrays that start off a 16-byte boundary."""
    x, dout, w, b = _inputs(2, 33, 32, BF16, 9)
    for shift in (1, 3):
        base = torch.empty(x.numel() + shift, dtype=BF16, device="cuda")
        xd = base[shift:].view(x.shape)
        xd.copy_(x)
        out, mean, rstd = gsr.group_norm_forward(ctx, xd, 8, w.cuda(), b.cuda(), activation="gelu")
        want = ref.group_norm(x.double(), 8, w.double(), b.double(), 1e-5, "gelu", dtype=BF16)
        ref.check(out, want["out"], "out")


def test_feature_maps_and_in_place(gsr, ctx):
    x, dout, w, b = _inputs(2, 12, 16, F16, 10)
    xd = x.cuda().view(2, 3, 4, 16)
    out, mean, rstd = gsr.group_norm_forward(ctx, xd, 4, w.cuda(), b.cuda())
    assert out.shape == xd.shape
    dd = dout.cuda().view(2, 3, 4, 16)
    dx, _, _ = gsr.group_norm_backward(ctx, dd, xd, 4, w.cuda(), b.cuda(), mean, rstd)
    same, _, _ = gsr.group_norm_backward(ctx, dd, xd, 4, w.cuda(), b.cuda(), mean, rstd, dl_dx=dd)
    assert same.data_ptr() == dd.data_ptr() and torch.equal(same, dx)
    inplace, _, _ = gsr.group_norm_forward(ctx, xd, 4, w.cuda(), b.cuda(), out=xd)
    assert torch.equal(inplace, out)


def test_not_finite_stays_in_its_group(gsr, ctx):
    x, dout, w, b = _inputs(2, 40, 16, F32, 11)
    x[0, 3, 5] = float("nan")
    out, _, _ = gsr.group_norm_forward(ctx, x.cuda(), 4, w.cuda(), b.cuda())
    bad = torch.isnan(out).any(dim=1).cpu()
    assert bad[0, 4:8].all() and not bad[0, :4].any() and not bad[0, 8:].any() and not bad[1].any()


def test_same_bits_on_every_run(gsr, ctx):
    x, dout, w, b = (t.cuda() for t in _inputs(3, 5000, 64, BF16, 12))
    runs = []
    for _ in range(3):
        out, mean, rstd = gsr.group_norm_forward(ctx, x, 8, w, b)
        runs.append((out, mean, rstd) + gsr.group_norm_backward(ctx, dout, x, 8, w, b, mean, rstd))
    for run in runs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(run, runs[0]))


def test_gradient_against_differences(gsr, ctx):
    x, dout, w, b = _inputs(2, 21, 12, F32, 13)
    out, mean, rstd = gsr.group_norm_forward(ctx, x.cuda(), 3, w.cuda(), b.cuda())
    dx, dw, db = gsr.group_norm_backward(ctx, dout.cuda(), x.cuda(), 3, w.cuda(), b.cuda(), mean, rstd)
    bounds = ref.group_norm(x.double(), 3, w.double(), b.double(), 1e-5, "silu", dout.double())
    h = 1e-5
    for i, (name, got) in enumerate((("dx", dx), ("dweight", dw), ("dbias", db))):
        args = [x.double(), w.double(), b.double()]
        d = torch.randn(args[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
        ends = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * h * d
            ends.append((ref.group_norm(moved[0], 3, moved[1], moved[2], 1e-5, "silu")["out"][0] * dout).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(slope - (got.cpu().double() * d).sum()) <= (bounds[name][1] * d.abs()).sum() + 1e-6


def test_on_another_stream(gsr, ctx):
    x, dout, w, b = (t.cuda() for t in _inputs(2, 3000, 64, F16, 14))
    first = gsr.group_norm_forward(ctx, x, 8, w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = gsr.group_norm_forward(ctx, x, 8, w, b, stream=side)
    third = gsr.group_norm_forward(ctx, x, 8, w, b)
    torch.cuda.synchronize()
    for other in (second, third):
        assert all(torch.equal(p, q) for p, q in zip(first, other))


def test_empty(gsr, ctx):
    x = torch.empty(2, 0, 16, device="cuda")
    out, mean, rstd = gsr.group_norm_forward(ctx, x, 4)
    assert out.shape == x.shape
    _, dw, db = gsr.group_norm_backward(ctx, x, x, 4, None, None, mean, rstd)
    assert (dw == 0).all() and (db == 0).all()


def test_refusals(gsr, ctx):
    x = torch.randn(2, 5, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    for bad in (dict(groups=3), dict(groups=0), dict(groups=-1), dict(groups=4, eps=0.0),
                dict(groups=4, eps=float("nan"))):
        with pytest.raises((gsr.GsrError, RuntimeError)):
            gsr.group_norm_forward(ctx, x, weight=w, bias=w, **bad)
    with pytest.raises(gsr.GsrError):
        wide = torch.randn(1, 2, 4104, device="cuda")
        gsr.group_norm_forward(ctx, wide, 8)
    for call in (lambda: gsr.group_norm_forward(ctx, x, 4, activation="relu"),
                 lambda: gsr.group_norm_forward(ctx, x.cpu(), 4),
                 lambda: gsr.group_norm_forward(ctx, x.double(), 4),
                 lambda: gsr.group_norm_forward(ctx, x.transpose(1, 2), 5),
                 lambda: gsr.group_norm_forward(ctx, x, 4, weight=w[:8]),
                 lambda: gsr.group_norm_forward(ctx, x, 4, weight=w.half()),
                 lambda: gsr.group_norm_forward(ctx, x, 4, out=x.half())):
        with pytest.raises(ValueError):
            call()
