"""Layer norm behind a residual sum against its 64-bit form, forward and backward."""
import pytest
import torch

import token_layer_reference as ref

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


def _inputs(shape, dtype, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    c = shape[-1]
    x = (torch.randn(shape, generator=g) * (0.5 + torch.rand(c, generator=g)) + torch.randn(c, generator=g)).to(dtype)
    more = [torch.randn(shape, generator=g).to(dtype) for _ in range(3)]
    w, b = 1 + 0.3 * torch.randn(c, generator=g), 0.3 * torch.randn(c, generator=g)
    return x, more[0] if residual else None, more[1], more[2] if residual else None, w, b


def _dev(t):
    return None if t is None else t.cuda()


def _double(t):
    return None if t is None else t.double()


def _compare(gsr, ctx, x, residual, dout, dtotal, w, b, eps=1e-5, place=_dev):
    xd, rd, dd, td = (place(t) for t in (x, residual, dout, dtotal))
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, xd, _dev(w), _dev(b), residual=rd, eps=eps)
    dx, dw, db = gsr.layer_norm_backward(ctx, dd, total, _dev(w), mean, rstd, dl_dtotal=td)
    want = ref.layer_norm(x.double(), w, b, eps, x.dtype, _double(residual), dout.double(), _double(dtotal))
    got = {"out": out, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dw, "dbias": db}
    if residual is not None:
        got["total"] = total
    for name, t in got.items():
        ref.check(t, want[name], name)


CHANNELS = [1, 2, 3, 7, 8, 31, 32, 33, 64, 72, 77, 127, 128, 129, 250, 256, 257, 511, 512, 577, 1000, 1024, 1025, 1280,
            2047, 2048, 2050, 2056, 4096, 4099, 5000, 8192, 8200, 16381, 16384]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("c", CHANNELS)
def test_parity(gsr, ctx, dtype, c):
    for rows, residual in ((1, True), (5, False), (37, True)):
        _compare(gsr, ctx, *_inputs((rows, c), dtype, 100 * c + rows, residual))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,c", [(20000, 64), (9001, 128), (3000, 1280), (3001, 577), (1500, 2048), (700, 4096),
                                    (100003, 8), (40001, 5), (400, 16384)])
def test_many_rows(gsr, ctx, dtype, rows, c):
    _compare(gsr, ctx, *_inputs((rows, c), dtype, rows))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,c", [(2, 8193), (75, 8704), (76, 8720), (77, 9000), (153, 12352), (230, 16376), (310, 16383)])
def test_rows_over_two_blocks(gsr, ctx, dtype, rows, c):
    """Rows of more than 8,192 channels, around the number that are under way at a time."""
    _compare(gsr, ctx, *_inputs((rows, c), dtype, c, rows % 2 == 0))


def test_rows_over_two_blocks_in_place_and_captured(gsr, ctx):
    x, r, dout, dt, w, b = (t.cuda() for t in _inputs((2, 90, 10000), BF16, 12))
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, b, residual=r)
    dx, dw, db = gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=dt)
    y, s, d = x.clone(), r.clone(), dout.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, m, q = gsr.layer_norm_forward(ctx, y, w, b, residual=s, out=y, total=s)
        _, ew, eb = gsr.layer_norm_backward(ctx, d, s, w, m, q, dl_dtotal=dt, dl_dx=d)
    for _ in range(2):
        y.copy_(x)
        s.copy_(r)
        d.copy_(dout)
        graph.replay()
        for got, want in ((y, out), (s, total), (m, mean), (q, rstd), (d, dx), (ew, dw), (eb, db)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_missing_parameters(gsr, ctx, weight, bias):
    x, r, dout, dt, w, b = _inputs((50, 96), F32, 5)
    _compare(gsr, ctx, x, r, dout, dt, w if weight else None, b if bias else None)


def test_residual_without_a_gradient_of_its_own(gsr, ctx):
    x, r, dout, _, w, b = _inputs((2, 20, 96), BF16, 6)
    _compare(gsr, ctx, x, r, dout, None, w, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_heads_of_a_projection(gsr, ctx, dtype):
    """Queries and keys as slices of one projection, each head with its own statistics; the
    gradients go into slices of the projection's gradient."""
    g = torch.Generator().manual_seed(7)
    for c in (64, 72, 80, 33):
        both = torch.randn(2, 31, 2, 5, c, generator=g).to(dtype)
        dout = torch.randn(2, 31, 5, c, generator=g).to(dtype)
        w = 1 + 0.3 * torch.randn(c, generator=g)
        dev, grad = both.cuda(), torch.full_like(both, 9.0).cuda()
        for part in (0, 1):
            x = dev[:, :, part]
            out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w.cuda())
            assert total is x and mean.shape == (2, 31, 5)
            gsr.layer_norm_backward(ctx, dout.cuda(), x, w.cuda(), mean, rstd, dl_dx=grad[:, :, part])
            want = ref.layer_norm(both[:, :, part].double(), w, None, 1e-5, dtype, None, dout.double())
            ref.check(out, want["out"], "out")
            ref.check(grad[:, :, part], want["dx"], "dx")
            if part == 0:
                assert (grad[:, :, 1] == 9.0).all()


def test_strided_rows_and_a_shared_residual(gsr, ctx):
    """Every third token of a wider array, and a residual that all items share by a stride of 0."""
    x, _, dout, _, w, b = _inputs((3, 8, 40), F16, 8)
    wide = torch.zeros(3, 24, 56, dtype=F16, device="cuda")
    wide[:, ::3, 8:48] = x.cuda()
    shared = torch.randn(8, 40, generator=torch.Generator().manual_seed(1)).to(F16)
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, wide[:, ::3, 8:48], w.cuda(), b.cuda(),
                                                    residual=shared.cuda().expand(3, 8, 40))
    want = ref.layer_norm(x.double(), w, b, 1e-5, F16, shared.expand(3, 8, 40).double())
    ref.check(out, want["out"], "out")
    ref.check(total, want["total"], "total")
    assert (wide[:, 1::3] == 0).all() and (wide[:, ::3, :8] == 0).all() and (wide[:, ::3, 48:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_arrays(gsr, ctx, dtype, shift):
    def place(t):
        if t is None:
            return None
        base = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        return base[shift:].view(t.shape).copy_(t)

    for c in (64, 1280):
        _compare(gsr, ctx, *_inputs((33, c), dtype, 9), place=place)


def test_in_place(gsr, ctx):
    x, r, dout, dt, w, b = (t.cuda() for t in _inputs((2, 30, 256), BF16, 10))
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, b, residual=r)
    dx, _, _ = gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=dt)
    for place in (dout, dt):
        keep = place.clone()
        same, _, _ = gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=dt, dl_dx=place)
        assert same.data_ptr() == place.data_ptr() and torch.equal(same, dx)
        place.copy_(keep)
    for places in (dict(out=x, total=r), dict(out=r, total=x)):
        a, c = x.clone(), r.clone()
        swap = {k: (a if v is x else c) for k, v in places.items()}
        y, s, _, _ = gsr.layer_norm_forward(ctx, a, w, b, residual=c, **swap)
        assert torch.equal(y, out) and torch.equal(s, total)
    plain, _, _, _ = gsr.layer_norm_forward(ctx, x, w, b)
    y, _, _, _ = gsr.layer_norm_forward(ctx, x, w, b, out=x)
    assert torch.equal(y, plain)


def test_values_far_from_zero_and_constant_rows(gsr, ctx):
    x, _, dout, _, w, b = _inputs((40, 320), F32, 11, False)
    _compare(gsr, ctx, x + 1000.0, None, dout, None, w, b)
    _compare(gsr, ctx, torch.full_like(x, 0.75), None, dout, None, w, b)
    _compare(gsr, ctx, torch.zeros_like(x), None, dout, None, w, b)
    x[:, 3] = 3e3
    _compare(gsr, ctx, x, None, dout, None, w, b)


def test_large_values_of_f16(gsr, ctx):
    """Squares beyond f16, sums beyond f16: the sum is infinite, its row not a number."""
    x, r, _, _, w, b = _inputs((6, 128), F16, 12)
    x[2], r[2] = 6e4, 0.0
    x[2, ::2] = -6e4
    x[4, 5], r[4, 5] = 6e4, 6e4
    out, total, _, _ = gsr.layer_norm_forward(ctx, x.cuda(), w.cuda(), b.cuda(), residual=r.cuda())
    assert total[4, 5] == float("inf") and torch.isnan(out[4]).all()
    rows = [0, 1, 2, 3, 5]
    want = ref.layer_norm(x[rows].double(), w, b, 1e-5, F16, r[rows].double())
    ref.check(out[rows], want["out"], "out")


def test_not_finite_stays_in_its_row(gsr, ctx):
    x, r, dout, _, w, b = (t.cuda() for t in _inputs((40, 2048), F32, 13))
    x[3, 5], x[7, 0] = float("nan"), float("inf")
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, b, residual=r)
    dx, _, _ = gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd)
    for t in (out, dx):
        bad = torch.isnan(t).any(dim=1)
        assert bad[3] and bad[7] and bad.sum() == 2


def test_same_bits_on_every_run(gsr, ctx):
    x, r, dout, dt, w, b = (t.cuda() for t in _inputs((5000, 512), BF16, 14))
    runs = []
    for _ in range(3):
        out, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, b, residual=r)
        runs.append((out, total, mean, rstd) + gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=dt))
    for run in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(run, runs[0]))


def test_gradient_against_differences(gsr, ctx):
    x, _, dout, dt, w, b = _inputs((21, 48), F32, 15)
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x.cuda(), w.cuda(), b.cuda())
    got = gsr.layer_norm_backward(ctx, dout.cuda(), total, w.cuda(), mean, rstd, dl_dtotal=dt.cuda())
    bounds = ref.layer_norm(x.double(), w, b, 1e-5, F32, None, dout.double(), dt.double())

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-5, F32)["out"][0] * dout).sum() + (x * dt).sum()

    h, args = 1e-5, [x.double(), w.double(), b.double()]
    for i, (name, t) in enumerate(zip(("dx", "dweight", "dbias"), got)):
        d = torch.randn(args[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
        ends = [loss(*args[:i], args[i] + sign * h * d, *args[i + 1:]) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(slope - (t.cpu().double() * d).sum()) <= (bounds[name][1] * d.abs()).sum() + 1e-6


def test_offsets_beyond_32_bits(gsr, ctx):
    """Rows more than 2^31 elements apart."""
    base = torch.empty((1 << 32) + 4096, dtype=BF16, device="cuda")
    x, _, dout, _, w, b = _inputs((3, 512), BF16, 16, False)
    far, far_out = (base.as_strided((3, 512), (1 << 31, 1), at) for at in (0, 1024))
    far.copy_(x.cuda())
    want, _, mean, rstd = gsr.layer_norm_forward(ctx, x.cuda(), w.cuda(), b.cuda())
    got, _, _, _ = gsr.layer_norm_forward(ctx, far, w.cuda(), b.cuda(), out=far_out)
    assert torch.equal(got, want)
    dx, dw, db = gsr.layer_norm_backward(ctx, dout.cuda(), x.cuda(), w.cuda(), mean, rstd)
    same = gsr.layer_norm_backward(ctx, dout.cuda(), far, w.cuda(), mean, rstd, dl_dx=far_out)
    assert all(torch.equal(p, q) for p, q in zip(same, (dx, dw, db)))


def test_empty(gsr, ctx):
    x = torch.empty(2, 0, 16, device="cuda")
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x)
    assert out.shape == x.shape and mean.shape == (2, 0)
    _, dw, db = gsr.layer_norm_backward(ctx, x, x, None, mean, rstd)
    assert (dw == 0).all() and (db == 0).all()


def test_refusals(gsr, ctx):
    x = torch.randn(2, 5, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gsr.GsrError):
            gsr.layer_norm_forward(ctx, x, w, eps=eps)
    with pytest.raises(gsr.GsrError):
        gsr.layer_norm_forward(ctx, torch.randn(2, 16392, device="cuda"))
    with pytest.raises(gsr.GsrError):
        gsr.layer_norm_forward(ctx, x, out=torch.empty(5, 16, device="cuda").expand(2, 5, 16))
    with pytest.raises(gsr.GsrError):
        out = torch.empty_like(x)
        gsr.layer_norm_forward(ctx, x, residual=x, out=out, total=out)
    for call in (lambda: gsr.layer_norm_forward(ctx, x.cpu()),
                 lambda: gsr.layer_norm_forward(ctx, x.double()),
                 lambda: gsr.layer_norm_forward(ctx, x[0, 0]),
                 lambda: gsr.layer_norm_forward(ctx, x[None, None]),
                 lambda: gsr.layer_norm_forward(ctx, x.transpose(1, 2)),
                 lambda: gsr.layer_norm_forward(ctx, x, weight=w[:8]),
                 lambda: gsr.layer_norm_forward(ctx, x, weight=w.half()),
                 lambda: gsr.layer_norm_forward(ctx, x, residual=x.half()),
                 lambda: gsr.layer_norm_forward(ctx, x, residual=x[:1]),
                 lambda: gsr.layer_norm_forward(ctx, x, total=x),
                 lambda: gsr.layer_norm_forward(ctx, x, out=x.half()),
                 lambda: gsr.layer_norm_backward(ctx, x, x, w, w, w)):
        with pytest.raises(ValueError):
            call()
