"""Cross attention's gradients beside outliers: what one item, head or row holds must
not cost the others their precision."""
import pytest
import torch

import decoder_reference as ref

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


def _inputs(b, lq, lk, hq, hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q, dout = (torch.randn(b, lq, hq, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(b, lk, hk, d, generator=g).to(dtype) for _ in range(2))
    return q, k, v, dout


def _run(gsr, ctx, q, k, v, dout, **opts):
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = gsr.cross_attention_forward(ctx, *dev, **opts)
    return (out, lse, *gsr.cross_attention_backward(ctx, *dev, out, lse, dout.cuda(), **opts))


def _check(want, got, part):
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
        ref.check(part(t.cpu()), tuple(part(w) for w in want[name]), name)


@pytest.mark.parametrize("lq", [1, 5, 200])
@pytest.mark.parametrize("lk", [90, 300])
@pytest.mark.parametrize("value", [1e3, 6e4])
def test_outliers_stay_in_their_head(gsr, ctx, lq, lk, value):
    """One large v and one large row of dL/dout in item 0's first heads: item 1's
    gradients, and those of item 0's other key head, keep their bounds."""
    q, k, v, dout = _inputs(2, lq, lk, 4, 2, 64, F16, lq + lk)
    v[0, 5, 0, 7] = value
    dout[0, lq // 2, 0] *= 1000.0
    want = ref.attention(q.double(), k.double(), v.double(), torch.ones(2, lk, dtype=torch.bool), 0.125, F16, dout.double())
    got = _run(gsr, ctx, q, k, v, dout)
    _check(want, got, lambda t: t[1:])
    for name, t, heads in (("dq", got[2], slice(2, 4)), ("dk", got[3], slice(1, 2)), ("dv", got[4], slice(1, 2))):
        ref.check(t[:1, :, heads], tuple(w[:1, :, heads] for w in want[name]), name)


@pytest.mark.parametrize("value", [1e3, 6e4])
def test_outlier_rows_leave_the_other_queries(gsr, ctx, value):
    """dL/dq of each query keeps its bound beside one large row of dL/dout in its own head."""
    q, k, v, dout = _inputs(1, 200, 300, 2, 1, 64, F16, 3)
    v[0, 5, 0, 7] = value
    dout[0, 3, 0] *= 1000.0
    want = ref.attention(q.double(), k.double(), v.double(), torch.ones(1, 300, dtype=torch.bool), 0.125, F16, dout.double())
    ref.check(_run(gsr, ctx, q, k, v, dout)[2], want["dq"], "dq")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_nan_stays_in_its_item(gsr, ctx, dtype):
    q, k, v, dout = _inputs(3, 150, 200, 4, 2, 64, dtype, 4)
    clean = _run(gsr, ctx, q, k, v, dout)
    v[1, 7, 0, 3] = float("nan")
    dout[1, 9, 2, 5] = float("inf")
    got = _run(gsr, ctx, q, k, v, dout)
    for a, b in zip(got, clean):
        assert torch.equal(a[::2], b[::2])


@pytest.mark.parametrize("b,lq,lk,hq,hk,d,size", [(10, 2, 80, 4, 4, 104, 1.0), (6, 3, 282, 8, 4, 72, 3.0),
                                                  (1, 1, 202, 3, 3, 72, 3.0), (1, 2, 258, 8, 2, 88, 8.0)])
def test_products_below_the_range_keep_small_gradients(gsr, ctx, b, lq, lk, hq, hk, d, size):
    """|dL/dout| |v| below 2^16 cannot take ds out of f16's range: ds is not scaled down."""
    q, k, v, dout = _inputs(b, lq, lk, hq, hk, d, F16, 1)
    q, v, dout = size * q, 30.0 * v, 10.0 * dout
    want = ref.attention(q.double(), k.double(), v.double(), torch.ones(b, lk, dtype=torch.bool), 0.3, F16, dout.double())
    for name, got in zip(("dq", "dk", "dv"), _run(gsr, ctx, q, k, v, dout, scale=0.3)[2:]):
        ref.check(got, want[name], name)


@pytest.mark.parametrize("lk", [2, 200])
def test_ds_at_its_bound(gsr, ctx, lk):
    """Two keys with half of the weight each and opposite values: ds is half of |dL/dout| |v|, 320,000."""
    q = torch.full((1, 150, 1, 64), 1e-3).to(F16)
    q[..., 0] = 0.125
    k = torch.zeros(1, lk, 1, 64).to(F16)
    k[:, 2:, :, 0] = -800.0
    v = torch.full((1, lk, 1, 64), 100.0).to(F16)
    v[:, 1] = -100.0
    dout = torch.zeros(1, 150, 1, 64).to(F16)
    dout[:, 7] = 100.0
    valid = torch.ones(1, lk, dtype=torch.bool)
    want = ref.attention(q.double(), k.double(), v.double(), valid, 1.0, F16, dout.double())
    assert want["dk"][0].abs().max() == 40000
    for name, got in zip(("dq", "dk", "dv"), _run(gsr, ctx, q, k, v, dout, scale=1.0)[2:]):
        ref.check(got, want[name], name)
