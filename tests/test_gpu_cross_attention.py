"""Cross attention to states of another length against its 64-bit form."""
import math

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


def _inputs(b, lq, lk, hq, hk, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    q, dout = (torch.randn(b, lq, hq, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(b, lk, hk, d, generator=g).to(dtype) for _ in range(2))
    return q * size, k, v, dout


def _valid(b, lk, lengths, mask):
    valid = torch.ones(b, lk, dtype=torch.bool)
    if lengths is not None:
        valid &= torch.arange(lk) < lengths[:, None]
    if mask is not None:
        valid &= mask.bool()
    return valid


def _compare(gsr, ctx, q, k, v, dout, lengths=None, mask=None, scale=None, backward=True, poison=True):
    valid = _valid(k.shape[0], k.shape[1], lengths, mask)
    want = ref.attention(q.double(), k.double(), v.double(), valid, scale or q.shape[3] ** -0.5, q.dtype,
                         dout.double() if backward else None)
    kd, vd = k.cuda(), v.cuda()
    if poison:   # what an invalid key holds must reach nothing
        kd[~valid.cuda()] = float("nan")
        vd[~valid.cuda()] = float("inf")
    opts = dict(kv_lengths=None if lengths is None else lengths.cuda(), key_mask=None if mask is None else mask.cuda(),
                scale=scale)
    out, lse = gsr.cross_attention_forward(ctx, q.cuda(), kd, vd, **opts)
    ref.check(lse, want["lse"], "lse")
    ref.check(out, want["out"], "out")
    if backward:
        grads = gsr.cross_attention_backward(ctx, q.cuda(), kd, vd, out, lse, dout.cuda(), **opts)
        for name, got in zip(("dq", "dk", "dv"), grads):
            ref.check(got, want[name], name)
    return want


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [8, 32, 64, 72, 96, 128])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 300), (5, 77), (16, 256), (129, 127), (300, 130)])
def test_parity(gsr, ctx, dtype, d, lq, lk):
    _compare(gsr, ctx, *_inputs(2, lq, lk, 4, 2, d, dtype, lq + lk + d))


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 2), (6, 3), (20, 1)])
@pytest.mark.parametrize("lq", [1, 3, 40])
def test_head_groups(gsr, ctx, hq, hk, lq):
    _compare(gsr, ctx, *_inputs(1, lq, 140, hq, hk, 64, BF16, hq + hk + lq))


@pytest.mark.parametrize("lq", [1, 2, 15, 16, 17, 64, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("lk", [63, 64, 65, 128, 129, 257])
def test_lengths_around_the_tiles(gsr, ctx, lq, lk):
    _compare(gsr, ctx, *_inputs(1, lq, lk, 2, 1, 64, F16, lq * lk))


@pytest.mark.parametrize("lq", [1, 7, 50, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_of_the_items(gsr, ctx, lq, d):
    """Item lengths of zero, one, a tile's edges and all keys; values outside are clamped."""
    args = _inputs(8, lq, 260, 2, 2, d, BF16, lq)
    lengths = torch.tensor([0, 1, 127, 128, 129, 256, 260, 259], dtype=torch.int32)
    want = _compare(gsr, ctx, *args, lengths=lengths)
    assert (want["out"][0][0] == 0).all()
    q, k, v, _ = args
    wild = torch.tensor([-5, 1, 127, 128, 129, 256, 1 << 30, 259], dtype=torch.int32).cuda()
    out, lse = gsr.cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda(), kv_lengths=wild)
    same, lse2 = gsr.cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda(), kv_lengths=lengths.cuda())
    assert torch.equal(out, same) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lq", [1, 4, 140])
@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_masks(gsr, ctx, lq, kind):
    """Scattered masks, one that leaves nothing, one key, whole tiles out, with and without lengths."""
    args = _inputs(5, lq, 515, 4, 2, 64, BF16, lq)
    mask = torch.rand(5, 515, generator=torch.Generator().manual_seed(1)) < 0.5
    mask[1] = False
    mask[2] = False
    mask[2, 300] = True
    mask[3, 64:400] = False
    mask[4] = True
    stored = mask.to(kind) if kind == torch.bool else mask.to(kind) * 7
    _compare(gsr, ctx, *args, mask=stored)
    _compare(gsr, ctx, *args, mask=stored, lengths=torch.tensor([500, 515, 300, 65, 0], dtype=torch.int32))


@pytest.mark.parametrize("lq,lk", [(1, 20000), (3, 9001), (33, 6000), (700, 2100), (2100, 77)])
def test_long(gsr, ctx, lq, lk):
    _compare(gsr, ctx, *_inputs(1, lq, lk, 2, 1, 128, BF16, lk), lengths=torch.tensor([lk - 3], dtype=torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [40, 64, 128])
@pytest.mark.parametrize("b,hq,hk,lq,lk,lengths", [(2, 8, 4, 600, 1000, None), (3, 8, 8, 520, 1300, [1300, 0, 401]),
                                                   (1, 16, 4, 1100, 2100, None), (5, 12, 12, 260, 140, [140, 1, 128, 129, 77])])
def test_many_tiles(gsr, ctx, dtype, d, b, hq, hk, lq, lk, lengths):
    """Several steps per tile and several tiles per SM, whole and cut."""
    lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    _compare(gsr, ctx, *_inputs(b, lq, lk, hq, hk, d, dtype, d + lq), lengths=lengths)


def test_growing_scores_over_many_tiles(gsr, ctx):
    """Scores that grow along the keys, tile after tile, and rows that grow alone."""
    for d in (64, 128):
        q, k, v, dout = _inputs(1, 700, 1500, 8, 8, d, BF16, d)
        k = (k * torch.linspace(0.1, 12.0, 1500)[None, :, None, None]).to(BF16)
        q[:, ::37] *= 4.0
        _compare(gsr, ctx, q, k, v, dout)


def test_large_scores(gsr, ctx):
    """Scores of several hundred: one key takes a row, and the running maximum moves late."""
    q, k, v, dout = _inputs(1, 200, 400, 2, 2, 64, F16, 3, size=30.0)
    k = (k * torch.linspace(0.2, 3.0, 400)[None, :, None, None]).to(F16)
    _compare(gsr, ctx, q, k, v, dout)
    for lq in (1, 200):
        _compare(gsr, ctx, q[:, :lq], k.flip(1), v, dout[:, :lq], scale=0.5)


def test_strides(gsr, ctx):
    """Heads before tokens, packed projections, shared items and heads, gradients written into views."""
    g = torch.Generator().manual_seed(9)
    for lq in (2, 150):
        q = torch.randn(2, 4, lq, 64, generator=g).to(BF16).cuda().transpose(1, 2)
        kv = torch.randn(2, 300, 2, 2, 64, generator=g).to(BF16).cuda()
        dout = torch.randn(2, 4, lq, 64, generator=g).to(BF16).cuda().transpose(1, 2)
        k, v = kv[:, :, 0], kv[:, :, 1]
        shared = torch.randn(1, 300, 1, 64, generator=g).to(BF16).cuda().expand(2, 300, 2, 64)
        for kk, vv in ((k, v), (shared, v), (k[:1].expand_as(k), shared)):
            dense = [t.contiguous() for t in (q, kk, vv, dout)]
            out, lse = gsr.cross_attention_forward(ctx, *dense[:3])
            want = gsr.cross_attention_backward(ctx, *dense[:3], out, lse, dense[3])
            room = torch.zeros(2, 4, lq, 64, dtype=BF16, device="cuda").transpose(1, 2)
            got, lse2 = gsr.cross_attention_forward(ctx, q, kk, vv, out=room)
            assert torch.equal(got, out) and torch.equal(lse, lse2)
            grad = torch.full_like(kv, 7.0)
            dq = torch.zeros(2, 4, lq, 64, dtype=BF16, device="cuda").transpose(1, 2)
            gsr.cross_attention_backward(ctx, q, kk, vv, got, lse2, dout, dl_dq=dq, dl_dk=grad[:, :, 0],
                                         dl_dv=grad[:, :, 1])
            assert torch.equal(dq, want[0]) and torch.equal(grad[:, :, 0], want[1])
            assert torch.equal(grad[:, :, 1], want[2])


def test_same_bits_on_every_run(gsr, ctx):
    for lq, lk in ((1, 5000), (300, 900)):
        q, k, v, dout = (t.cuda() for t in _inputs(2, lq, lk, 8, 2, 128, BF16, 5))
        runs = []
        for _ in range(3):
            out, lse = gsr.cross_attention_forward(ctx, q, k, v)
            runs.append((out, lse) + gsr.cross_attention_backward(ctx, q, k, v, out, lse, dout))
        for run in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(run, runs[0]))


def test_gradient_against_differences(gsr, ctx):
    q, k, v, dout = _inputs(1, 40, 150, 4, 2, 32, F16, 6)
    lengths = torch.tensor([141], dtype=torch.int32)
    valid = _valid(1, 150, lengths, None)
    out, lse = gsr.cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda(), kv_lengths=lengths.cuda())
    grads = gsr.cross_attention_backward(ctx, q.cuda(), k.cuda(), v.cuda(), out, lse, dout.cuda(),
                                         kv_lengths=lengths.cuda())
    args = [q.double(), k.double(), v.double()]
    bounds = ref.attention(*args, valid, 32 ** -0.5, F16, dout.double())
    h = 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(args[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
        ends = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * h * d
            ends.append((ref.attention(*moved, valid, 32 ** -0.5, F16)["out"][0] * dout.double()).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        got = (grads[i].cpu().double() * d).sum()
        assert abs(slope - got) <= (bounds[name][1] * d.abs()).sum() + 1e-6


def test_empty(gsr, ctx):
    q, k, v, dout = (t.cuda() for t in _inputs(2, 5, 7, 2, 1, 64, BF16, 7))
    none = k[:, :0]
    out, lse = gsr.cross_attention_forward(ctx, q, none, none)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = gsr.cross_attention_backward(ctx, q, none, none, out, lse, dout)
    assert (dq == 0).all() and dk.numel() == 0
    out, lse = gsr.cross_attention_forward(ctx, q[:, :0], k, v)
    assert out.numel() == 0
    dq, dk, dv = gsr.cross_attention_backward(ctx, q[:, :0], k, v, out, lse, dout[:, :0])
    assert (dk == 0).all() and (dv == 0).all()
    out, lse = gsr.cross_attention_forward(ctx, q[:0], k[:0], v[:0])
    assert out.numel() == 0 and lse.numel() == 0


def test_other_stream_and_graph(gsr, ctx):
    q, k, v, dout = (t.cuda() for t in _inputs(2, 200, 700, 4, 2, 64, F16, 8))
    mask = (torch.rand(2, 700) < 0.7).cuda()

    def step():
        out, lse = gsr.cross_attention_forward(ctx, q, k, v, key_mask=mask)
        one, lse1 = gsr.cross_attention_forward(ctx, q[:, :1], k, v, key_mask=mask)
        return (out, lse, one, lse1) + gsr.cross_attention_backward(ctx, q, k, v, out, lse, dout, key_mask=mask)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = gsr.cross_attention_forward(ctx, q, k, v, key_mask=mask, stream=side)
    again = step()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(a, b) for a, b in zip(again, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(gsr, ctx):
    q, k, v, dout = (t.cuda() for t in _inputs(2, 5, 7, 2, 1, 64, BF16, 7))
    f = gsr.cross_attention_forward
    for call in (lambda: f(ctx, q[..., :60], k[..., :60], v[..., :60]),                    # head_dim
                 lambda: f(ctx, *(torch.zeros(1, 2, 1, 136, dtype=BF16, device="cuda"),) * 3),
                 lambda: f(ctx, torch.zeros(2, 5, 3, 64, dtype=BF16, device="cuda"), *(k.expand(2, 7, 2, 64),) * 2),
                 lambda: f(ctx, q, k, v, scale=0.0), lambda: f(ctx, q, k, v, scale=-1.0),
                 lambda: f(ctx, q, k, v, scale=float("nan")),
                 lambda: f(ctx, q, k[:, :1].expand_as(k), v),                              # tokens that share memory
                 lambda: f(ctx, torch.zeros(2, 5, 2, 68, dtype=BF16, device="cuda")[..., 4:], k, v),  # alignment
                 lambda: f(ctx, torch.zeros(2, 5, 2, 68, dtype=BF16, device="cuda")[..., :64], k, v),  # strides
                 lambda: f(ctx, q, k, v, out=q[:1].expand_as(q))):
        with pytest.raises(gsr.GsrError) as e:
            call()
        assert e.value.code == 1
    for call in (lambda: f(ctx, q.float(), k.float(), v.float()), lambda: f(ctx, q, k.half(), v),
                 lambda: f(ctx, q, k, v[:, :6]), lambda: f(ctx, q[0], k, v), lambda: f(ctx, q.cpu(), k, v),
                 lambda: f(ctx, q.transpose(2, 3), k, v),
                 lambda: f(ctx, q, k, v, kv_lengths=torch.ones(2, dtype=torch.int64, device="cuda")),
                 lambda: f(ctx, q, k, v, kv_lengths=torch.ones(3, dtype=torch.int32, device="cuda")),
                 lambda: f(ctx, q, k, v, key_mask=torch.ones(2, 6, dtype=torch.bool, device="cuda")),
                 lambda: f(ctx, q, k, v, key_mask=torch.ones(2, 7, device="cuda")),
                 lambda: f(ctx, q, k, v, lse=torch.ones(2, 2, 4, device="cuda"))):
        with pytest.raises(ValueError):
            call()


def test_too_many_steps_are_refused(gsr, ctx):
    q = torch.zeros(1, 1 << 17, 1, 8, dtype=BF16, device="cuda").expand(1, 1 << 17, 1024, 8)
    k = torch.zeros(1, 1 << 24, 1, 8, dtype=BF16, device="cuda")
    with pytest.raises(gsr.GsrError, match="2\\^31 steps") as e:
        gsr.cross_attention_forward(ctx, q, k, k, out=q)
    assert e.value.code == 1


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_of_many_lengths(gsr, ctx, d):
    """More items than a warp has lanes, some without keys, shares that start in any of them."""
    b, lq, lk = 75, 130, 300
    q, k, v, dout = _inputs(b, lq, lk, 2, 1, d, F16, 71)
    lengths = torch.tensor([(37 * i) % 301 if i % 5 else 0 for i in range(b)], dtype=torch.int32)
    _compare(gsr, ctx, q, k, v, dout, lengths=lengths)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_jump_inside_a_tile(gsr, ctx, dtype, d):
    """The largest scores in the second half of a tile, in one key, in a tail, and lower ones behind them."""
    q, k, v, dout = _inputs(2, 300, 700, 2, 1, d, dtype, 5 + d)
    q[..., 0] = 4.0
    level = torch.zeros(700)
    level[64:128], level[192:256], level[300], level[390:450], level[690:] = 10.0, 20.0, 25.0, -15.0, 33.0
    level = torch.stack([level, level.flip(0)])
    k = (0.2 * k).to(dtype)
    k[:, :, 0, 0] = level.to(dtype)
    _compare(gsr, ctx, q, k, v, dout, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq", [4, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity(gsr, ctx, dtype, lq, d):
    """Valid keys whose scores are -inf weigh nothing, the first ones and whole tiles among them."""
    q, k, v, dout = _inputs(2, lq, 400, 2, 1, d, dtype, 6 + d)
    q[..., 0] = 1.0
    none = torch.zeros(2, 400, dtype=torch.bool)
    none[0, :64] = none[0, 100:110] = none[0, 256:384] = True
    none[1, :200] = none[1, 399] = True
    k[none] = 0.0
    want = ref.attention(q.double(), k.double(), v.double(), ~none, d ** -0.5, dtype)
    k[..., 0] = torch.where(none[:, :, None], float("-inf"), k[..., 0])
    out, lse = gsr.cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda())
    ref.check(lse, want["lse"], "lse")
    ref.check(out, want["out"], "out")


@pytest.mark.parametrize("lq,lk,d", [(1, 2066, 104), (3, 1321, 8), (5, 2286, 32)])
def test_small_gradients_of_single_rows(gsr, ctx, lq, lk, d):
    """f16 key gradients of a few queries, most of whose probabilities are far below 1."""
    for seed in range(6):
        q, k, v, dout = _inputs(2, lq, lk, 2, 2, d, F16, seed, size=4.0)
        _compare(gsr, ctx, q, k, v, 1.9 * dout)


def test_gradients_of_large_values(gsr, ctx):
    """f16 values and output gradients whose products pass f16's range."""
    q, k, v, dout = _inputs(1, 150, 300, 2, 1, 128, F16, 8)
    v, dout = (9000.0 * v).clamp(-6e4, 6e4), 0.01 * dout
    valid = torch.ones(1, 300, dtype=torch.bool)
    for factor in (1.0, 1e-3):
        want = ref.attention(q.double(), k.double(), v.double(), valid, 128 ** -0.5, F16, (factor * dout).double())
        dev = [t.cuda() for t in (q, k, v)]
        out, lse = gsr.cross_attention_forward(ctx, *dev)
        grads = gsr.cross_attention_backward(ctx, *dev, out, lse, (factor * dout).cuda())
        for name, got in zip(("dq", "dk", "dv"), grads):
            ref.check(got, want[name], name)
