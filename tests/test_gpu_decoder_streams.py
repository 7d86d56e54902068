"""The decoder operators' workspace under captured graphs and several streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gsr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_tile_bin_gb300 as g
    return g


@pytest.fixture
def ctx(gsr):
    c = gsr.Context(0)
    yield c
    torch.cuda.synchronize()
    c.close()


def _step(gsr, ctx, lq, lk, seed, dtype=torch.float16):
    """A masked attention step and a norm's, forward and backward, as a function of a stream."""
    g = torch.Generator().manual_seed(seed)
    q, dout = (torch.randn(2, lq, 4, 64, generator=g).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn(2, lk, 2, 64, generator=g).to(dtype).cuda() for _ in range(2))
    mask = (torch.rand(2, lk, generator=g) < 0.7).cuda()
    x, dy = (torch.randn(2, 5 * lk, 96, generator=g).to(dtype).cuda() for _ in range(2))

    def step(stream=None):
        out, lse = gsr.cross_attention_forward(ctx, q, k, v, key_mask=mask, stream=stream)
        grads = gsr.cross_attention_backward(ctx, q, k, v, out, lse, dout, key_mask=mask, stream=stream)
        y, mean, rstd = gsr.group_norm_forward(ctx, x, 6, stream=stream)
        norm_grads = gsr.group_norm_backward(ctx, dy, x, 6, None, None, mean, rstd, stream=stream)
        one, lse1 = gsr.cross_attention_forward(ctx, q[:, :1], k, v, key_mask=mask, stream=stream)
        return (out, lse, *grads, y, mean, rstd, *norm_grads, one, lse1)

    return step


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_replay_after_the_workspace_has_grown(gsr, ctx):
    step = _step(gsr, ctx, 200, 700, 1)
    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert _same(got, want)
    larger = _step(gsr, ctx, 1500, 6000, 2)
    first = larger()
    # Memory that other tensors take meanwhile keeps what they hold.
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for t in got:
        t.zero_()
    graph.replay()
    second = larger()
    graph.replay()
    torch.cuda.synchronize()
    assert _same(got, want) and _same(second, first)
    assert all((t == 7).all() for t in others)


def test_streams_of_one_capture(gsr, ctx):
    """Steps on forked streams of one capture share the context's workspace."""
    steps = [_step(gsr, ctx, 300 + 40 * i, 900 + 100 * i, 10 + i) for i in range(3)]
    want = [step() for step in steps]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in steps[1:]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for side in sides:
            side.wait_stream(main)
        got = [steps[0]()]
        for step, side in zip(steps[1:], sides):
            with torch.cuda.stream(side):
                got.append(step())
        again = steps[0]()
        for side in sides:
            main.wait_stream(side)
    for _ in range(3):
        for t in [t for one in got for t in one] + list(again):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, want)) and _same(again, want[0])


def test_synchronize(gsr, ctx):
    ctx.synchronize()
    step = _step(gsr, ctx, 200, 300, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    ctx.synchronize(side)
    assert side.query() and _same(step(), got)
    ctx.synchronize()


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_beside_other_kernels(gsr, ctx, d):
    """Few rows against more tiles than their ring has stages, on branches of a graph beside
    kernels that fill the SMs: warps that are held up at any point."""
    g = torch.Generator().manual_seed(d)
    few = []
    for lk in (300, 450, 700):
        q = torch.randn(3, 3, 4, d, generator=g).bfloat16().cuda()
        k, v = (torch.randn(3, lk, 4, d, generator=g).bfloat16().cuda() for _ in range(2))
        few.append((q, k, v, gsr.cross_attention_forward(ctx, q, k, v)))
    big = _step(gsr, ctx, 300, 2000, 3, torch.bfloat16)
    want = big()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in few]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        got = [[] for _ in few]
        for side in sides:
            side.wait_stream(main)
        heavy = [big(), big()]
        for (q, k, v, _), side, outs in zip(few, sides, got):
            with torch.cuda.stream(side):
                outs += [gsr.cross_attention_forward(ctx, q, k, v) for _ in range(20)]
        for side in sides:
            main.wait_stream(side)
    for _ in range(40):
        for outs in got:
            for out, _ in outs:
                out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(_same(one, f[3]) for f, outs in zip(few, got) for one in outs)
        assert all(_same(h, want) for h in heavy)
