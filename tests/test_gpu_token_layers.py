"""Token layers as a decoder uses them: norms, recurrences in both directions and attention
in a row, captured, on branches beside each other, and beyond a grid's and 32 bits' limits."""
import glob
import importlib
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import token_layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))


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


# -- a layer: norm, projection, recurrences both ways, residual sum and norm -----------------

def _parameters(c, seed):
    g = torch.Generator().manual_seed(seed)
    p = {"w0": 1 + 0.2 * torch.randn(c, generator=g), "b0": 0.2 * torch.randn(c, generator=g),
         "w1": 1 + 0.2 * torch.randn(c, generator=g), "b1": 0.2 * torch.randn(c, generator=g),
         "to": torch.randn(c, 6 * c, generator=g) / c ** 0.5, "back": torch.randn(2 * c, c, generator=g) / (2 * c) ** 0.5}
    p["to"][:, c:2 * c] *= 0.5
    return p


def _forward(gsr, ctx, x, residual, p, lengths):
    """Returns the outputs and what the backward needs."""
    c = x.shape[2]
    y, total, m0, r0 = gsr.layer_norm_forward(ctx, x, p["w0"], p["b0"], residual=residual)
    proj = y @ p["to"]
    runs = []
    for k, reverse in ((0, False), (3, True)):
        v, f, o = proj[:, :, k * c:(k + 3) * c].split(c, dim=2)
        runs.append(gsr.gated_recurrence_forward(ctx, v, f, o, lengths=lengths, reverse=reverse))
    mixed = torch.cat([runs[0][0], runs[1][0]], dim=2)
    out, total1, m1, r1 = gsr.layer_norm_forward(ctx, mixed @ p["back"], p["w1"], p["b1"], residual=total)
    return (out, total1), (y, total, m0, r0, proj, runs, mixed, m1, r1)


def _backward(gsr, ctx, dout, dtotal1, total1, kept, p, lengths):
    y, total, m0, r0, proj, runs, mixed, m1, r1 = kept
    c = y.shape[2]
    d1, dw1, db1 = gsr.layer_norm_backward(ctx, dout, total1, p["w1"], m1, r1, dl_dtotal=dtotal1)
    dmixed = d1 @ p["back"].T
    dback = mixed.reshape(-1, 2 * c).T @ d1.reshape(-1, c)
    dproj = torch.empty_like(proj)
    for n, (k, reverse) in enumerate(((0, False), (3, True))):
        v, f, o = proj[:, :, k * c:(k + 3) * c].split(c, dim=2)
        gv, gf, go = dproj[:, :, k * c:(k + 3) * c].split(c, dim=2)
        gsr.gated_recurrence_backward(ctx, dmixed[:, :, n * c:(n + 1) * c], v, f, o, runs[n][2], lengths=lengths,
                                      reverse=reverse, dl_dx=gv, dl_dforget=gf, dl_dgate=go)
    dy = dproj @ p["to"].T
    dto = y.reshape(-1, c).T @ dproj.reshape(-1, 6 * c)
    dx, dw0, db0 = gsr.layer_norm_backward(ctx, dy, total, p["w0"], m0, r0, dl_dtotal=d1)
    return {"x": dx, "w0": dw0, "b0": db0, "w1": dw1, "b1": db1, "to": dto, "back": dback}


def _plain(x, residual, p, lengths):
    """The same in 64 bits on the CPU, for autograd."""
    def norm(t, w, b):
        t = t - t.mean(-1, keepdim=True)
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5) * w + b

    c = x.shape[2]
    total = x + residual
    proj = norm(total, p["w0"], p["b0"]) @ p["to"]
    sides = []
    for k, reverse in ((0, False), (3, True)):
        v, f, o = proj[:, :, k * c:(k + 3) * c].split(c, dim=2)
        items = []
        for i, n in enumerate(lengths):
            h, hs = torch.zeros(c, dtype=torch.float64), []
            for t in (range(n - 1, -1, -1) if reverse else range(n)):
                a = torch.sigmoid(f[i, t])
                h = a * h + (1 - a) * v[i, t]
                hs.append(h)
            hs = hs[::-1] if reverse else hs
            hs = torch.stack(hs) if hs else torch.zeros(0, c, dtype=torch.float64)
            items.append(torch.cat([hs, torch.zeros(x.shape[1] - n, c, dtype=torch.float64)]))
        sides.append(torch.stack(items) * torch.nn.functional.silu(o))
    total1 = torch.cat(sides, dim=2) @ p["back"] + total
    return norm(total1, p["w1"], p["b1"]), total1


def test_a_layer_and_its_gradients(gsr, ctx):
    """In float, against autograd in 64 bits.  Each of the layer's eight steps is off by at most
    128 F of its largest values (the operators' own bounds; products of up to 2 c = 96 terms),
    and no step spreads an error by more than 8 times (norms by 1 / sigma of sums of two unit
    normals, projections by the largest singular values of random matrices): 8 * 8 * 128 F."""
    g = torch.Generator().manual_seed(3)
    b, n, c = 3, 200, 48
    x, residual, dout, dtotal = (torch.randn(b, n, c, generator=g) for _ in range(4))
    lens = [200, 0, 131]
    p = _parameters(c, 4)
    dev = {k: v.cuda() for k, v in p.items()}
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    torch.backends.cuda.matmul.allow_tf32 = False
    (out, total1), kept = _forward(gsr, ctx, x.cuda(), residual.cuda(), dev, lengths)
    got = _backward(gsr, ctx, dout.cuda(), dtotal.cuda(), total1, kept, dev, lengths)
    wide = {k: v.double().requires_grad_() for k, v in p.items()}
    wide["x"] = x.double().requires_grad_()
    want, want_total = _plain(wide["x"], residual.double(), wide, lens)
    ((want * dout).sum() + (want_total * dtotal).sum()).backward()
    pairs = [("out", out, want.detach()), ("total", total1, want_total.detach())]
    pairs += [(k, got[k], wide[k].grad) for k in got]
    for name, a, w in pairs:
        error = (a.cpu().double() - w).abs().max() / w.abs().max()
        assert error <= 64 * 128 * ref.F, (name, float(error))


# -- graphs, streams, other kernels --------------------------------------------------------------

def _step(gsr, ctx, seed, tokens, c, dtype=BF16):
    """A layer's operators and their gradients, as a function of a stream."""
    g = torch.Generator().manual_seed(seed)
    x, r, dout = (torch.randn(2, tokens, c, generator=g).to(dtype).cuda() for _ in range(3))
    whole = torch.randn(2, tokens, 3 * c, generator=g)
    whole[:, :, c:2 * c] += 3
    v, f, o = whole.to(dtype).cuda().split(c, dim=2)
    w = torch.ones(c, device="cuda")
    lengths = torch.tensor([tokens, tokens // 3], dtype=torch.int32, device="cuda")

    def step(stream=None):
        y, total, mean, rstd = gsr.layer_norm_forward(ctx, x, w, w, residual=r, stream=stream)
        results = [y, total, mean, rstd]
        results += gsr.layer_norm_backward(ctx, dout, total, w, mean, rstd, dl_dtotal=y, stream=stream)
        for reverse in (False, True):
            run = gsr.gated_recurrence_forward(ctx, v, f, o, lengths=lengths, reverse=reverse, stream=stream)
            results += run[:2]
            results += gsr.gated_recurrence_backward(ctx, dout, v, f, o, run[2], lengths=lengths, reverse=reverse,
                                                     stream=stream)
        one = gsr.gated_recurrence_forward(ctx, v[:, :1], f[:, :1], o[:, :1], initial=run[1], keep=False, stream=stream)
        return results + list(one[:2])

    return step


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_share_a_workspace(gsr, ctx):
    steps = [_step(gsr, ctx, 1, 700, 64), _step(gsr, ctx, 2, 3000, 130)]
    want = [step() for step in steps]
    graphs, got = [], []
    for step in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step())
    # The workspace grows behind both; what others hold meanwhile stays as it is.
    larger = _step(gsr, ctx, 3, 20000, 256)
    first = larger()
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(32)]
    for k in (0, 1, 1, 0):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert _same(got[k], want[k])
    assert _same(larger(), first) and all((t == 7).all() for t in others)
    ctx.synchronize()


def test_streams_of_one_context(gsr, ctx):
    steps = [_step(gsr, ctx, 10 + i, 500 + 700 * i, 64 + 33 * i, (BF16, F32, F16)[i]) for i in range(3)]
    want = [step() for step in steps]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = []
        for side, step in zip(sides, steps):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                got.append(step())
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, want))
    assert _same(steps[0](sides[1]), want[0])
    ctx.synchronize()


def test_recurrences_beside_attention(gsr, ctx):
    """Contexts of their own on branches of one graph: recurrences beside each other and beside
    attention, which both take tensor memory, shared memory and whole SMs."""
    contexts = [ctx] + [gsr.Context(0) for _ in range(3)]
    steps = [_step(gsr, c, 20 + i, 2500 + 900 * i, 128 + 64 * i) for i, c in enumerate(contexts[:3])]
    g = torch.Generator().manual_seed(5)
    q = torch.randn(2, 900, 8, 128, generator=g).to(BF16).cuda()
    k, v = (torch.randn(2, 3000, 4, 128, generator=g).to(BF16).cuda() for _ in range(2))

    def attend():
        out, lse = gsr.cross_attention_forward(contexts[3], q, k, v)
        return (out, lse, *gsr.cross_attention_backward(contexts[3], q, k, v, out, lse, q))

    work = steps + [attend]
    want = [f() for f in work]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in work[1:]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for side in sides:
            side.wait_stream(main)
        got = [[work[0]() for _ in range(3)]]
        for side, f in zip(sides, work[1:]):
            with torch.cuda.stream(side):
                got.append([f() for _ in range(3)])
        for side in sides:
            main.wait_stream(side)
    for _ in range(20):
        for runs in got:
            for run in runs:
                for t in run:
                    t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(_same(run, w) for runs, w in zip(got, want) for run in runs)
    for c in contexts:
        c.synchronize()
    for c in contexts[1:]:
        c.close()


def _held_up(tmp_path, name, helper):
    """The outputs of a helper over a build in which the warps of one source sleep pseudo-random
    times, and those of this one."""
    from gaussian_splatting_tile_bin_gb300 import build as b
    source, obj, lib = os.path.join(b.CSRC, name), str(tmp_path / "held_up.o"), str(tmp_path / "libgsr.so")
    objects = [o for o in glob.glob(os.path.join(b.BUILD, "*.o")) if os.path.basename(o) != name + ".o"]
    assert len(objects) == len(b.sources()) - 1
    subprocess.check_call([b._nvcc(), *b.NVCC_FLAGS, "-DGSR_RACE_CANARY", "-c", source, "-o", obj])
    subprocess.check_call([b._nvcc(), *b.ARCH, "-shared", "-o", lib, obj, *objects])
    out = tmp_path / "canary.npz"
    r = subprocess.run([sys.executable, os.path.join(HERE, helper + ".py"), str(out)],
                       env=dict(os.environ, GSR_LIBRARY=lib), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    sys.path.insert(0, HERE)
    want, got = importlib.import_module(helper).outputs(), np.load(out)
    assert set(got.files) == set(want)
    for name, value in want.items():
        assert np.array_equal(got[name].view(np.uint8), value.view(np.uint8)), name


def test_warps_that_are_held_up_change_no_bit(gsr, tmp_path):
    """Where the recurrence's wait for and hand over maps and states."""
    _held_up(tmp_path, "recurrence.cu", "recurrence_canary_run")


def test_blocks_that_share_rows_are_held_up(gsr, tmp_path):
    """Where the layer norm's warps hand their sums to the other block of a row."""
    _held_up(tmp_path, "layernorm.cu", "layer_norm_canary_run")


# -- sizes -----------------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_(t-1) + b_t along dimension 1, in 64 bits by doubling."""
    a, b = a.clone(), b.clone()
    shift = 1
    while shift < a.shape[1]:
        b[:, shift:] = b[:, shift:] + a[:, shift:] * b[:, :-shift]
        a[:, shift:] = a[:, shift:] * a[:, :-shift]
        shift *= 2
    return b


def _check_long(gsr, ctx, b, n, c, dtype, keep):
    """Values and gradients within the bounds of a recurrence whose steps are off by `step` against
    magnitudes of at most `top`: an error lives as long as the state does, at most 1 / (1 - a)."""
    g = torch.Generator("cuda").manual_seed(n + c)
    x, f, dout = (torch.randn(b, n, c, generator=g, device="cuda") for _ in range(3))
    f = (f.clamp(-2, 2) + keep).to(dtype)
    x, dout = x.to(dtype), dout.to(dtype)
    out, final, states = gsr.gated_recurrence_forward(ctx, x, f)
    dx, df, _, first = gsr.gated_recurrence_backward(ctx, dout, x, f, None, states)
    a, s = torch.sigmoid(f.double()), torch.sigmoid(-f.double())
    h = _scan(a, s * x.double())
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    dh = _scan(after.flip(1), dout.double().flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    rel = (2 * f.double().abs() + 12) * ref.F
    life = 1 / s.min()
    top, top_g = x.double().abs().max(), dh.abs().max()
    e_h = life * 2 * (rel.max() * torch.minimum(a, s).max() * 2 + 4 * ref.F) * top
    e_g = life * 2 * (rel.max() * torch.minimum(a, s).max() + 4 * ref.F) * 2 * top_g
    for got, want, bound in ((out, h, e_h), (final, h[:, -1], e_h), (dx, dh * s, e_g * s + 8 * rel * (dh * s).abs()),
                             (df, dh * (before - x.double()) * a * s,
                              (e_g * (before - x.double()).abs() + dh.abs() * 2 * e_h) * a * s
                              + 8 * rel * (dh * (before - x.double()) * a * s).abs())):
        error = (got.double() - want).abs()
        assert (error <= bound + ref.rounding(want, got.dtype)).all(), float((error - bound).max())


@pytest.mark.parametrize("b,n,c,dtype,keep", [(1, 1 << 20, 3, F32, 1.0), (1, 300001, 2, BF16, 4.0), (65536, 17, 2, F16, 1.0),
                                              (1, 130, 65536, BF16, 1.0), (20000, 130, 1, F32, 1.0), (3, 40000, 66, BF16, 6.0)])
def test_long_and_wide_recurrences(gsr, ctx, b, n, c, dtype, keep):
    _check_long(gsr, ctx, b, n, c, dtype, keep)


def test_more_rows_than_a_grid_has(gsr, ctx):
    """70 million short rows: rows, copies ahead of them and the sums over all of them."""
    n, c = 70_000_003, 2
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(n, c, generator=g, device="cuda").to(F16)
    out, total, mean, rstd = gsr.layer_norm_forward(ctx, x)
    assert total is x
    rows = torch.cat([torch.arange(1000), torch.arange(n - 1000, n)]).cuda()
    want = ref.layer_norm(x[rows].cpu().double(), None, None, 1e-5, F16)
    ref.check(out[rows], want["out"], "out")
    ref.check(mean[rows], want["mean"], "mean")
    dx, dw, db = gsr.layer_norm_backward(ctx, torch.ones_like(x), x, None, mean, rstd)
    # dL/dout = 1 has nothing left after its mean; each block's count is exact, their sum's tree
    # rounds a dozen times.
    assert ((db.double() - n).abs() <= 12 * ref.F * n).all() and (dx.float().abs() <= 1e-3).all()
    hats = ((x.float() - mean[:, None]) * rstd[:, None]).double().sum(0)
    assert ((dw.double() - hats).abs() <= 1e-6 * n).all()


def test_projection_parts_across_devices_memory(gsr, ctx):
    """Items of a batch more than 2^32 elements apart."""
    b, n, c = 3, 200, 32
    stride = (1 << 31) + 64
    base = torch.empty(2 * stride + 8 * n * c, dtype=BF16, device="cuda")
    g = torch.Generator().manual_seed(8)
    near = [torch.randn(b, n, c, generator=g).to(BF16).cuda() for _ in range(4)]
    far = [base.as_strided((b, n, c), (stride, c, 1), i * n * c) for i in range(8)]
    for to, t in zip(far, near):
        to.copy_(t)
    out, final, states = gsr.gated_recurrence_forward(ctx, *near[:3])
    got, end, kept = gsr.gated_recurrence_forward(ctx, *far[:3], out=far[4])
    assert torch.equal(got, out) and torch.equal(end, final) and torch.equal(kept, states)
    grads = gsr.gated_recurrence_backward(ctx, near[3], *near[:3], states)
    same = gsr.gated_recurrence_backward(ctx, far[3], *far[:3], states, dl_dx=far[5], dl_dforget=far[6], dl_dgate=far[7])
    assert all(torch.equal(p, q) for p, q in zip(same, grads))
