"""The gated linear recurrence against its 64-bit form, forward and backward."""
import pytest
import torch

import token_layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("dx", "dforget", "dgate", "dinitial")


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


def _inputs(b, n, c, dtype, seed, gate=True, state=True, keep=2.0):
    g = torch.Generator().manual_seed(seed)
    x, f, o, dout = (torch.randn(b, n, c, generator=g) for _ in range(4))
    f = 2.0 * f + keep
    first, last = torch.randn(b, c, generator=g), torch.randn(b, c, generator=g)
    x, f, o, dout = (t.to(dtype) for t in (x, f, o, dout))
    return dict(x=x, forget=f, gate=o if gate else None, dout=dout, initial=first if state else None,
                dfinal=last if state else None)


def _dev(t):
    return None if t is None else t.cuda()


def _run(gsr, ctx, t, lengths=None, reverse=False, place=_dev):
    at = {k: place(v) if k in ("x", "forget", "gate", "dout") else _dev(v) for k, v in t.items()}
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    how = dict(lengths=lens, reverse=reverse)
    out, final, states = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=at["initial"], **how)
    grads = gsr.gated_recurrence_backward(ctx, at["dout"], at["x"], at["forget"], at["gate"], states,
                                          dl_dfinal=at["dfinal"], **how)
    return dict(zip(("out", "final") + NAMES, (out, final) + grads))


def _want(t, lengths=None, reverse=False):
    b, n, _ = t["x"].shape
    lens = [n] * b if lengths is None else [min(max(v, 0), n) for v in lengths]
    wide = {k: None if v is None else v.double() for k, v in t.items()}
    return ref.recurrence(wide["x"], wide["forget"], wide["gate"], wide["initial"], lens, reverse, t["x"].dtype,
                          dout=wide["dout"], dfinal=wide["dfinal"])


def _compare(gsr, ctx, t, lengths=None, reverse=False, place=_dev):
    got, want = _run(gsr, ctx, t, lengths, reverse, place), _want(t, lengths, reverse)
    assert (got["dgate"] is None) == (t["gate"] is None)
    for name, value in want.items():
        ref.check(got[name], value, name)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 513])
def test_parity(gsr, ctx, dtype, reverse, n):
    for c, gate, state in ((66, True, True), (5, False, False), (64, True, False)):
        _compare(gsr, ctx, _inputs(2, n, c, dtype, 10 * n + c, gate, state), reverse=reverse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 2, 3, 31, 32, 33, 63, 64, 65, 77, 127, 128, 130, 250, 512, 1280])
def test_channels(gsr, ctx, dtype, c):
    _compare(gsr, ctx, _inputs(3, 150, c, dtype, c), lengths=[150, 3, 66], reverse=c % 2 == 1)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4095, 4096, 4097, 9001])
@pytest.mark.parametrize("reverse", [False, True])
def test_long(gsr, ctx, n, reverse):
    """Many blocks of tokens, and what joins them."""
    for dtype in (F32, BF16):
        _compare(gsr, ctx, _inputs(2, n, 10, dtype, n), lengths=[n, n - 70], reverse=reverse)


def test_memory_over_many_blocks(gsr, ctx):
    """Forget gates near 1: the first state reaches the last token, and its gradient the first."""
    for reverse in (False, True):
        t = _inputs(1, 6000, 8, F32, 21, keep=12.0)
        _compare(gsr, ctx, t, reverse=reverse)
        t["x"] = torch.zeros_like(t["x"])
        _compare(gsr, ctx, t, reverse=reverse)


@pytest.mark.parametrize("reverse", [False, True])
def test_lengths(gsr, ctx, reverse):
    """Items without tokens, with one, at and around the ends of blocks; lengths out of range
    are clamped; what lies behind an item's length is not read, and its results are 0."""
    lengths = [0, 1, 2, 63, 64, 65, 128, 129, 299, 300, 301, -5]
    for dtype in (F32, F16):
        t = _inputs(len(lengths), 300, 70, dtype, 22)
        want = _want(t, lengths, reverse)
        for i, n in enumerate(lengths):
            for k in ("x", "forget", "gate", "dout"):
                t[k][i, max(n, 0):] = float("nan")
        got = _run(gsr, ctx, t, lengths, reverse)
        for name, value in want.items():
            ref.check(got[name], value, name)


def test_no_states_behind_an_items_length(gsr, ctx):
    """The blocks behind the last token are left as they were, and not read."""
    t = {k: _dev(v) for k, v in _inputs(3, 200, 34, F32, 23).items()}
    lengths = torch.tensor([200, 0, 64], dtype=torch.int32, device="cuda")
    states = torch.full((3, 4, 34), float("nan"), device="cuda")
    gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"], initial=t["initial"], lengths=lengths, states=states)
    assert torch.isnan(states[1]).all() and torch.isnan(states[2, 1:]).all()
    assert not torch.isnan(states[0]).any() and torch.equal(states[[0, 2], 0], t["initial"][[0, 2]])
    grads = gsr.gated_recurrence_backward(ctx, t["dout"], t["x"], t["forget"], t["gate"], states, lengths=lengths)
    assert not any(torch.isnan(g).any() for g in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_one_by_one(gsr, ctx, dtype):
    """Single tokens, each from the state behind the last, give what the sequence gives."""
    t = _inputs(3, 20, 130, dtype, 24)
    want = _want(t)
    t = {k: _dev(v) for k, v in t.items()}
    state, outs = t["initial"].clone(), []
    for k in range(20):
        one = [t[n][:, k:k + 1] for n in ("x", "forget", "gate")]
        out, new, states = gsr.gated_recurrence_forward(ctx, *one, initial=state, keep=False, final=state)
        assert states is None and new is state
        outs.append(out)
    ref.check(torch.cat(outs, 1), want["out"], "out")
    ref.check(state, want["final"], "final")


def test_pieces_of_a_sequence(gsr, ctx):
    """A sequence cut in two, forward state and backward gradient handed over, within both bounds."""
    t = _inputs(2, 500, 40, F32, 25)
    want = _want(t)
    d = {k: _dev(v) for k, v in t.items()}
    parts = [{k: d[k][:, s].contiguous() for k in ("x", "forget", "gate", "dout")} for s in (slice(0, 210), slice(210, 500))]
    state, runs = d["initial"], []
    for p in parts:
        out, state, states = gsr.gated_recurrence_forward(ctx, p["x"], p["forget"], p["gate"], initial=state)
        runs.append((out, states))
    grad, grads = d["dfinal"], []
    for p, (_, states) in zip(parts[::-1], runs[::-1]):
        *g, grad = gsr.gated_recurrence_backward(ctx, p["dout"], p["x"], p["forget"], p["gate"], states, dl_dfinal=grad)
        grads.insert(0, g)
    ref.check(torch.cat([r[0] for r in runs], 1), want["out"], "out")
    ref.check(state, want["final"], "final")
    for i, name in enumerate(NAMES[:3]):
        ref.check(torch.cat([g[i] for g in grads], 1), want[name], name)
    ref.check(grad, want["dinitial"], "dinitial")


@pytest.mark.parametrize("dtype", [F32, F16])
def test_parts_of_a_projection(gsr, ctx, dtype):
    """Values, forget and gate logits as slices of one projection, even and odd widths; the
    gradients go into slices of its gradient."""
    for c in (64, 33):
        t = _inputs(2, 140, c, dtype, 26 + c)
        whole = torch.cat([t["x"], t["forget"], t["gate"]], dim=2).cuda()
        grad = torch.zeros_like(whole)
        x, f, o = whole.split(c, dim=2)
        lengths = torch.tensor([140, 81], dtype=torch.int32, device="cuda")
        out, final, states = gsr.gated_recurrence_forward(ctx, x, f, o, initial=_dev(t["initial"]), lengths=lengths)
        gx, gf, go = grad.split(c, dim=2)
        grad.fill_(7.0)
        gsr.gated_recurrence_backward(ctx, _dev(t["dout"]), x, f, o, states, dl_dfinal=_dev(t["dfinal"]), lengths=lengths,
                                      dl_dx=gx, dl_dforget=gf, dl_dgate=go)
        want = _want(t, [140, 81])
        ref.check(out, want["out"], "out")
        for name, part in zip(NAMES, (gx, gf, go)):
            ref.check(part, want[name], name)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_arrays(gsr, ctx, shift):
    def place(t):
        if t is None:
            return None
        base = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        return base[shift:].view(t.shape).copy_(t)

    for dtype in (BF16, F32):
        _compare(gsr, ctx, _inputs(2, 131, 64, dtype, 27), place=place)


def test_values_that_items_share(gsr, ctx):
    """Inputs with a stride of 0 over the batch."""
    t = _inputs(3, 90, 20, F32, 28)
    for k in ("x", "gate"):
        t[k] = t[k][:1].expand(3, 90, 20)
    at = {k: (v[:1].cuda().expand(3, 90, 20) if k in ("x", "gate") else _dev(v)) for k, v in t.items()}
    out, final, states = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=at["initial"])
    grads = gsr.gated_recurrence_backward(ctx, at["dout"], at["x"], at["forget"], at["gate"], states, dl_dfinal=at["dfinal"])
    want = _want(t)
    for name, got in zip(("out", "final") + NAMES, (out, final) + grads):
        ref.check(got, want[name], name)


def test_in_place(gsr, ctx):
    t = {k: _dev(v) for k, v in _inputs(2, 700, 66, BF16, 29).items()}
    out, final, states = gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"], initial=t["initial"])
    grads = gsr.gated_recurrence_backward(ctx, t["dout"], t["x"], t["forget"], t["gate"], states, dl_dfinal=t["dfinal"])
    d, last = t["dout"].clone(), t["dfinal"].clone()
    same = gsr.gated_recurrence_backward(ctx, d, t["x"], t["forget"], t["gate"], states, dl_dfinal=last, dl_dx=d,
                                         dl_dinitial=last)
    assert same[0].data_ptr() == d.data_ptr() and same[3].data_ptr() == last.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(same, grads))
    for name in ("x", "forget", "gate"):
        at = {k: v.clone() for k, v in t.items()}
        y, end, _ = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=at["initial"],
                                                 out=at[name], final=at["initial"])
        assert torch.equal(y, out) and torch.equal(end, final)


def test_extreme_logits(gsr, ctx):
    """Gates that are fully open or shut, at the types' largest values and infinities."""
    for dtype in (F32, BF16, F16):
        t = _inputs(1, 140, 12, dtype, 30)
        top = 6e4 if dtype == F16 else 1e30
        for row, value in ((3, top), (5, -top), (60, 100.0), (66, -100.0), (70, 20.0), (71, -20.0), (100, float("inf")),
                           (101, -float("inf"))):
            t["forget"][0, row] = value
        t["gate"][0, 9], t["gate"][0, 80] = 80.0, -80.0
        _compare(gsr, ctx, t)
        _compare(gsr, ctx, t, reverse=True)


def test_not_finite_stays_in_its_channel(gsr, ctx):
    t = {k: _dev(v) for k, v in _inputs(2, 300, 40, F32, 31).items()}
    clean, end, _ = gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"])
    t["x"][0, 100, 5], t["forget"][1, 200, 7] = float("nan"), float("nan")
    out, final, states = gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"])
    bad = torch.zeros(2, 300, 40, dtype=torch.bool, device="cuda")
    bad[0, 100:, 5] = bad[1, 200:, 7] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])
    assert torch.isnan(final[0, 5]) and torch.isnan(final[1, 7]) and torch.isnan(final).sum() == 2
    grads = gsr.gated_recurrence_backward(ctx, t["dout"], t["x"], t["forget"], t["gate"], states)
    for g in grads[:3]:
        where = torch.isnan(g).any(dim=1)
        assert where[0].nonzero().flatten().tolist() in ([], [5]) and where[1].nonzero().flatten().tolist() in ([], [7])


def test_same_bits_on_every_run(gsr, ctx):
    t = _inputs(3, 3000, 130, BF16, 32)
    runs = [_run(gsr, ctx, t, [3000, 2000, 1111], True) for _ in range(4)]
    for run in runs[1:]:
        assert all(torch.equal(run[k], runs[0][k]) for k in run)


def test_gradient_against_differences(gsr, ctx):
    t = _inputs(2, 70, 6, F32, 33)
    lengths = [70, 41]
    got, bounds = _run(gsr, ctx, t, lengths, True), _want(t, lengths, True)
    keys = ("x", "forget", "gate", "initial")
    args = [t[k].double() for k in keys]

    def loss(x, f, o, first):
        r = ref.recurrence(x, f, o, first, lengths, True, F32)
        return (r["out"][0] * t["dout"]).sum() + (r["final"][0] * t["dfinal"]).sum()

    h = 1e-5
    for i, name in enumerate(NAMES):
        d = torch.randn(args[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
        ends = [loss(*args[:i], args[i] + sign * h * d, *args[i + 1:]) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(slope - (got[name].cpu().double() * d).sum()) <= (bounds[name][1] * d.abs()).sum() + 1e-6, name


def test_on_another_stream(gsr, ctx):
    t = {k: _dev(v) for k, v in _inputs(2, 2500, 66, F16, 34).items()}
    args = (t["x"], t["forget"], t["gate"])
    first = gsr.gated_recurrence_forward(ctx, *args, initial=t["initial"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = gsr.gated_recurrence_forward(ctx, *args, initial=t["initial"], stream=side)
    third = gsr.gated_recurrence_forward(ctx, *args, initial=t["initial"])
    torch.cuda.synchronize()
    for other in (second, third):
        assert all(torch.equal(p, q) for p, q in zip(first, other))


def test_captured(gsr, ctx):
    """A step in a graph, replayed over new inputs."""
    t = {k: _dev(v) for k, v in _inputs(2, 1500, 66, BF16, 35).items()}

    def step():
        out, final, states = gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"], initial=t["initial"])
        return (out, final) + gsr.gated_recurrence_backward(ctx, t["dout"], t["x"], t["forget"], t["gate"], states,
                                                            dl_dfinal=t["dfinal"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (36, 37, 38):
        for k, v in _inputs(2, 1500, 66, BF16, seed).items():
            t[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_offsets_beyond_32_bits(gsr, ctx):
    """Tokens more than 2^31 elements apart over the whole sequence."""
    n, c = 130, 16
    token = (1 << 32) // n // 64 * 64
    base = torch.empty((1 << 32) + 4096, dtype=BF16, device="cuda")
    t = {k: _dev(v) for k, v in _inputs(1, n, c, BF16, 39).items()}
    far = [base.as_strided((1, n, c), (n * token, token, 1), 64 * i) for i in range(7)]
    for place, k in zip(far, ("x", "forget", "gate", "dout")):
        place.copy_(t[k])
    want, end, states = gsr.gated_recurrence_forward(ctx, t["x"], t["forget"], t["gate"])
    got, _, _ = gsr.gated_recurrence_forward(ctx, *far[:3], out=far[4])
    assert torch.equal(got, want)
    grads = gsr.gated_recurrence_backward(ctx, t["dout"], t["x"], t["forget"], t["gate"], states)
    same = gsr.gated_recurrence_backward(ctx, far[3], *far[:3], states, dl_dx=far[4], dl_dforget=far[5], dl_dgate=far[6])
    assert all(torch.equal(p, q) for p, q in zip(same, grads))


def test_empty(gsr, ctx):
    x = torch.empty(2, 0, 16, device="cuda")
    first = torch.randn(2, 16, device="cuda")
    out, final, states = gsr.gated_recurrence_forward(ctx, x, x, initial=first)
    assert out.shape == x.shape and torch.equal(final, first) and states.shape == (2, 0, 16)
    out, final, _ = gsr.gated_recurrence_forward(ctx, x, x)
    assert (final == 0).all()
    *_, back = gsr.gated_recurrence_backward(ctx, x, x, x, None, states, dl_dfinal=first)
    assert torch.equal(back, first)
    none = torch.empty(0, 5, 16, device="cuda")
    out, final, _ = gsr.gated_recurrence_forward(ctx, none, none)
    assert out.shape == none.shape and final.shape == (0, 16)


def test_refusals(gsr, ctx):
    x = torch.randn(2, 5, 16, device="cuda")
    state = torch.zeros(2, 16, device="cuda")
    states = torch.zeros(2, 1, 16, device="cuda")
    with pytest.raises(gsr.GsrError):
        gsr.gated_recurrence_forward(ctx, x, x, out=torch.empty(5, 16, device="cuda").expand(2, 5, 16))
    with pytest.raises(gsr.GsrError):
        wide = torch.zeros(1, 1, 65537, device="cuda")
        gsr.gated_recurrence_forward(ctx, wide, wide)
    for call in (lambda: gsr.gated_recurrence_forward(ctx, x.cpu(), x),
                 lambda: gsr.gated_recurrence_forward(ctx, x.double(), x),
                 lambda: gsr.gated_recurrence_forward(ctx, x[0], x[0]),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x.half()),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x[:, :4]),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x, x[:1]),
                 lambda: gsr.gated_recurrence_forward(ctx, x.transpose(1, 2), x.transpose(1, 2)),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x, initial=state.half()),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x, initial=state[:1]),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x, lengths=torch.zeros(2, device="cuda")),
                 lambda: gsr.gated_recurrence_forward(ctx, x, x, keep=False, states=states),
                 lambda: gsr.gated_recurrence_backward(ctx, x, x, x, None, states, dl_dgate=x),
                 lambda: gsr.gated_recurrence_backward(ctx, x, x, x, None, states[:, :0]),
                 lambda: gsr.gated_recurrence_backward(ctx, x, x, x, x, state)):
        with pytest.raises(ValueError):
            call()
