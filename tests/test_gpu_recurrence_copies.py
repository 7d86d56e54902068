"""The gated recurrence over arrays that its tiles are copied from in bulk: channels in whole
16 bytes, every end of a tile and of a group of tiles, both directions, ragged items, in place."""
import pytest
import torch

from test_gpu_gated_recurrence import BF16, F16, F32, NAMES, _compare, _dev, _inputs, _run, _want, ctx, gsr  # noqa: F401
import token_layer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("c", [8, 16, 24, 56, 64, 72, 128, 136])
def test_widths(gsr, ctx, dtype, reverse, c):  # noqa: F811
    _compare(gsr, ctx, _inputs(3, 270, c, dtype, c, gate=c % 16 == 0), lengths=[270, 129, 65], reverse=reverse)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n", [17, 64, 65, 127, 128, 129, 191, 192, 193, 511, 512, 513, 1023, 1024, 1025, 1153, 2048, 2049, 2177,
                               3101, 4097])
def test_ends_of_tiles_and_groups(gsr, ctx, n, reverse):  # noqa: F811
    for dtype, c in ((F32, 4), (BF16, 8)):
        _compare(gsr, ctx, _inputs(1, n, c, dtype, n), reverse=reverse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reverse", [False, True])
def test_ragged_items(gsr, ctx, dtype, reverse):  # noqa: F811
    """Lengths at and around the ends of tiles; what lies behind them is not a number and reaches
    nothing."""
    lengths = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1024, 1025, 1100, -3, 5000]
    t = _inputs(len(lengths), 1100, 16, dtype, 41)
    want = _want(t, lengths, reverse)
    for i, n in enumerate(lengths):
        for k in ("x", "forget", "gate", "dout"):
            t[k][i, max(n, 0):] = float("nan")
    got = _run(gsr, ctx, t, lengths, reverse)
    for name, value in want.items():
        ref.check(got[name], value, name)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_in_place(gsr, ctx, dtype, reverse):  # noqa: F811
    t = {k: _dev(v) for k, v in _inputs(3, 1500, 64, dtype, 42).items()}
    how = dict(lengths=torch.tensor([1500, 700, 1333], dtype=torch.int32, device="cuda"), reverse=reverse)
    args = (t["x"], t["forget"], t["gate"])
    out, final, states = gsr.gated_recurrence_forward(ctx, *args, initial=t["initial"], **how)
    grads = gsr.gated_recurrence_backward(ctx, t["dout"], *args, states, dl_dfinal=t["dfinal"], **how)
    for _ in range(3):
        for name in ("x", "forget", "gate"):
            at = {k: v.clone() for k, v in t.items()}
            y, end, _ = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=at["initial"],
                                                     out=at[name], final=at["initial"], **how)
            assert torch.equal(y, out) and torch.equal(end, final)
        d, last = t["dout"].clone(), t["dfinal"].clone()
        same = gsr.gated_recurrence_backward(ctx, d, *args, states, dl_dfinal=last, dl_dx=d, dl_dinitial=last, **how)
        assert same[0].data_ptr() == d.data_ptr() and all(torch.equal(a, b) for a, b in zip(same, grads))


def test_shared_and_strided_items(gsr, ctx):  # noqa: F811
    """Inputs of one item for all, and every second token of a wider array."""
    t = _inputs(3, 300, 32, BF16, 43)
    for k in ("x", "gate"):
        t[k] = t[k][:1].expand(3, 300, 32)
    wide = torch.zeros(3, 600, 96, dtype=BF16, device="cuda")
    wide[:, ::2, 32:64] = t["forget"].cuda()
    at = (t["x"][:1].cuda().expand(3, 300, 32), wide[:, ::2, 32:64], t["gate"][:1].cuda().expand(3, 300, 32))
    grad = torch.full((3, 600, 96), 5.0, dtype=BF16, device="cuda")
    out, final, states = gsr.gated_recurrence_forward(ctx, *at, initial=_dev(t["initial"]))
    grads = gsr.gated_recurrence_backward(ctx, _dev(t["dout"]), *at, states, dl_dfinal=_dev(t["dfinal"]),
                                          dl_dforget=grad[:, ::2, 32:64])
    want = _want(t)
    for name, got in zip(("out", "final") + NAMES, (out, final) + grads):
        ref.check(got, want[name], name)
    assert (grad[:, 1::2] == 5).all() and (grad[:, :, :32] == 5).all() and (grad[:, :, 64:] == 5).all()


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_major_arrays(gsr, ctx, dtype, reverse):  # noqa: F811
    """Views of [tokens, batch, channels]: the items' stride is less than the tokens'."""
    t = _inputs(3, 400, 72, dtype, 47)
    _compare(gsr, ctx, t, lengths=[400, 0, 277], reverse=reverse,
             place=lambda v: None if v is None else v.transpose(0, 1).contiguous().cuda().transpose(0, 1))


def test_windows_that_overlap(gsr, ctx):  # noqa: F811
    """Inputs whose tokens share channels, and whose items share tokens, with the next."""
    t = _inputs(3, 300, 64, BF16, 48)
    g = torch.Generator().manual_seed(49)
    at = {}
    for name in ("x", "forget", "gate"):
        base = (2 * torch.randn(300 * 32 + 2 * 800 + 64, generator=g)).bfloat16()
        t[name], at[name] = (v.as_strided((3, 300, 64), (800, 32, 1)) for v in (base, base.cuda()))
    out, final, states = gsr.gated_recurrence_forward(ctx, at["x"], at["forget"], at["gate"], initial=_dev(t["initial"]))
    grads = gsr.gated_recurrence_backward(ctx, _dev(t["dout"]), at["x"], at["forget"], at["gate"], states,
                                          dl_dfinal=_dev(t["dfinal"]))
    want = _want(t)
    for name, got in zip(("out", "final") + NAMES, (out, final) + grads):
        ref.check(got, want[name], name)


def test_extremes_over_groups(gsr, ctx):  # noqa: F811
    """Tiles and groups whose gates are shut or open throughout: maps of no state, and of nothing
    but the state."""
    for dtype in (F32, BF16):
        t = _inputs(1, 3000, 8, dtype, 44)
        t["forget"][0, 300:700] = -60.0
        t["forget"][0, 1100:1101] = -float("inf")
        t["forget"][0, 1500:2900, :4] = float("inf")
        for reverse in (False, True):
            _compare(gsr, ctx, t, reverse=reverse)


def test_not_finite_over_groups(gsr, ctx):  # noqa: F811
    """An infinite state, then gates that are shut; a gate that is not a number: nothing waits for
    ever, nothing else changes, and runs agree."""
    t = {k: _dev(v) for k, v in _inputs(1, 5000, 64, F32, 45).items()}
    args = (t["x"], t["forget"], t["gate"])
    clean, _, _ = gsr.gated_recurrence_forward(ctx, *args)
    t["x"][0, 50, 3] = float("inf")
    t["forget"][0, 2000:2600, 3] = -200.0
    t["forget"][0, 10, 9] = float("nan")
    runs = []
    for _ in range(4):
        out, final, states = gsr.gated_recurrence_forward(ctx, *args)
        runs.append((out, final, states) + gsr.gated_recurrence_backward(ctx, t["dout"], *args, states))
    ctx.synchronize()
    others = [c for c in range(64) if c not in (3, 9)]
    assert torch.equal(out[..., others], clean[..., others]) and torch.isnan(out[0, 10:, 9]).all()
    for run in runs[1:]:
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(run, runs[0]))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,c", [(9, 64), (9, 33), (300, 64), (300, 66), (300, 33), (3000, 64)])
def test_not_finite_stays_in_its_channel(gsr, ctx, dtype, n, c):  # noqa: F811
    """Beside its neighbour in a pair too: in the values, both gates, the gradients and the states."""
    t = {k: _dev(v) for k, v in _inputs(2, n, c, dtype, 47).items()}
    clean = _run(gsr, ctx, t)
    places = {"x": (0, n // 2, 5), "forget": (1, n // 3, 6), "gate": (0, n // 2, 9), "dout": (1, n - 1, 12)}
    for value in (float("nan"), float("inf"), -float("inf")):
        for key, place in places.items():
            bad = {k: v.clone() for k, v in t.items()}
            bad[key][place] = value
            got = _run(gsr, ctx, bad)
            others = torch.ones(c, dtype=torch.bool, device="cuda")
            others[place[2]] = False
            for name, want in clean.items():
                assert torch.equal(got[name][..., others], want[..., others]), (key, name)
                assert torch.equal(got[name][1 - place[0]], want[1 - place[0]]), (key, name)
            if key in ("x", "forget") and value != value:
                assert torch.isnan(got["out"][place[0], place[1]:, place[2]]).all()
                assert torch.isnan(got["final"][place[0], place[2]])
            if key == "forget" and value != value:   # what the state meets reaches every gradient before it
                assert torch.isnan(got["dx"][place[0], :place[1] + 1, place[2]]).all()
                assert torch.isnan(got["dinitial"][place[0], place[2]])


def test_random_shapes(gsr, ctx):  # noqa: F811
    g = torch.Generator().manual_seed(46)
    pick = lambda *values: values[int(torch.randint(len(values), (1,), generator=g))]  # noqa: E731
    for seed in range(60):
        b, n = pick(1, 2, 5), int(torch.randint(1, 1400, (1,), generator=g))
        c = pick(1, 3, 8, 16, 33, 40, 64, 66, 80, 130)
        t = _inputs(b, n, c, pick(F32, BF16, F16), seed, gate=pick(True, False), state=pick(True, False), keep=pick(-1.0, 2.0, 5.0))
        lengths = pick(None, [int(torch.randint(0, n + 1, (1,), generator=g)) for _ in range(b)])
        _compare(gsr, ctx, t, lengths=lengths, reverse=pick(True, False))
    ctx.synchronize()
