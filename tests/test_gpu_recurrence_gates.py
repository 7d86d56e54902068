"""The gated recurrence's forward where a gate shuts something out: states and values orders of
magnitude apart, within bounds that are relative to each gate."""
import pytest
import torch

from test_gpu_gated_recurrence import BF16, F16, F32, _dev, ctx, gsr  # noqa: F401
import recurrence_gate_reference as ref

pytestmark = pytest.mark.gpu


# h, x, f of a step: a large state that is shut out of a small value, a large value that is shut
# out of a small state, a state of 0 before an open gate.
STEPS = [(1e6, 0.01, -18.4), (1e3, 1e-3, -13.0), (-2e2, 0.0, -8.0), (5.0, 0.0, -16.0), (3.0, 0.0, -20.0),
         (0.01, 1e6, 20.0), (0.5, 1e4, 15.0), (0.0, 1.3, 10.0), (0.0, 1.3, 12.0), (0.0, 1.3, 16.0), (0.0, -1.3, 18.0)]


def _inputs(b, n, c, dtype, seed, gate=True):
    """Values over six orders of magnitude, gates between 8 and 20 either way."""
    g = torch.Generator().manual_seed(seed)

    def wide(*shape):
        return torch.randn(shape, generator=g).sign() * 10.0 ** (6 * torch.rand(shape, generator=g) - 3)

    f = torch.randn(b, n, c, generator=g).sign() * (8 + 12 * torch.rand(b, n, c, generator=g))
    o = torch.randn(b, n, c, generator=g).to(dtype)
    return dict(x=wide(b, n, c).to(dtype), forget=f.to(dtype), gate=o if gate else None, initial=wide(b, c),
                dout=torch.randn(b, n, c, generator=g).to(dtype), dfinal=torch.randn(b, c, generator=g))


def _single_steps(n, last):
    """STEPS as the first or last of n tokens; the others keep what there is."""
    c = len(STEPS)
    t = dict(x=torch.zeros(1, n, c), forget=torch.full((1, n, c), 30.0), gate=torch.ones(1, n, c), dout=torch.ones(1, n, c),
             initial=torch.zeros(1, c), dfinal=torch.ones(1, c))
    for i, (h, x, f) in enumerate(STEPS):
        t["initial"][0, i] = h
        t["x"][0, n - 1 if last else 0, i], t["forget"][0, n - 1 if last else 0, i] = x, f
    return t


def _compare(gsr, ctx, t, lengths=None, reverse=False):  # noqa: F811
    b, n, _ = t["x"].shape
    lens = torch.tensor(lengths or [n] * b, dtype=torch.int32, device="cuda")
    out, final, _ = gsr.gated_recurrence_forward(ctx, *(_dev(t[k]) for k in ("x", "forget", "gate")), initial=_dev(t["initial"]),
                                                 lengths=lens, reverse=reverse)
    wide = {k: None if v is None else v.double() for k, v in t.items()}
    want = ref.recurrence(wide["x"], wide["forget"], wide["gate"], wide["initial"], lengths or [n] * b, reverse, t["x"].dtype)
    ref.check(out, want["out"], "out")
    ref.check(final, want["final"], "final")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n", [1, 2, 16, 17, 64, 70, 129, 300, 1200])
def test_open_and_shut_gates(gsr, ctx, dtype, reverse, n):  # noqa: F811
    for c, gate in ((40, True), (66, True), (33, True), (64, False)):
        lengths = [n, max(n - 7, 0)]
        _compare(gsr, ctx, _inputs(2, n, c, dtype, 100 * n + c, gate), lengths, reverse)


@pytest.mark.parametrize("n", [1, 16, 17, 65, 140])
@pytest.mark.parametrize("last", [False, True])
def test_single_steps(gsr, ctx, n, last):  # noqa: F811
    _compare(gsr, ctx, _single_steps(n, last))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_a_token_more_changes_no_bit_of_those_before(gsr, ctx, dtype):  # noqa: F811
    """16 tokens, which a thread runs alone, and the first 16 of 17, which go in tiles."""
    for c in (40, 33):
        t = {k: _dev(v) for k, v in _inputs(2, 17, c, dtype, 7).items()}
        runs = [gsr.gated_recurrence_forward(ctx, *(t[k][:, :n] for k in ("x", "forget", "gate")), initial=t["initial"])[0]
                for n in (16, 17)]
        assert torch.equal(runs[0], runs[1][:, :16])
