"""The recurrence's bounds that are relative to each gate: their values are the other 64-bit
form's, a step in float of the right form stays within them, and the two forms that lose a
gate's bits do not."""
import pytest
import torch

import recurrence_gate_reference as ref
import token_layer_reference as layers

F32 = torch.float32


def _inputs(n, c, seed):
    """States, values and gradients over six orders of magnitude, gates mostly open or shut."""
    g = torch.Generator().manual_seed(seed)
    wide = lambda *shape: torch.randn(shape, generator=g).sign() * 10.0 ** (6 * torch.rand(shape, generator=g) - 3)  # noqa: E731
    f = torch.randn(1, n, c, generator=g).sign() * (8 + 12 * torch.rand(1, n, c, generator=g))
    return wide(1, n, c), f, torch.randn(1, n, c, generator=g), wide(1, c), wide(1, n, c), wide(1, c)


@pytest.mark.parametrize("reverse", [False, True])
def test_values(reverse):
    x, f, o, first, dout, last = (t.double() for t in _inputs(40, 6, 1))
    for lengths in ([40], [17], [0]):
        got = ref.recurrence(x, f, o, first, lengths, reverse, F32, dout, last)
        want = layers.recurrence(x, f, o, first, lengths, reverse, F32, dout, last)
        for name, (value, _) in want.items():
            assert torch.allclose(got[name][0], value, rtol=1e-13, atol=0), name


def _run(x, f, first, form):
    """A float run whose steps take one of the forms."""
    small = torch.exp(-f.double().abs()).float()
    small = small / (1 + small)
    large = 1 - small
    a, s = torch.where(f < 0, small, large), torch.where(f < 0, large, small)
    h, states = first, []
    for t in range(x.shape[1]):
        if form == "both gates":
            h = a[:, t] * h + s[:, t] * x[:, t]
        elif form == "a from 1 - a":
            h = (1 - s[:, t]) * h + s[:, t] * x[:, t]
        else:
            h = x[:, t] + a[:, t] * (h - x[:, t])
        states.append(h)
    return torch.stack(states, 1)


@pytest.mark.parametrize("form,right", [("both gates", True), ("a from 1 - a", False), ("from the difference", False)])
def test_forms_of_a_step(form, right):
    x, f, _, first, _, _ = _inputs(200, 64, 2)
    value, bound = ref.recurrence(x.double(), f.double(), None, first, [200], False, F32)["out"]
    assert bool(((_run(x, f, first, form).double() - value).abs() <= bound).all()) == right
