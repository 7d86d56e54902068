"""The 64-bit forms of the token layers' operators, against central differences of
their own forward passes."""
import pytest
import torch

import token_layer_reference as ref

F32 = torch.float32


def _slope(loss, x, d, h=1e-5):
    return (loss(x + h * d) - loss(x - h * d)) / (2 * h)


def test_layer_norm_gradient():
    torch.manual_seed(1)
    x, dout, dtotal = (torch.randn(3, 5, 12, dtype=torch.float64) for _ in range(3))
    w, b = torch.randn(12, dtype=torch.float64), torch.randn(12, dtype=torch.float64)
    g = ref.layer_norm(x, w, b, 1e-5, F32, None, dout, dtotal)

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-5, F32)["out"][0] * dout).sum() + (x * dtotal).sum()

    for i, name in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        d = torch.randn_like(args[i])
        assert abs(_slope(lambda t: loss(*args[:i], t, *args[i + 1:]), args[i], d) - (g[name][0] * d).sum()) < 1e-7


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_recurrence_gradient(reverse, gated):
    torch.manual_seed(2)
    x, f, o, dout = (torch.randn(3, 9, 4, dtype=torch.float64) for _ in range(4))
    first, last = torch.randn(3, 4, dtype=torch.float64), torch.randn(3, 4, dtype=torch.float64)
    lengths = [9, 0, 5]
    args = [x, f, o, first]

    def run(x, f, o, first, **grads):
        return ref.recurrence(x, f, o if gated else None, first, lengths, reverse, F32, **grads)

    def loss(*args):
        r = run(*args)
        return (r["out"][0] * dout).sum() + (r["final"][0] * last).sum()

    g = run(*args, dout=dout, dfinal=last)
    for i, name in enumerate(("dx", "dforget", "dgate", "dinitial")):
        if name in g:
            d = torch.randn_like(args[i])
            slope = _slope(lambda t: loss(*args[:i], t, *args[i + 1:]), args[i], d)
            assert abs(slope - (g[name][0] * d).sum()) < 1e-7, name


def test_recurrence_directions_and_lengths():
    """The reverse direction is the forward one of the item's tokens turned round."""
    torch.manual_seed(3)
    x, f, o = (torch.randn(2, 7, 3, dtype=torch.float64) for _ in range(3))
    lengths = [4, 7]
    back = ref.recurrence(x, f, o, None, lengths, True, F32)
    for i, n in enumerate(lengths):
        turned = [t[i:i + 1, :n].flip(1) for t in (x, f, o)]
        want = ref.recurrence(*turned, None, [n], False, F32)
        # (equal but for the last bits of a vectorised sigmoid)
        assert (back["out"][0][i, :n] - want["out"][0][0].flip(0)).abs().max() < 1e-14
        assert (back["final"][0][i] - want["final"][0][0]).abs().max() < 1e-14
        assert (back["out"][0][i, n:] == 0).all()
