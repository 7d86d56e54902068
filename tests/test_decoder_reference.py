"""The 64-bit forms the decoder's GPU tests compare with, against central
differences of their own forward passes."""
import pytest
import torch

import decoder_reference as ref


def _differences(loss, x, direction, h=1e-5):
    return (loss(x + h * direction) - loss(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_group_norm_gradient(act):
    torch.manual_seed(3)
    x, dout = torch.randn(2, 9, 12, dtype=torch.float64), torch.randn(2, 9, 12, dtype=torch.float64)
    w, b = torch.randn(12, dtype=torch.float64), torch.randn(12, dtype=torch.float64)
    g = ref.group_norm(x, 3, w, b, 1e-5, act, dout)
    for name, value, loss in (
            ("dx", x, lambda t: (ref.group_norm(t, 3, w, b, 1e-5, act)["out"][0] * dout).sum()),
            ("dweight", w, lambda t: (ref.group_norm(x, 3, t, b, 1e-5, act)["out"][0] * dout).sum()),
            ("dbias", b, lambda t: (ref.group_norm(x, 3, w, t, 1e-5, act)["out"][0] * dout).sum())):
        d = torch.randn_like(value)
        assert abs(_differences(loss, value, d) - (g[name][0] * d).sum()) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient(interleaved):
    torch.manual_seed(4)
    x, dout = (torch.randn(2, 5, 3, 20, dtype=torch.float64) for _ in range(2))
    pos, freq, sections = torch.rand(2, 5, 3) * 9, torch.rand(8), [3, 1, 4]
    d = torch.randn_like(x)

    def loss(t):
        return (ref.rotary(t, pos, freq, sections, interleaved, torch.float32)[0] * dout).sum()

    g = ref.rotary(dout, pos, freq, sections, interleaved, torch.float32, backward=True)[0]
    assert abs(_differences(loss, x, d) - (g * d).sum()) < 1e-8


def test_attention_gradient():
    torch.manual_seed(5)
    q, dout = (torch.randn(2, 7, 4, 8, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(2, 11, 2, 8, dtype=torch.float64) for _ in range(2))
    valid = torch.rand(2, 11) < 0.6
    g = ref.attention(q, k, v, valid, 0.3, torch.bfloat16, dout)
    for i, name in enumerate(("dq", "dk", "dv")):
        def loss(t):
            args = [q, k, v]
            args[i] = t
            return (ref.attention(*args, valid, 0.3, torch.bfloat16)["out"][0] * dout).sum()

        value = (q, k, v)[i]
        d = torch.randn_like(value)
        assert abs(_differences(loss, value, d) - (g[name][0] * d).sum()) < 1e-7


def test_attention_without_keys():
    q, k = torch.randn(1, 3, 2, 8, dtype=torch.float64), torch.randn(1, 5, 1, 8, dtype=torch.float64)
    g = ref.attention(q, k, k, torch.zeros(1, 5, dtype=torch.bool), 0.3, torch.float16, q)
    assert (g["out"][0] == 0).all() and (g["lse"][0] == -float("inf")).all()
    assert all((g[n][0] == 0).all() for n in ("dq", "dk", "dv"))
