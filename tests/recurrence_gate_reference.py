"""The gated recurrence in 64 bits on the CPU, with bounds that are relative to each gate.

SMALL is the relative error of the smaller of a and 1 - a: the exponential's argument is off by
two roundings (2 |f| F of the value), the fast exponential and reciprocal by 2 ulp each, a sum
and a product by one.  The larger is 1 minus the smaller, rounded: it carries the smaller's
error in proportion, and one F.  A step h = a h + (1 - a) x then adds

    (rel_a + 2 F) a m + (rel_s + 2 F) (1 - a) |x| + 8 F m'

to a times the error so far, where m = a m + (1 - a) |x| are the sums of magnitudes (m' behind the
step): each gate's error counts against what that gate lets through and nothing else.  2 F are
a gate's product and its part of the map's; 8 F cover the step's own sum and, where a
run starts, what composing the maps before it rounds (the run's and the tile's folds and the
sums that put a state into them, two roundings each).  The gradient's chain is the same with
p = a (p + dout silu(o)).
"""
import torch

from decoder_reference import F, TINY, check, rounding  # noqa: F401 (check is re-exported)

F32 = torch.float32


def gates(forget):
    """a, 1 - a and their relative errors."""
    a, s = torch.sigmoid(forget), torch.sigmoid(-forget)
    small = (2 * forget.abs() + 12) * F
    ratio = torch.exp(-forget.abs())                       # smaller / larger
    large = small * ratio + F
    return a, s, torch.where(forget < 0, small, large), torch.where(forget < 0, large, small)


def recurrence(x, forget, gate, initial, lengths, reverse, dtype, dout=None, dfinal=None):
    """x, forget, gate [b, n, c] double, initial, dfinal [b, c] or None, lengths a list.
    Returns {name: (value, bound)}; what lies behind an item's length is 0."""
    b, n, c = x.shape
    a, s, rel_a, rel_s = gates(forget)
    live = (torch.arange(n) < torch.tensor(lengths)[:, None])[:, :, None]
    tokens = range(n - 1, -1, -1) if reverse else range(n)
    keep = lambda t, new, old: torch.where(live[:, t], new, old)  # noqa: E731
    h, e_h, before, e_before = (torch.zeros(b, n, c, dtype=torch.float64) for _ in range(4))
    v = torch.zeros(b, c, dtype=torch.float64) if initial is None else initial.double()
    m, e = v.abs(), torch.zeros_like(v)
    for t in tokens:
        before[:, t], e_before[:, t] = v, e
        kept, entered = a[:, t] * m, s[:, t] * x[:, t].abs()
        e = keep(t, a[:, t] * e + (rel_a[:, t] + 2 * F) * kept + (rel_s[:, t] + 2 * F) * entered + 8 * F * (kept + entered), e)
        v = keep(t, a[:, t] * v + s[:, t] * x[:, t], v)
        m = keep(t, kept + entered, m)
        h[:, t], e_h[:, t] = v, e
    out = {"final": (v, e + TINY[F32])}
    opened = slope = torch.ones_like(h)
    e_opened = e_slope = torch.zeros_like(h)
    if gate is not None:
        sig = torch.sigmoid(gate)
        opened, slope = gate * sig, sig * (1 + gate * (1 - sig))
        rel_gate = (2 * gate.abs() + 14) * F
        e_opened = rel_gate * opened.abs()
        e_slope = sig * rel_gate * (1 + 2 * gate.abs())

    def cut(value, bound):
        return torch.where(live, value, 0.0), torch.where(live, bound + rounding(value, dtype), 0.0)

    y = h * opened
    out["out"] = cut(y, e_h * opened.abs() + h.abs() * e_opened + 2 * F * y.abs())
    if dout is None:
        return out
    into, e_into = dout * opened, dout.abs() * e_opened + 2 * F * (dout * opened).abs()
    g, e_g = torch.zeros_like(h), torch.zeros_like(h)
    p = torch.zeros(b, c, dtype=torch.float64) if dfinal is None else dfinal.double()
    m, e = p.abs(), torch.zeros_like(p)
    for t in reversed(tokens):
        mv = m + into[:, t].abs()
        ev = e + e_into[:, t] + F * mv
        g[:, t], e_g[:, t] = p + into[:, t], ev
        e = keep(t, a[:, t] * ev + (rel_a[:, t] + 10 * F) * a[:, t] * mv, e)
        p, m = keep(t, a[:, t] * (p + into[:, t]), p), keep(t, a[:, t] * mv, m)
    d = before - x
    dx, df = g * s, g * d * a * s
    out["dx"] = cut(dx, e_g * s + dx.abs() * (rel_s + 2 * F))
    out["dforget"] = cut(df, (e_g * d.abs() + g.abs() * (e_before + 2 * F * d.abs())) * a * s
                         + df.abs() * (rel_a + rel_s + 4 * F))
    if gate is not None:
        do = dout * h * slope
        out["dgate"] = cut(do, dout.abs() * (e_h * slope.abs() + h.abs() * e_slope) + 4 * F * do.abs())
    out["dinitial"] = (p, e + TINY[F32])
    return out
