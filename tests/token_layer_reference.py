"""Plain 64-bit forms of the token layers' operators on the CPU, and the bounds that
a float kernel's results have to stay within: the first order of the kernel's own
roundings, propagated through the formulas in 64 bits.

Layer norm.  A sum over channels passes fewer than DEPTH additions (at most 64 in a
thread, then a tree over threads and warps); sums over rows at most ROWS in one
chain.

Recurrence.  REL is the relative error of the smaller of a and 1 - a: the
exponential's argument -|f| log2 e is off by two roundings (2 |f| F of the value),
the fast exponential and reciprocal by 2 ulp each, a sum and a product by one.  The larger of
the two is 1 minus the smaller.  A step's errors count twice, once in the block's
composition and once in the token's own run, against the sums of magnitudes
m_t = a m_(t-1) + (1 - a) |x_t|, which bound what a composition adds and cancels.
"""
import torch

from decoder_reference import F, check, rounding  # noqa: F401 (check is re-exported)

DEPTH = 96
ROWS = 1024


def layer_norm(x, weight, bias, eps, dtype, residual=None, dout=None, dtotal=None):
    """x [..., c] double.  Returns {name: (value, bound)}."""
    c = x.shape[-1]
    out = {}
    if residual is not None:
        whole = x + residual
        out["total"] = (whole, rounding(whole, dtype) + F * whole.abs())
        # the kernel adds in float and rounds to dtype; the norm is that of the stored sum
        x = (x.float() + residual.float()).to(dtype).double()
    w = torch.ones(c, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(c, dtype=torch.float64) if bias is None else bias.double()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    var = (d * d).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    hat = d * rstd
    e_mean = F * (DEPTH * x.abs().mean(-1, keepdim=True) + 2 * mean.abs())
    e_var = (DEPTH + 6) * F * var + e_mean ** 2
    rel = e_var / (2 * (var + eps)) + 6 * F
    e_hat = rstd * (e_mean + F * d.abs()) + hat.abs() * (rel + F)
    y = hat * w + b
    out["out"] = (y, w.abs() * e_hat + 3 * F * ((hat * w).abs() + b.abs()) + rounding(y, dtype))
    out["mean"] = (mean[..., 0], e_mean[..., 0])
    out["rstd"] = (rstd[..., 0], (rstd * rel)[..., 0])
    if dout is not None:
        g = dout * w
        e_g = F * g.abs()
        m1, m2 = g.mean(-1, keepdim=True), (g * hat).mean(-1, keepdim=True)
        e_m1 = ((DEPTH + 2) * F * g.abs()).mean(-1, keepdim=True)
        e_m2 = (g.abs() * e_hat + (DEPTH + 4) * F * (g * hat).abs()).mean(-1, keepdim=True)
        core = g - m1 - hat * m2
        dx = rstd * core
        e_dx = rstd * (e_g + e_m1 + hat.abs() * e_m2 + e_hat * m2.abs()
                       + 4 * F * (g.abs() + m1.abs() + (hat * m2).abs())) + (rel + 2 * F) * dx.abs()
        if dtotal is not None:
            e_dx = e_dx + F * (dx.abs() + dtotal.abs())
            dx = dx + dtotal
        out["dx"] = (dx, e_dx + rounding(dx, dtype))
        rows = [t.reshape(-1, c) for t in (dout, hat, e_hat)]
        terms = min(rows[0].shape[0], ROWS) + DEPTH
        out["dweight"] = ((rows[0] * rows[1]).sum(0),
                          (rows[0].abs() * rows[2] + terms * F * (rows[0] * rows[1]).abs()).sum(0))
        out["dbias"] = (rows[0].sum(0), (terms * F * rows[0].abs()).sum(0))
    return out


def _order(tokens, length, reverse):
    return range(length - 1, -1, -1) if reverse else range(length)


def recurrence(x, forget, gate, initial, lengths, reverse, dtype, dout=None, dfinal=None):
    """x, forget, gate [b, n, c] double, initial, dfinal [b, c] or None, lengths a list.
    Returns {name: (value, bound)}; what lies behind an item's length is 0."""
    b, n, c = x.shape
    a, s = torch.sigmoid(forget), torch.sigmoid(-forget)
    small = torch.minimum(a, s)
    rel = (2 * forget.abs() + 12) * F
    rel = torch.where(small > 0, rel, 0.0)          # an infinite logit leaves nothing of the smaller
    step = 2 * (torch.where(small > 0, rel * small, 0.0) + 4 * F)
    h = torch.zeros(b, n, c, dtype=torch.float64)
    e_h, before, e_before = h.clone(), h.clone(), h.clone()
    final = torch.zeros(b, c, dtype=torch.float64) if initial is None else initial.double().clone()
    e_final = torch.zeros_like(final)
    for i in range(b):
        v, e = final[i], e_final[i]
        m = v.abs()
        for t in _order(n, lengths[i], reverse):
            before[i, t], e_before[i, t] = v, e
            e = a[i, t] * e + step[i, t] * (m + x[i, t].abs())
            v = a[i, t] * v + s[i, t] * x[i, t]
            m = a[i, t] * m + s[i, t] * x[i, t].abs()
            h[i, t], e_h[i, t] = v, e
        final[i], e_final[i] = v, e
    live = torch.zeros(b, n, 1, dtype=torch.bool)
    for i in range(b):
        live[i, :lengths[i]] = True
    if gate is None:
        opened = slope = torch.ones_like(h)
        e_opened = e_slope = torch.zeros_like(h)
    else:
        sig = torch.sigmoid(gate)
        opened, slope = gate * sig, sig * (1 + gate * (1 - sig))
        rel_gate = (2 * gate.abs() + 14) * F
        e_opened = rel_gate * opened.abs()
        e_slope = sig * rel_gate * (1 + 2 * gate.abs())
    y = h * opened

    def cut(value, bound):
        return torch.where(live, value, 0.0), torch.where(live, bound, 0.0)

    out = {"out": cut(y, e_h * opened.abs() + h.abs() * e_opened + 2 * F * y.abs() + rounding(y, dtype)),
           "final": (final, e_final)}
    if dout is None:
        return out
    into, e_into = dout * opened, dout.abs() * e_opened + 2 * F * (dout * opened).abs()
    g, e_g = torch.zeros_like(h), torch.zeros_like(h)
    first = torch.zeros(b, c, dtype=torch.float64) if dfinal is None else dfinal.double().clone()
    e_first = torch.zeros_like(first)
    for i in range(b):
        p, e = first[i], e_first[i]
        m = p.abs()
        for t in reversed(_order(n, lengths[i], reverse)):
            v, ev, mv = p + into[i, t], e + e_into[i, t] + F * (m + into[i, t].abs()), m + into[i, t].abs()
            g[i, t], e_g[i, t] = v, ev
            e = a[i, t] * ev + step[i, t] * mv
            p, m = a[i, t] * v, a[i, t] * mv
        first[i], e_first[i] = p, e
    dx = g * s
    d = before - x
    df = g * d * a * s
    out["dx"] = cut(dx, e_g * s + dx.abs() * (rel + 4 * F) + rounding(dx, dtype))
    out["dforget"] = cut(df, (e_g * d.abs() + g.abs() * (e_before + 2 * F * d.abs())) * a * s
                         + df.abs() * (2 * rel + 6 * F) + rounding(df, dtype))
    if gate is not None:
        do = dout * h * slope
        out["dgate"] = cut(do, dout.abs() * (e_h * slope.abs() + h.abs() * e_slope) + 4 * F * do.abs()
                           + rounding(do, dtype))
    out["dinitial"] = (first, e_first)
    return out
