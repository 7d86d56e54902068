"""Plain 64-bit forms of the decoder's operators on the CPU, and the bounds that
a float kernel's results have to stay within.

U is the unit roundoff of each storage type and F float's.  A bound is the first
order of the kernel's own roundings, propagated through the formulas in 64 bits:
one rounding to the storage type at each place where the kernels round (outputs,
the softmax' probabilities and ds before their products), float roundings
elsewhere, sums of n terms at n F times the sum of magnitudes.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# The smallest magnitudes of f16 are spaced 2^-24 apart (2^-25 is half of that).
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}
F = 2.0 ** -24


def rounding(value, dtype):
    return U[dtype] * value.abs() + TINY[dtype]


# -- group norm ---------------------------------------------------------------

def activation(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def activation_slope(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def group_norm(x, groups, weight, bias, eps, act, dout=None, dtype=torch.float32):
    """x [n, s, c] double.  Returns {name: (value, bound)}."""
    n, s, c = x.shape
    shape = (n, s, groups, c // groups)
    count = s * (c // groups)
    xg = x.view(shape)
    w = weight.view(shape[2:]) if weight is not None else torch.ones(shape[2:], dtype=torch.float64)
    b = bias.view(shape[2:]) if bias is not None else torch.zeros(shape[2:], dtype=torch.float64)
    mean = xg.mean(dim=(1, 3), keepdim=True)
    var = ((xg - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    hat = (xg - mean) * rstd
    z = hat * w + b
    y = activation(z, act)
    # A merge of means rounds a few times per level of its tree; each rounding is
    # relative to the mean or to a difference of means (at most the spread).
    spread = (xg - mean).abs().amax(dim=(1, 3), keepdim=True)
    e_mean = 64 * F * (mean.abs() + spread)
    e_hat = rstd * e_mean + 64 * F * hat.abs() + hat.abs() * rstd ** 2 * e_mean * spread
    e_z = w.abs() * e_hat + 4 * F * (z.abs() + b.abs())
    # The slope of silu and gelu is below 1.13; the fast exponential is off by a
    # few roundings of its scaled argument.
    e_y = 1.13 * e_z + 16 * F * y.abs() * (1 + z.abs()) + rounding(y, dtype)
    out = {"out": (y, e_y), "mean": (mean, e_mean), "rstd": (rstd, rstd ** 3 * e_mean * spread + 64 * F * rstd)}
    if dout is not None:
        g = dout.view(shape)
        slope = activation_slope(z, act)
        dz = g * slope
        # |act''| is below 0.8 for gelu and 0.5 for silu
        e_dz = g.abs() * (0.8 * e_z + 16 * F * (1 + z.abs()))
        e_dz = e_dz if act != "none" else 2 * F * dz.abs()
        terms = min(count, 1024) * F
        db, dw = dz.sum(dim=(0, 1)), (dz * hat).sum(dim=(0, 1))
        e_db = (e_dz + terms * dz.abs()).sum(dim=(0, 1))
        e_dw = (e_dz * hat.abs() + dz.abs() * e_hat + terms * (dz * hat).abs()).sum(dim=(0, 1))
        gw = dz * w
        m1, m2 = gw.mean(dim=(1, 3), keepdim=True), (gw * hat).mean(dim=(1, 3), keepdim=True)
        e_gw = e_dz * w.abs()
        e_m1 = (e_gw + terms * gw.abs()).mean(dim=(1, 3), keepdim=True)
        e_m2 = (e_gw * hat.abs() + gw.abs() * e_hat + terms * (gw * hat).abs()).mean(dim=(1, 3), keepdim=True)
        dx = rstd * (gw - m1 - hat * m2)
        e_rstd = out["rstd"][1]
        e_dx = rstd * (e_gw + e_m1 + hat.abs() * e_m2 + e_hat * m2.abs()
                       + 4 * F * (gw.abs() + m1.abs() + (hat * m2).abs()))
        e_dx = e_dx + e_rstd / rstd * dx.abs() + rounding(dx, dtype)
        out.update(dx=(dx, e_dx), dweight=(dw, e_dw), dbias=(db, e_db))
    flat = {"out": (n, s, c), "dx": (n, s, c), "dweight": (c,), "dbias": (c,), "mean": (n, groups),
            "rstd": (n, groups)}
    return {k: tuple(t.expand(v[0].shape).reshape(flat[k]) for t in v) for k, v in out.items()}


# -- rotary positions -----------------------------------------------------------

def rotary(x, positions, frequencies, sections, interleaved, dtype, backward=False):
    """x [b, t, h, d] double, positions [b, t, axes].  Returns (value, bound)."""
    half = sum(sections)
    value, bound = x.clone(), torch.zeros_like(x)
    i = 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            theta = positions[:, :, axis].double() * frequencies[i].double()
            if backward:
                theta = -theta
            c, s = torch.cos(theta)[:, :, None], torch.sin(theta)[:, :, None]
            one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, v = x[..., one], x[..., two]
            value[..., one], value[..., two] = u * c - v * s, u * s + v * c
            # sine and cosine within 2 ulp, their composition and the rotation a few roundings
            for at in (one, two):
                bound[..., at] = 8 * F * (u.abs() + v.abs()) + rounding(value[..., at], dtype)
            i += 1
    return value, bound


# -- cross attention --------------------------------------------------------------

def attention(q, k, v, valid, scale, dtype, dout=None):
    """q [b, lq, hq, d], k and v [b, lk, hk, d] double, valid [b, lk] bool.  Returns
    {name: (value, bound)} of out, lse and, with dout, dq, dk, dv."""
    b, lq, hq, d = q.shape
    lk, hk = k.shape[1:3]
    group = hq // hk
    u = U[dtype]

    def rows(t):      # [b, hk, group * lq, d]
        return t.view(b, lq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * lq, d)

    def unrows(t):
        return t.view(b, hk, group, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d)

    mask = valid[:, None, None, :]
    kt = torch.where(valid[:, :, None, None], k, 0.0).transpose(1, 2)
    vt = torch.where(valid[:, :, None, None], v, 0.0).transpose(1, 2)
    qt = rows(q)
    s = torch.where(mask, scale * (qt @ kt.transpose(2, 3)), -math.inf)
    # d products summed in float, the scale and the exponential's argument
    e_s = scale * 2 * d * F * (qt.abs() @ kt.abs().transpose(2, 3)) + 8 * F * torch.where(mask, s, 0.0).abs() + 8 * F
    top = s.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(dim=3, keepdim=True)
    lse = top + torch.log(total)
    p = p / torch.where(total == 0, 1.0, total)
    n = 2 * lk * F
    e_lse = (p * e_s).sum(dim=3, keepdim=True) + n + 4 * F * torch.where(total > 0, lse, 0.0).abs()
    e_p = p * (e_s + e_lse + 8 * F)                    # before the rounding to the storage type
    # Probabilities below f16's normal range round to a spacing of 2^-24 of the
    # row's largest, which is at most 2^8 times their scale in the kernel.
    e_pr = e_p + u * p + (2.0 ** -24 if dtype == torch.float16 else 0.0) * mask
    o = p @ vt
    e_o = e_pr @ vt.abs() + n * (p @ vt.abs()) + 8 * F * o.abs() + rounding(o, dtype)
    out = {"out": (unrows(o), unrows(e_o)),
           "lse": (lse.view(b, hq, lq), e_lse.expand(lse.shape).reshape(b, hq, lq))}
    if dout is not None:
        do = rows(dout)
        dv = p.transpose(2, 3) @ do
        m = 2 * group * lq * F
        e_dv = (e_pr + m * p).transpose(2, 3) @ do.abs() + rounding(dv, dtype)
        dp = do @ vt.transpose(2, 3)
        e_dp = 2 * d * F * (do.abs() @ vt.abs().transpose(2, 3))
        delta = (do * o).sum(dim=3, keepdim=True)
        e_delta = ((e_o + 2 * d * F * o.abs()) * do.abs()).sum(dim=3, keepdim=True)
        ds = p * (dp - delta)
        e_ds = e_p * (dp - delta).abs() + p * (e_dp + e_delta + 4 * F * (dp.abs() + delta.abs())) + rounding(ds, dtype)
        dq = scale * (ds @ kt)
        e_dq = scale * ((e_ds + n * ds.abs()) @ kt.abs()) + rounding(dq, dtype) + 4 * F * dq.abs()
        dk = scale * (ds.transpose(2, 3) @ qt)
        e_dk = scale * ((e_ds + m * ds.abs()).transpose(2, 3) @ qt.abs()) + rounding(dk, dtype) + 4 * F * dk.abs()
        out["dq"] = (unrows(dq), unrows(e_dq))
        out["dk"] = (dk.transpose(1, 2), e_dk.transpose(1, 2))
        out["dv"] = (dv.transpose(1, 2), e_dv.transpose(1, 2))
    return out


def check(got, want, name=""):
    """|got - value| <= bound elementwise, infinities equal; returns the largest share of the bound."""
    value, bound = want
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    same = got == value
    error = torch.where(same, 0.0, (got - value).abs())
    bad = ~(error <= bound)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4].tolist(), value[bad][:4].tolist(), bound[bad][:4].tolist())
    return float((error / bound.clamp_min(1e-300)).max()) if error.numel() else 0.0
