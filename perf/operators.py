"""Cases that measure the operators of an image-to-Gaussians decoder: group norm
with an activation, rotary positions with several axes, and cross attention to
the image tokens of all views.

`own` chooses what `run` computes with: the plain form (elementary torch
operations in 32 bits, rounded once at the end) or the package's kernels.  Token
counts are those of 16x16 patches: 2,500 for an 800x800 view, 8,160 for
1920x1080, 256 for 256x256 and 16 for 64x64.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
GRID = 50            # patches along a side of an 800x800 view
RADIUS = 23.7        # silhouette mask: patches within this of the view's centre


def listed():
    return [
        # One refined Gaussian token per scene against four 800x800 views (serving, one token at a time).
        {"name": "attend_token", "op": "attend", "train": False, "dtype": "bf16", "batch": 4, "q_len": 1,
         "kv_len": 10000, "q_heads": 16, "kv_heads": 4, "dim": 128, "drop": 0, "mask": False},
        # The smallest call: 16 tokens of a 64x64 image against one 256x256 view; latency counts.
        {"name": "attend_small", "op": "attend", "train": False, "dtype": "f16", "batch": 1, "q_len": 16,
         "kv_len": 256, "q_heads": 8, "kv_heads": 8, "dim": 64, "drop": 0, "mask": False},
        # Preview of two scenes, the second with one of its four views missing.
        {"name": "attend_views", "op": "attend", "train": False, "dtype": "bf16", "batch": 2, "q_len": 2500,
         "kv_len": 10000, "q_heads": 16, "kv_heads": 16, "dim": 64, "drop": 2500, "mask": False},
        # The largest: a token per 1920x1080 tile against four such views, shared key heads.
        {"name": "attend_large", "op": "attend", "train": False, "dtype": "f16", "batch": 1, "q_len": 8160,
         "kv_len": 32640, "q_heads": 16, "kv_heads": 4, "dim": 128, "drop": 0, "mask": False},
        # A training step's attention over three views with the patches outside the silhouette masked.
        {"name": "train_views", "op": "attend", "train": True, "dtype": "bf16", "batch": 2, "q_len": 2500,
         "kv_len": 7500, "q_heads": 16, "kv_heads": 4, "dim": 128, "drop": 0, "mask": True},
        # Training against a few pooled tokens of each scene: short odd lengths that differ over the batch.
        {"name": "train_short", "op": "attend", "train": True, "dtype": "f16", "batch": 12, "q_len": 1023,
         "kv_len": 77, "q_heads": 8, "kv_heads": 8, "dim": 64, "drop": 6, "mask": False},
        # Positions (view, row, column) onto the keys of four 800x800 views of two scenes.
        {"name": "rotary_views", "op": "rotary", "backward": False, "dtype": "bf16", "batch": 2, "len": 10000,
         "heads": 16, "dim": 128, "sections": "16,24,24", "pairs": "halves", "float_positions": False},
        # The gradient through fractional query positions, in float32, with dimensions that are not rotated.
        {"name": "rotary_queries", "op": "rotary", "backward": True, "dtype": "f32", "batch": 1, "len": 2500,
         "heads": 8, "dim": 72, "sections": "10,11,11", "pairs": "neighbours", "float_positions": True},
        # One small feature map: latency counts.
        {"name": "norm_small", "op": "norm", "train": False, "dtype": "f16", "samples": 1, "positions": 256,
         "channels": 64, "groups": 8, "act": "silu"},
        # Feature maps of four 800x800 views at a quarter of the resolution.
        {"name": "norm_views", "op": "norm", "train": False, "dtype": "bf16", "samples": 4, "positions": 40000,
         "channels": 256, "groups": 32, "act": "silu"},
        # A training step's norm at half the resolution.
        {"name": "norm_train", "op": "norm", "train": True, "dtype": "bf16", "samples": 4, "positions": 160000,
         "channels": 128, "groups": 32, "act": "silu"},
        # Training in float32 on odd crops, three channels to a group.
        {"name": "norm_odd", "op": "norm", "train": True, "dtype": "f32", "samples": 3, "positions": 6767,
         "channels": 96, "groups": 32, "act": "gelu"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rotary", "norm"])
    if op == "attend":
        while True:
            kv_heads = rng.choice([1, 2, 4, 8, 16])
            case = {"op": op, "train": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"]),
                    "batch": _log_int(rng, 1, 16), "q_len": _log_int(rng, 1, 8160),
                    "kv_len": _log_int(rng, 1, 32640), "kv_heads": kv_heads,
                    "q_heads": kv_heads * rng.choice([1, 2, 4]), "dim": rng.choice([32, 64, 72, 80, 96, 128]),
                    "drop": 0, "mask": rng.random() < 0.3}
            if rng.random() < 0.5:   # every item keeps at least one key
                case["drop"] = rng.randint(0, (case["kv_len"] - 1) // max(1, case["batch"] - 1))
            if case["mask"]:
                case["kv_len"] = max(case["kv_len"], 2500)
            cost = case["batch"] * case["q_heads"] * case["q_len"] * case["kv_len"] * case["dim"]
            if cost * (3.5 if case["train"] else 1) <= 16 * 8160 * 32640 * 128 / 2:
                return case
    if op == "rotary":
        dim = rng.choice([32, 64, 72, 96, 128])
        axes = rng.choice([1, 2, 3, 4])
        half = dim // 2 - rng.choice([0, 4])
        sections = [half // axes] * axes
        sections[-1] += half - sum(sections)
        return {"op": op, "backward": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "batch": rng.randint(1, 3), "len": _log_int(rng, 1, 10000), "heads": _log_int(rng, 1, 16),
                "dim": dim, "sections": ",".join(map(str, sections)),
                "pairs": rng.choice(["halves", "neighbours"]), "float_positions": rng.random() < 0.5}
    groups = rng.choice([1, 4, 8, 32])
    channels = groups * rng.choice([1, 2, 3, 4, 8])
    samples = rng.randint(1, 6)
    return {"op": op, "train": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16", "f32"]),
            "samples": samples, "positions": _log_int(rng, 16, 81920000 // (samples * channels)),
            "channels": channels, "groups": groups, "act": rng.choice(["none", "silu", "gelu"])}


# -- inputs -----------------------------------------------------------------

def _lengths(case):
    return [case["kv_len"] - case["drop"] * (case["batch"] - 1 - i) for i in range(case["batch"])]


def _silhouette(kv_len):
    """Whether each of kv_len patch tokens, in rows of views of GRID x GRID, lies on the object."""
    i = torch.arange(kv_len)
    row, col = (i // GRID) % GRID, i % GRID
    c = (GRID - 1) / 2
    return (row - c) ** 2 + (col - c) ** 2 < RADIUS ** 2


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _frequencies(sections):
    return torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for s in sections]).float()


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=case["dtype"]):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(DTYPES[dtype])

    if case["op"] == "attend":
        b, lq, lk, hq, hk, d = (case[k] for k in ("batch", "q_len", "kv_len", "q_heads", "kv_heads", "dim"))
        x = {"q": normal(b, lq, hq, d), "k": normal(b, lk, hk, d), "v": normal(b, lk, hk, d),
             "lengths": None, "mask": None}
        if case["train"]:
            x["dout"] = normal(b, lq, hq, d)
        if case["drop"]:
            x["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
        if case["mask"]:
            x["mask"] = _silhouette(lk).to(DEV).expand(b, lk).contiguous()
        return x
    if case["op"] == "rotary":
        b, n, h, d = (case[k] for k in ("batch", "len", "heads", "dim"))
        axes = len(_sections(case))
        grid = torch.arange(n)
        columns = [grid // (GRID * GRID), (grid // GRID) % GRID, grid % GRID, grid % 7]
        positions = torch.stack([columns[(a + 3 - axes) % 4] for a in range(axes)], dim=1)
        positions = positions.expand(b, n, axes).to(DEV)
        if case["float_positions"]:
            positions = positions + torch.rand((b, n, axes), generator=gen, device=DEV)
        else:
            positions = positions.to(torch.int32)
        return {"x": normal(b, n, h, d), "positions": positions.contiguous(),
                "frequencies": _frequencies(_sections(case)).to(DEV)}
    n, s, c = (case[k] for k in ("samples", "positions", "channels"))
    offset = normal(c, dtype="f32")
    scale = normal(c, dtype="f32").abs() + 0.5
    x = (torch.randn((n, s, c), generator=gen, device=DEV) * scale + offset).to(DTYPES[case["dtype"]])
    out = {"x": x, "weight": 1 + 0.2 * normal(c, dtype="f32"), "bias": 0.2 * normal(c, dtype="f32")}
    if case["train"]:
        out["dout"] = normal(n, s, c)
    return out


def prepare(case, seed):
    state = dict(case, **_inputs(case, seed))
    if own:
        import gaussian_splatting_tile_bin_gb300 as gsr
        state["gsr"] = gsr
        state["ctx"] = gsr.Context(0)
    if case["op"] == "rotary":
        state["sections"] = _sections(case)
    return state


# -- one pass ---------------------------------------------------------------

def run(state):
    return {"attend": _attend, "rotary": _rotary, "norm": _norm}[state["op"]](state)


def _attend(st):
    if own:
        gsr, ctx = st["gsr"], st["ctx"]
        keys = {"kv_lengths": st["lengths"], "key_mask": st["mask"]}
        out, lse = gsr.cross_attention_forward(ctx, st["q"], st["k"], st["v"], **keys)
        if not st["train"]:
            return out, lse
        return (out,) + tuple(gsr.cross_attention_backward(ctx, st["q"], st["k"], st["v"], out, lse, st["dout"],
                                                           **keys))
    q, k, v = st["q"], st["k"], st["v"]
    b, lq, hq, d = q.shape
    lk, hk = k.shape[1], k.shape[2]
    group, scale = hq // hk, 1.0 / math.sqrt(d)
    valid = torch.ones((b, lk), dtype=torch.bool, device=q.device)
    if st["lengths"] is not None:
        valid &= torch.arange(lk, device=q.device) < st["lengths"][:, None]
    if st["mask"] is not None:
        valid &= st["mask"]
    # One matrix per item and key head: the group's query heads as group * lq rows.
    count, rows = b * hk, group * lq

    def by_query(t):
        return t.view(b, lq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(count, rows, d)

    def by_key(t):
        return t.transpose(1, 2).reshape(count, lk, d)

    valid = valid.repeat_interleave(hk, dim=0)[:, None]
    qs, ks, vs = by_query(q), by_key(k), by_key(v)
    dos = by_query(st["dout"]) if st["train"] else None
    results = [torch.empty_like(t) for t in (qs, qs, ks, vs)]   # out, dq, dk, dv
    lse = torch.empty((count, rows), dtype=torch.float32, device=q.device)
    step = max(1, (1 << 29) // (rows * lk))
    for i in range(0, count, step):
        at = slice(i, i + step)
        live = valid[at].transpose(1, 2)
        qm, km, vm = qs[at].float(), torch.where(live, ks[at].float(), 0.0), torch.where(live, vs[at].float(), 0.0)
        s = torch.where(valid[at], (qm @ km.transpose(1, 2)) * scale, float("-inf"))
        top = s.amax(dim=2, keepdim=True)
        top = torch.where(top == float("-inf"), 0.0, top)
        p = torch.exp(s - top)
        del s
        total = p.sum(dim=2, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        o = p @ vm
        results[0][at] = o.to(q.dtype)
        lse[at] = (top + torch.log(total))[:, :, 0]
        if st["train"]:
            do = dos[at].float()
            results[3][at] = (p.transpose(1, 2) @ do).to(q.dtype)
            ds = p * (do @ vm.transpose(1, 2) - (do * o).sum(dim=2, keepdim=True)) * scale
            results[1][at] = (ds @ km).to(q.dtype)
            results[2][at] = (ds.transpose(1, 2) @ qm).to(q.dtype)
    out, dq = (t.view(b, hk, group, lq, d).permute(0, 3, 1, 2, 4).reshape(q.shape) for t in results[:2])
    if not st["train"]:
        return out, lse.view(b, hq, lq)
    dk, dv = (t.view(b, hk, lk, d).transpose(1, 2).contiguous() for t in results[2:])
    return out, dq, dk, dv


def _rotary(st):
    interleaved = st["pairs"] == "neighbours"
    if own:
        gsr = st["gsr"]
        call = gsr.rotary_backward if st["backward"] else gsr.rotary_forward
        return call(st["ctx"], st["x"], st["positions"], st["frequencies"], st["sections"],
                    interleaved=interleaved)
    x = st["x"].float()
    axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device=x.device),
                                   torch.tensor(st["sections"], device=x.device))
    angle = st["positions"].float()[:, :, axis] * st["frequencies"]
    cos, sin = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    if st["backward"]:
        sin = -sin
    half = st["frequencies"].numel()
    if interleaved:
        u, w = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], dim=-1).flatten(-2)
    else:
        u, w = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1).to(st["x"].dtype)


EPS = 1e-5


def _norm(st):
    if own:
        gsr, ctx = st["gsr"], st["ctx"]
        out, mean, rstd = gsr.group_norm_forward(ctx, st["x"], st["groups"], st["weight"], st["bias"], eps=EPS,
                                                 activation=st["act"])
        if not st["train"]:
            return out
        return (out,) + tuple(gsr.group_norm_backward(ctx, st["dout"], st["x"], st["groups"], st["weight"],
                                                      st["bias"], mean, rstd, activation=st["act"]))
    n, s, c = st["x"].shape
    shape = (n, s, st["groups"], c // st["groups"])
    w, bias = st["weight"].view(shape[2:]), st["bias"].view(shape[2:])
    x = st["x"].float().view(shape)
    x = x - x.mean(dim=(1, 3), keepdim=True)
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=(1, 3), keepdim=True) + EPS)
    x = x * rstd
    z = x * w + bias
    if st["act"] == "silu":
        gate = 1.0 / (1.0 + torch.exp(-z))
    elif st["act"] == "gelu":
        gate = 0.5 * (1.0 + torch.erf(z / math.sqrt(2.0)))
    else:
        gate = torch.ones_like(z)
    out = (z * gate).view(n, s, c).to(st["x"].dtype)
    if not st["train"]:
        return out
    if st["act"] == "silu":
        slope = gate * (1.0 + z * (1.0 - gate))
    elif st["act"] == "gelu":
        slope = gate + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    else:
        slope = gate
    dz = st["dout"].float().view(shape) * slope
    db, dw = dz.sum(dim=(0, 1)).view(c), (dz * x).sum(dim=(0, 1)).view(c)
    g = dz * w
    dx = rstd * (g - g.mean(dim=(1, 3), keepdim=True) - x * (g * x).mean(dim=(1, 3), keepdim=True))
    return out, dx.view(n, s, c).to(st["x"].dtype), dw, db


# -- what a pass cannot do without -------------------------------------------

def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "attend":
        rows = case["batch"] * case["q_len"] * case["q_heads"]
        if case["mask"]:
            kept = torch.cumsum(_silhouette(case["kv_len"]).long(), 0)
            keys = [int(kept[n - 1]) for n in _lengths(case)]
        else:
            keys = _lengths(case)
        kv = sum(keys) * case["kv_heads"] * case["dim"] * size
        q = rows * case["dim"] * size
        product = 2.0 * sum(keys) * case["q_len"] * case["q_heads"] * case["dim"]
        if case["train"]:   # forward q k v -> out; backward q k v out dout -> dq dk dv; two and five products
            return {"bytes": 4 * q + 4 * kv, "flops": 7 * product}
        return {"bytes": 2 * q + 2 * kv + 4 * rows, "flops": 2 * product}
    if case["op"] == "rotary":
        tokens = case["batch"] * case["len"]
        half = sum(_sections(case))
        return {"bytes": 2 * tokens * case["heads"] * case["dim"] * size + 4 * tokens * len(_sections(case)),
                "flops": 6.0 * tokens * case["heads"] * half}
    count = case["samples"] * case["positions"] * case["channels"]
    if case["train"]:   # x, dout -> out, dx
        return {"bytes": 4 * count * size, "flops": 35.0 * count}
    return {"bytes": 2 * count * size, "flops": 10.0 * count}


# -- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, x)
    return _exact_rotary(case, x) if case["op"] == "rotary" else _exact_norm(case, x)


def _exact_attend(case, x):
    b, lq, hq, d = x["q"].shape
    lk, hk = x["k"].shape[1:3]
    lens = _lengths(case)
    keep = _silhouette(lk).to(DEV) if case["mask"] else torch.ones(lk, dtype=torch.bool, device=DEV)
    out = torch.zeros((b, lq, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, lq), -math.inf, dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(out)
    dk, dv = (torch.zeros((b, lk, hk, d), dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(b):
        index = torch.nonzero(keep[:lens[i]]).flatten()
        if index.numel() == 0:
            continue
        for h in range(hq):
            hh = h // (hq // hk)
            km, vm = x["k"][i, index, hh].double(), x["v"][i, index, hh].double()
            for r in range(0, lq, 2048):
                qm = x["q"][i, r:r + 2048, h].double()
                logits = torch.einsum("rd,kd->rk", qm, km) / math.sqrt(d)
                norm = torch.logsumexp(logits, dim=1)
                prob = torch.exp_(logits.sub_(norm[:, None]))
                o = torch.einsum("rk,kd->rd", prob, vm)
                out[i, r:r + 2048, h] = o
                lse[i, h, r:r + 2048] = norm
                if case["train"]:
                    do = x["dout"][i, r:r + 2048, h].double()
                    dv[i].index_put_((index, torch.tensor(hh, device=DEV)), torch.einsum("rk,rd->kd", prob, do),
                                     accumulate=True)
                    dp = torch.einsum("rd,kd->rk", do, vm)
                    ds = prob * (dp - torch.einsum("rk,rk->r", prob, dp)[:, None]) / math.sqrt(d)
                    dq[i, r:r + 2048, h] = torch.einsum("rk,kd->rd", ds, km)
                    dk[i].index_put_((index, torch.tensor(hh, device=DEV)), torch.einsum("rk,rd->kd", ds, qm),
                                     accumulate=True)
    return (out, dq, dk, dv) if case["train"] else (out, lse)


def _exact_rotary(case, x):
    sections = _sections(case)
    half = sum(sections)
    value = x["x"].double().clone()
    first = 0
    for a, count in enumerate(sections):
        for i in range(first, first + count):
            turn = x["positions"][:, :, a].double() * x["frequencies"][i].double()
            if case["backward"]:
                turn = -turn
            one, two = (2 * i, 2 * i + 1) if case["pairs"] == "neighbours" else (i, i + half)
            z = torch.complex(value[..., one], value[..., two])
            z = z * torch.polar(torch.ones_like(turn), turn)[:, :, None]
            value[..., one], value[..., two] = z.real, z.imag
        first += count
    return value


def _exact_norm(case, x):
    n, s, c = x["x"].shape
    width = c // case["groups"]
    out = torch.empty((n, s, c), dtype=torch.float64, device=DEV)
    dx = torch.empty_like(out) if case["train"] else None
    dw, db = (torch.zeros(c, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(n):
        for g in range(case["groups"]):
            at = slice(g * width, (g + 1) * width)
            v = x["x"][i, :, at].double()
            var, mean = torch.var_mean(v, correction=0)
            hat = (v - mean) / torch.sqrt(var + EPS)
            z = hat * x["weight"][at].double() + x["bias"][at].double()
            if case["act"] == "silu":
                y, slope = z * torch.sigmoid(z), torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
            elif case["act"] == "gelu":
                phi = torch.special.ndtr(z)
                y, slope = z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            else:
                y, slope = z, torch.ones_like(z)
            out[i, :, at] = y
            if case["train"]:
                dz = x["dout"][i, :, at].double() * slope
                db[at] += dz.sum(0)
                dw[at] += (dz * hat).sum(0)
                dhat = dz * x["weight"][at].double()
                dx[i, :, at] = (dhat - dhat.mean() - hat * (dhat * hat).mean()) / torch.sqrt(var + EPS)
    return (out, dx, dw, db) if case["train"] else out
