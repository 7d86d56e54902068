"""Cases that measure the operators of a token layer of an image-to-Gaussians
decoder: layer norm with the residual sum in front of it, and a gated linear
recurrence over the tokens of all views.

`own` chooses what `run` computes with: the plain form (elementary torch
operations in 32 bits, rounded once at the end) or the package's kernels.  Token
counts are those of 16x16 patches: 2,500 for an 800x800 view, 8,160 for
1920x1080; widths are heads x head_dim of the decoder's attention (16 x 128,
16 x 80, 8 x 64).
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # One refined token of each of four scenes, behind a layer's residual sum (serving): latency counts.
        {"name": "norm_token", "op": "norm", "train": False, "dtype": "bf16", "batch": 4, "tokens": 1, "heads": 1,
         "channels": 2048, "residual": True},
        # The tokens of four 1920x1080 views between two layers of a preview.
        {"name": "norm_views", "op": "norm", "train": False, "dtype": "bf16", "batch": 1, "tokens": 32640, "heads": 1,
         "channels": 2048, "residual": True},
        # A training step's norm over four 800x800 views of two scenes.
        {"name": "norm_train", "op": "norm", "train": True, "dtype": "bf16", "batch": 2, "tokens": 10000, "heads": 1,
         "channels": 1280, "residual": True},
        # The norm of each head's queries, a slice of a wider projection, in training.
        {"name": "norm_heads", "op": "norm", "train": True, "dtype": "f16", "batch": 2, "tokens": 2500, "heads": 16,
         "channels": 128, "residual": False},
        # Training in float32 on odd crops and an odd width: 8 x 72 features and one of the view's own.
        {"name": "norm_odd", "op": "norm", "train": True, "dtype": "f32", "batch": 3, "tokens": 2255, "heads": 1,
         "channels": 577, "residual": False},
        # One more token of each of four scenes, from the state of those before (serving): latency counts.
        {"name": "recur_token", "op": "recur", "train": False, "dtype": "bf16", "batch": 4, "tokens": 1,
         "channels": 2048, "gate": True, "reverse": False, "drop": 0, "initial": True},
        # The largest forward: the tokens of four 1920x1080 views, one long sequence.
        {"name": "recur_views", "op": "recur", "train": False, "dtype": "bf16", "batch": 1, "tokens": 32640,
         "channels": 2048, "gate": True, "reverse": False, "drop": 0, "initial": False},
        # A training step over four 800x800 views of two scenes, the second with one view missing.
        {"name": "recur_train", "op": "recur", "train": True, "dtype": "bf16", "batch": 2, "tokens": 10000,
         "channels": 1280, "gate": True, "reverse": False, "drop": 2500, "initial": False},
        # Training backwards over short sequences whose odd lengths differ over the batch.
        {"name": "recur_short", "op": "recur", "train": True, "dtype": "f16", "batch": 12, "tokens": 1023,
         "channels": 512, "gate": True, "reverse": True, "drop": 61, "initial": True},
        # Few odd channels in float32 over a long sequence: the work lies along the tokens alone.
        {"name": "recur_narrow", "op": "recur", "train": True, "dtype": "f32", "batch": 1, "tokens": 32640,
         "channels": 77, "gate": False, "reverse": True, "drop": 0, "initial": False},
    ]


LARGEST = 32640 * 2048 * 8   # bytes of the largest cases' arrays


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = {"op": rng.choice(["norm", "recur"]), "train": rng.random() < 0.6,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "batch": _log_int(rng, 1, 16),
                "tokens": _log_int(rng, 1, 32640)}
        if case["op"] == "norm":
            case["heads"] = rng.choice([1, 1, 1, 4, 16])
            case["channels"] = rng.choice([32, 64, 72, 80, 96, 128] if case["heads"] > 1 else
                                          [64, 77, 128, 256, 512, 577, 1024, 1280, 2048, 2050, 4096])
            case["residual"] = rng.random() < 0.5
        else:
            case["channels"] = rng.choice([16, 64, 77, 128, 250, 512, 768, 1280, 2048])
            case["gate"] = rng.random() < 0.7
            case["reverse"] = rng.random() < 0.5
            case["drop"] = rng.randint(0, case["tokens"] // case["batch"]) if rng.random() < 0.5 else 0
            case["initial"] = rng.random() < 0.5
        if work(case)["bytes"] <= LARGEST:
            return case


# -- inputs -----------------------------------------------------------------

def _lengths(case):
    return [case["tokens"] - case["drop"] * (case["batch"] - 1 - i) for i in range(case["batch"])]


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    b, n, c = case["batch"], case["tokens"], case["channels"]

    def normal(*shape, dtype=dtype):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)

    if case["op"] == "norm":
        shape = (b, n, c) if case["heads"] == 1 else (b, n, case["heads"], c)
        offset = normal(c, dtype=torch.float32)
        scale = normal(c, dtype=torch.float32).abs() + 0.5
        if case["heads"] == 1:
            x = (torch.randn(shape, generator=gen, device=DEV) * scale + offset).to(dtype)
        else:   # the first half of a projection to queries and keys
            both = (torch.randn((b, n, 2) + shape[2:], generator=gen, device=DEV) * scale + offset).to(dtype)
            x = both[:, :, 0]
        state = {"x": x, "residual": normal(*shape) if case["residual"] else None,
                 "weight": 1 + 0.2 * normal(c, dtype=torch.float32), "bias": 0.2 * normal(c, dtype=torch.float32)}
        if case["train"]:
            state["dout"] = normal(*shape)
            # what reaches the sum past the layer that the norm feeds
            state["dtotal"] = normal(*shape) if case["residual"] else None
        return state
    # One projection of the tokens holds the values, the forget gates' logits and the output gates'.
    parts = 3 if case["gate"] else 2
    whole = torch.randn((b, n, parts * c), generator=gen, device=DEV)
    whole[:, :, c:2 * c] = 1.5 * whole[:, :, c:2 * c] + 3.0    # most tokens are kept for a while
    whole = whole.to(dtype)
    state = {"whole": whole, "initial": normal(b, c, dtype=torch.float32) if case["initial"] else None,
             "lengths": None}
    if case["drop"]:
        state["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    if case["train"]:
        state["dout"] = normal(b, n, c)
        state["dfinal"] = normal(b, c, dtype=torch.float32) if case["initial"] else None
    return state


def prepare(case, seed):
    state = dict(case, **_inputs(case, seed))
    if own:
        import gaussian_splatting_tile_bin_gb300 as gsr
        state["gsr"] = gsr
        state["ctx"] = gsr.Context(0)
    return state


# -- one pass ---------------------------------------------------------------

def run(state):
    return _norm(state) if state["op"] == "norm" else _recur(state)


def _norm(st):
    if own:
        gsr, ctx = st["gsr"], st["ctx"]
        out, total, mean, rstd = gsr.layer_norm_forward(ctx, st["x"], st["weight"], st["bias"],
                                                        residual=st["residual"], eps=EPS)
        results = (out,) if st["residual"] is None else (out, total)
        if st["train"]:
            results += tuple(gsr.layer_norm_backward(ctx, st["dout"], total, st["weight"], mean, rstd,
                                                     dl_dtotal=st["dtotal"]))
        return results
    dtype, w = st["x"].dtype, st["weight"]
    total = st["x"]
    if st["residual"] is not None:
        total = (st["x"].float() + st["residual"].float()).to(dtype)
    x = total.float()
    x = x - x.mean(dim=-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
    x = x * rstd
    out = (x * w + st["bias"]).to(dtype)
    results = (out,) if st["residual"] is None else (out, total)
    if st["train"]:
        dout = st["dout"].float().reshape(-1, w.numel())
        g = st["dout"].float() * w
        dx = rstd * (g - g.mean(dim=-1, keepdim=True) - x * (g * x).mean(dim=-1, keepdim=True))
        if st["dtotal"] is not None:
            dx = dx + st["dtotal"].float()
        results += (dx.to(dtype), (dout * x.reshape(dout.shape)).sum(dim=0), dout.sum(dim=0))
    return results


def _parts(st):
    parts = st["whole"].split(st["channels"], dim=2)
    return parts if st["gate"] else (*parts, None)


def _recur(st):
    x, forget, gate = _parts(st)
    if own:
        gsr, ctx = st["gsr"], st["ctx"]
        how = {"lengths": st["lengths"], "reverse": st["reverse"]}
        out, final, states = gsr.gated_recurrence_forward(ctx, x, forget, gate, initial=st["initial"],
                                                          keep=st["train"], **how)
        if not st["train"]:
            return out, final
        grad = torch.empty_like(st["whole"])   # the projection's gradient
        c = st["channels"]
        *_, dinitial = gsr.gated_recurrence_backward(
            ctx, st["dout"], x, forget, gate, states, dl_dfinal=st["dfinal"], **how, dl_dx=grad[:, :, :c],
            dl_dforget=grad[:, :, c:2 * c], dl_dgate=grad[:, :, 2 * c:] if st["gate"] else None)
        return out, final, grad, dinitial
    b, n, c = x.shape
    step = torch.arange(n, device=x.device).expand(b, n)
    length = torch.full((b, 1), n, device=x.device) if st["lengths"] is None else st["lengths"][:, None].long()
    valid = (step < length)[:, :, None]
    # Tokens in the order of the recurrence, and back.
    order = torch.where(step < length, length - 1 - step, step) if st["reverse"] else step
    index = order[:, :, None].expand(b, n, c)
    xs, keep = x.float().gather(1, index), 1.0 / (1.0 + torch.exp(-forget.float().gather(1, index)))
    enter = torch.where(valid, 1.0 / (1.0 + torch.exp(forget.float().gather(1, index))), 0.0)
    keep = torch.where(valid, keep, 1.0)
    first = torch.zeros((b, c), device=x.device) if st["initial"] is None else st["initial"]
    h = _scan(keep, torch.where(valid, enter * xs, 0.0), first)
    final = h[:, -1].clone()
    if gate is None:
        slope, opened = None, torch.ones_like(h)
    else:
        o = gate.float().gather(1, index)
        sig = 1.0 / (1.0 + torch.exp(-o))
        opened, slope = o * sig, sig * (1.0 + o * (1.0 - sig))
    out = torch.where(valid, h * opened, 0.0).gather(1, index).to(x.dtype)
    if not st["train"]:
        return out, final
    dout = st["dout"].float().gather(1, index)
    before = torch.cat([first[:, None], h[:, :-1]], dim=1)
    last = torch.zeros_like(first) if st["dfinal"] is None else st["dfinal"]
    # g_t = dh_t + a_(t+1) g_(t+1), from the last token on; what is behind a sequence keeps the final state's.
    after = torch.cat([keep[:, 1:], torch.ones_like(keep[:, :1])], dim=1)
    g = _scan(after.flip(1), torch.where(valid, dout * opened, 0.0).flip(1), last).flip(1)
    grads = [g * enter, g * (before - xs) * keep * enter]
    if gate is not None:
        grads.append(dout * h * slope)
    grad = torch.cat([torch.where(valid, t, 0.0).gather(1, index).to(x.dtype) for t in grads], dim=2)
    return out, final, grad, keep[:, 0] * g[:, 0]


def _scan(a, b, first):
    """h_t = a_t h_(t-1) + b_t along dimension 1, by doubling."""
    a, b = a.clone(), b.clone()
    b[:, 0] += a[:, 0] * first
    shift = 1
    while shift < a.shape[1]:
        b[:, shift:] = b[:, shift:] + a[:, shift:] * b[:, :-shift]
        a[:, shift:] = a[:, shift:] * a[:, :-shift]
        shift *= 2
    return b


# -- what a pass cannot do without -------------------------------------------

def work(case):
    size, b, n, c = SIZE[case["dtype"]], case["batch"], case["tokens"], case["channels"]
    if case["op"] == "norm":
        count = b * n * case["heads"] * c
        arrays = 4 if case["residual"] else 2                 # x, residual -> out, total
        if case["train"]:                                     # dout, dtotal -> dx (x or the sum is read already)
            arrays += 3 if case["residual"] else 2
        return {"bytes": arrays * count * size + 8 * c, "flops": (22.0 if case["train"] else 8.0) * count}
    count = sum(max(0, t) for t in _lengths(case)) * c
    arrays = 4 if case["gate"] else 3                         # x, forget, gate -> out
    if case["train"]:                                         # dout -> dx, dforget, dgate
        arrays += 4 if case["gate"] else 3
    return {"bytes": arrays * count * size + (8 * b * c if case["initial"] else 4 * b * c),
            "flops": (30.0 if case["train"] else 12.0) * count}


# -- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    return _exact_norm(case, x) if case["op"] == "norm" else _exact_recur(case, x)


def _exact_norm(case, t):
    c = case["channels"]
    x = t["x"].double()
    whole = x if t["residual"] is None else x + t["residual"].double()
    # the norm is that of the sum as it is stored
    rows = whole.to(t["x"].dtype).double().reshape(-1, c)
    var, mean = torch.var_mean(rows, dim=1, correction=0, keepdim=True)
    scale = torch.rsqrt(var + EPS)
    hat = (rows - mean) * scale
    out = torch.addcmul(t["bias"].double(), hat, t["weight"].double()).view(whole.shape)
    results = (out,) if t["residual"] is None else (out, whole)
    if case["train"]:
        dout = t["dout"].double().reshape(-1, c)
        dhat = dout * t["weight"].double()
        dx = scale * (dhat - dhat.sum(1, keepdim=True) / c
                      - hat * torch.einsum("rc,rc->r", dhat, hat)[:, None] / c)
        dx = dx.view(whole.shape)
        if t["dtotal"] is not None:
            dx = dx + t["dtotal"].double()
        results += (dx, torch.einsum("rc,rc->c", dout, hat), dout.sum(0))
    return results


def _exact_recur(case, t):
    """Token by token, item lengths by a mask."""
    b, n, c = case["batch"], case["tokens"], case["channels"]
    parts = [p.transpose(0, 1).double() for p in t["whole"].split(c, dim=2)]
    values, logits = parts[0], parts[1]
    opened = torch.nn.functional.silu(parts[2]) if case["gate"] else None
    live = [torch.tensor([k < m for m in _lengths(case)], device=DEV)[:, None] if case["drop"] else None
            for k in range(n)]
    tokens = range(n - 1, -1, -1) if case["reverse"] else range(n)
    keep, enter = torch.sigmoid(logits), torch.sigmoid(-logits)
    h = torch.zeros((b, c), dtype=torch.float64, device=DEV) if t["initial"] is None else t["initial"].double()
    path = torch.empty((n, b, c), dtype=torch.float64, device=DEV)
    before = torch.empty_like(path) if case["train"] else None
    for k in tokens:
        if before is not None:
            before[k] = h
        new = torch.lerp(h, values[k], enter[k])
        h = new if live[k] is None else torch.where(live[k], new, h)
        path[k] = h
    covered = torch.ones((n, b, 1), dtype=torch.bool, device=DEV)
    if case["drop"]:
        covered = torch.stack(live)
    out = path if opened is None else path * opened
    out = torch.where(covered, out, 0.0).transpose(0, 1)
    if not case["train"]:
        return out, h
    dout = t["dout"].transpose(0, 1).double()
    into = dout if opened is None else dout * opened
    g = torch.zeros((b, c), dtype=torch.float64, device=DEV) if t["dfinal"] is None else t["dfinal"].double()
    reached = torch.empty_like(path)
    for k in reversed(tokens):
        here = g + into[k]
        reached[k] = here
        new = here * keep[k]
        g = new if live[k] is None else torch.where(live[k], new, g)
    grads = [reached * enter, reached * (before - values) * keep * enter]
    if opened is not None:
        sig = torch.sigmoid(parts[2])
        grads.append(dout * path * (sig + opened * (1 - sig)))
    grad = torch.where(covered, torch.cat(grads, dim=2), 0.0).transpose(0, 1)
    return out, h, grad, g
