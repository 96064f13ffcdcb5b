"""Cases of a recurrent layer's further operators: the gated linear recurrence
(prompts, training steps, single tokens), the RMS norm with the residual's
addition and an 8-bit output, and low-rank adapters of many requests beside a
shared projection.

``own`` selects what ``run`` calls: the operators' plain form in elementary
torch operations (32-bit arithmetic, one rounding at the end), or the library.

Layouts are the sequence operators': activations [N, C, L] stored as L rows of
C channels, packed batches [1, C, T] with int32 ``offsets``; the norm and the
adapters work on rows [M, C].
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8, F8_MAX = torch.float8_e4m3fn, 448.0
SHARP, EPS = 8.0, 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One decoding step of the recurrence for a batch of running requests.
        dict(name="gated token bf16", op="gated_token", dtype="bf16", n=64, c=4096),
        # A prompt batch of equal lengths, ending with the state that decoding starts from.
        dict(name="gated prompt bf16", op="gated", dtype="bf16", n=8, l=2048, c=4096, packed=False, start=False),
        # One long document: few rows, a long axis.
        dict(name="gated long bf16", op="gated", dtype="bf16", n=1, l=65536, c=2560, packed=False, start=False),
        # Requests of unlike lengths packed in one row of tokens, continuing from cached states; odd sizes.
        dict(name="gated packed f16", op="gated", dtype="f16", n=13, l=9001, c=1160, packed=True, start=True),
        # A training step: output and every gradient.
        dict(name="gated train bf16", op="gated_train", dtype="bf16", n=8, l=2048, c=4096),
        # The norm before a projection with 8-bit inputs, one decoding step of a batch.
        dict(name="norm token f8", op="norm", dtype="bf16", m=32, c=4096, f8=True, group=0),
        # The same for a prompt batch, one scale for each 128 channels.
        dict(name="norm prompt f8", op="norm", dtype="bf16", m=8192, c=5120, f8=True, group=128),
        # A training step: output, new residual and every gradient.
        dict(name="norm train bf16", op="norm_train", dtype="bf16", m=16384, c=4096),
        # One token each of requests with adapters of their own, next to a projection.
        dict(name="adapters token bf16", op="adapters", dtype="bf16", m=32, k=4096, n=4096, r=16, e=24, f8=False, runs=False),
        # A larger decoding batch, odd sizes.
        dict(name="adapters batch f16", op="adapters", dtype="f16", m=203, k=2560, n=6913, r=24, e=40, f8=False, runs=False),
        # Prompts of several requests, one after the other.
        dict(name="adapters prompt bf16", op="adapters", dtype="bf16", m=8192, k=4096, n=8192, r=32, e=6, f8=False, runs=True),
        # Prompts whose rows the norm left in 8 bits.
        dict(name="adapters prompt f8", op="adapters", dtype="bf16", m=4100, k=5120, n=5120, r=64, e=8, f8=True, runs=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in lo .. hi (lo itself need not be one), even over the logarithm."""
    v = -(-int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // step) * step
    return min(v, hi // step * step)


def draw(rng):
    op = rng.choice(["gated_token", "gated", "gated", "gated_train", "norm", "norm", "norm_train", "adapters", "adapters", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    step = rng.choice([1, 8, 64])  # channels: any number, whole vectors, whole blocks
    if op == "gated_token":
        return dict(op=op, dtype=dtype, n=_log(rng, 1, 256), c=_log(rng, 256, 8192, step))
    if op in ("gated", "gated_train"):
        c = _log(rng, 192, 4096, step)
        tokens = _log(rng, 100, 2 ** (25 if op == "gated" else 24) // c)
        n = _log(rng, 1, min(32, tokens))
        if op == "gated_train":
            return dict(op=op, dtype=dtype, n=n, l=tokens // n, c=c)
        packed = rng.random() < 0.4
        return dict(op=op, dtype=dtype, n=n, l=tokens if packed else tokens // n, c=c, packed=packed, start=rng.random() < 0.5)
    if op in ("norm", "norm_train"):
        f8 = op == "norm" and rng.random() < 0.6
        group = rng.choice([0, 0, 32, 64, 128]) if f8 else 0
        c = _log(rng, 256, 16384, max(step, group))
        case = dict(op=op, dtype=dtype, m=_log(rng, 1, min(16384, 2 ** 25 // c)), c=c)
        return case if op == "norm_train" else dict(case, f8=f8, group=group)
    runs = rng.random() < 0.5
    k = _log(rng, 512, 8192, step)
    n = _log(rng, 512, 8192, rng.choice([1, 8, 64]))
    m = _log(rng, 64, min(8192, 2 ** 25 // max(k, n))) if runs else _log(rng, 1, 256)
    return dict(op=op, dtype=dtype, m=m, k=k, n=n, r=rng.choice([4, 8, 16, 16, 24, 32, 64, 128]), e=_log(rng, 1, 8 if runs else 48),
                f8=rng.random() < 0.3, runs=runs)


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("gated"):
        n, c = case["n"], case["c"]
        if op == "gated_token":
            return {"bytes": 4 * n * c * e + 8 * n * c + 4 * c, "flops": 20 * n * c}
        t = case["l"] * c if case.get("packed") else n * case["l"] * c
        if op == "gated":
            return {"bytes": 4 * t * e + 4 * n * c * (2 if case["start"] else 1) + 4 * c, "flops": 20 * t}
        return {"bytes": 8 * t * e + 8 * c, "flops": 60 * t}
    if op == "adapters":
        m, k, n, r = case["m"], case["k"], case["n"], case["r"]
        used = min(case["e"], m)
        return {"bytes": m * k * (1 if case["f8"] else e) + (4 * m if case["f8"] else 0) + 2 * m * n * e + used * r * (k + n) * e + 4 * (m + used),
                "flops": 2 * m * r * (k + n)}
    m, c = case["m"], case["c"]
    if op == "norm_train":
        return {"bytes": 6 * m * c * e + 2 * c * e, "flops": 16 * m * c}
    scales = 4 * m * (c // case["group"] if case["group"] else 1)
    return {"bytes": 3 * m * c * e + c * e + (m * c + scales if case["f8"] else m * c * e), "flops": 8 * m * c}


# ------------------------------------------------------------------ inputs --

def _offsets(n, total, gen):
    """Cuts 0 .. total into n sequences of unlike lengths (now and then empty ones)."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=gen).sort().values
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([total])])
    return off.to(torch.int32).to(DEV), int(off.diff().max())


def _rows(gen, dt, n, l, c):
    """Normal values [n, c, l], stored with l rows of c channels."""
    return torch.randn((n, l, c), generator=gen, device=DEV).to(dt).transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    if op == "adapters":
        m, k, n, r, e = (case[v] for v in ("m", "k", "n", "r", "e"))
        x = rand(m, k)
        s["x_scales"] = None
        if case["f8"]:
            s["x_scales"] = x.abs().amax(1, keepdim=True) / F8_MAX
            s["x"] = (x / s["x_scales"]).to(F8)
        else:
            s["x"] = x.to(dt)
        s["a"] = (rand(e, r, k) / math.sqrt(k)).to(dt)
        s["b"] = (rand(e, n, r) / math.sqrt(r)).to(dt)
        s["scaling"] = 0.5 + torch.rand(e, generator=gen, device=DEV)
        s["base"] = rand(m, n).to(dt)
        # Every adapter has a row where there are enough; a tenth of the requests have none.
        index = torch.cat([torch.randperm(e, generator=host), torch.randint(0, e, (m,), generator=host)])
        index = torch.where(torch.rand(m + e, generator=host) < 0.1, -1, index)
        if case["runs"]:
            cuts = torch.randint(0, m, (2 * e - 1,), generator=host).sort().values
            index = index[torch.searchsorted(cuts, torch.arange(m), right=True)]
        s["index"] = index[:m].to(torch.int32).to(DEV)
        if own:  # a serving program keeps the plan of its batch's shape
            from depthwise_stencil_implicit_amd import lm
            s["plan"] = lm.PreparedAdapters(s["x"], s["a"], s["b"], s["index"], base=s["base"], scaling=s["scaling"],
                                            x_scales=s["x_scales"])
        return s
    if op.startswith("norm"):
        m, c = case["m"], case["c"]
        s["x"], s["residual"] = rand(m, c).to(dt), (2 * rand(m, c)).to(dt)
        s["w"] = (1 + 0.1 * rand(c)).to(dt)
        if op == "norm_train":
            s["gy"], s["gresidual"] = rand(m, c).to(dt), rand(m, c).to(dt)
        elif own:  # a serving program keeps the plan of its batch's shape
            from depthwise_stencil_implicit_amd import lm
            s["plan"] = lm.PreparedRmsNorm(s["x"], s["w"], s["residual"], eps=EPS, out_dtype=F8 if case["f8"] else None,
                                           group=case["group"] or None)
        return s
    n, c = case["n"], case["c"]
    # Factors per step of 0.9 .. 0.999 at an open gate.
    k = -torch.log(0.9 + 0.099 * torch.rand(c, generator=gen, device=DEV))
    s["decay"] = torch.log(torch.expm1(k / SHARP))
    start = rand(n, c)
    if op == "gated_token":
        s["x"], s["r"], s["i"], s["state"] = rand(n, c).to(dt), rand(n, c).to(dt), rand(n, c).to(dt), start
        if own:  # a decoding loop keeps the plan of its step
            from depthwise_stencil_implicit_amd import lm
            s["plan"] = lm.PreparedGatedRecurrenceStep(s["x"], s["r"], s["i"], s["decay"], s["state"], sharpness=SHARP)
        return s
    packed = case.get("packed", False)
    s["offsets"], s["max_len"] = _offsets(n, case["l"], host) if packed else (None, None)
    for v in ("x", "r", "i") + (("gy",) if op == "gated_train" else ()):
        s[v] = _rows(gen, dt, 1 if packed else n, case["l"], c)
    s["state"] = start if case.get("start") else None
    return s


# -------------------------------------------------------------- plain forms --

def _factors(x, r, i, decay):
    """(a, m iota x, rho, iota, m, k) of rows of channels."""
    k = SHARP * torch.logaddexp(decay, torch.zeros_like(decay))
    rho, iota = torch.sigmoid(r), torch.sigmoid(i)
    log_a = -k * rho
    m = torch.sqrt(-torch.expm1(2 * log_a))
    return torch.exp(log_a), m * iota * x, rho, iota, m, k


def _scan(a, h, span):
    """h[t] += a[t] h[t-1] along dim 1, by doubling: log2(span) passes over whole tensors."""
    d = 1
    while d < span:
        h = torch.cat([h[:, :d], torch.addcmul(h[:, d:], a[:, d:], h[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return h


def _plain_gated(s):
    dt = s["x"].dtype
    offsets = s["offsets"]
    x, r, i = (s[v].float().transpose(1, 2) for v in ("x", "r", "i"))
    n, l, c = x.shape
    a, u, rho, iota, m, k = _factors(x, r, i, s["decay"])
    span = s["max_len"] or l
    if offsets is None:
        if s["state"] is not None:
            u[:, 0] += a[:, 0] * s["state"]
        h = _scan(a, u, span)
        last = h[:, -1]
    else:
        full = offsets.long().diff() > 0
        start = s["state"] if s["state"] is not None else torch.zeros(full.numel(), c, device=x.device)
        at = offsets.long()[:-1][full]
        u[0, at] += a[0, at] * start[full]
        cut = a.clone()
        cut[0, at] = 0
        h = _scan(cut, u, span)
        last = torch.where(full[:, None], h[0, (offsets.long()[1:] - 1).clamp(min=0)], start)
    out = {"y": h.transpose(1, 2).to(dt)}
    if "gy" not in s:
        return dict(out, state=last)
    gh = s["gy"].float().transpose(1, 2)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    gh = _scan(after.flip(1), gh.flip(1), l).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    dl = gh * (a * before - iota * x * a * a / m)
    back = lambda v: v.transpose(1, 2).to(dt)  # noqa: E731
    out["dx"] = back(gh * m * iota)
    out["di"] = back(gh * m * x * iota * (1 - iota))
    out["dr"] = back(-k * dl * rho * (1 - rho))
    out["ddecay"] = -SHARP * torch.sigmoid(s["decay"]) * (dl * rho).sum((0, 1))
    return out


def _plain_gated_token(s):
    a, u = _factors(s["x"].float(), s["r"].float(), s["i"].float(), s["decay"])[:2]
    s["state"].copy_(a * s["state"] + u)
    return {"y": s["state"].to(s["x"].dtype), "state": s["state"]}


def _plain_norm(s):
    case, dt = s["case"], s["x"].dtype
    v, w = s["x"].float() + s["residual"].float(), s["w"].float()
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    y = v * rstd * w
    out = {"residual": v.to(dt)}
    if "gy" in s:
        g = s["gy"].float()
        wg = w * g
        dx = s["gresidual"].float() + rstd * (wg - v * rstd * rstd * (wg * v).mean(1, keepdim=True))
        return dict(out, y=y.to(dt), dx=dx.to(dt), dw=(g * v * rstd).sum(0).to(dt))
    if not case["f8"]:
        return dict(out, y=y.to(dt))
    grouped = y.view(case["m"], -1, case["group"] or case["c"])
    top = grouped.abs().amax(2, keepdim=True)
    top = torch.where(top == 0, F8_MAX, top)  # a group of zeros: scale 1
    return dict(out, y=(grouped * (F8_MAX / top)).view_as(y).to(F8), scales=top[..., 0] / F8_MAX)


def _plain_adapters(s):
    """Products with every adapter, of which each row keeps its own's."""
    e, r, k = s["a"].shape
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = x * s["x_scales"]
    t = (x @ s["a"].float().view(e * r, k).t()).view(-1, e, r)
    mine = s["index"][:, None] == torch.arange(e, device=x.device)
    t = t * torch.where(mine, s["scaling"], 0.0)[..., None]
    y = t.view(-1, e * r) @ s["b"].float().transpose(1, 2).reshape(e * r, -1)
    return (s["base"].float() + y).to(s["base"].dtype)


# --------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "adapters":
            return _plain_adapters(s)
        if op.startswith("norm"):
            return _plain_norm(s)
        return _plain_gated_token(s) if op == "gated_token" else _plain_gated(s)

    if op == "adapters":
        return s["plan"].run(s["x"], s["a"], s["b"], s["index"], base=s["base"], scaling=s["scaling"], x_scales=s["x_scales"])
    if op == "norm":
        r = s["plan"].run(s["x"], s["w"], s["residual"])
        out = {"residual": r.residual, "y": r.y}
        return dict(out, scales=r.scales) if case["f8"] else out
    if op == "gated_token":
        return {"y": s["plan"].run(s["x"], s["r"], s["i"], s["decay"], s["state"]), "state": s["state"]}
    from depthwise_stencil_implicit_amd import lm
    if op == "norm_train":
        f = lm.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS, save=True)
        g = lm.rms_norm_backward(s["gy"], s["x"], s["w"], f.rstd, residual=s["residual"], gresidual=s["gresidual"])
        return {"y": f.y, "residual": f.residual, "dx": g.dx, "dw": g.dw}
    args = (s["x"], s["r"], s["i"], s["decay"])
    if op == "gated":
        f = lm.gated_recurrence(*args, sharpness=SHARP, state=s["state"], offsets=s["offsets"], max_len=s["max_len"], return_state=True)
        return {"y": f.y, "state": f.state}
    f = lm.gated_recurrence(*args, sharpness=SHARP, save=True)
    g = lm.gated_recurrence_backward(s["gy"], *args, sharpness=SHARP, saved=f.saved)
    return {"y": f.y, "dx": g.dx, "dr": g.dr, "di": g.di, "ddecay": g.ddecay}


# ------------------------------------------------------- definition, 64 bits --

def _exact_gated(s):
    """Token by token: every batch row at once, the packed sequences one after the other."""
    case = s["case"]
    x, r, i, decay = (s[v].double() for v in ("x", "r", "i", "decay"))
    k = SHARP * torch.log1p(torch.exp(decay))[:, None]
    gate_r, gate_i = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    a = torch.exp(-k * gate_r)
    m = torch.sqrt(-torch.expm1(-2 * k * gate_r))
    u = m * gate_i * x
    state = s["state"].double() if s["state"] is not None else torch.zeros((case["n"], case["c"]), dtype=torch.float64, device=x.device)
    h = torch.empty_like(x)
    if s["offsets"] is None:
        before = torch.empty_like(x) if "gy" in s else None
        now = state
        for t in range(case["l"]):
            if before is not None:
                before[..., t] = now
            now = a[..., t] * now + u[..., t]
            h[..., t] = now
        last = now
    else:
        off, last = s["offsets"].tolist(), state.clone()
        for q in range(case["n"]):
            now = state[q]
            for t in range(off[q], off[q + 1]):
                now = a[0, :, t] * now + u[0, :, t]
                h[0, :, t] = now
            last[q] = now
    if "gy" not in s:
        return {"y": h, "state": last}
    g = s["gy"].double()
    dx, dr, di = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dk = torch.zeros(case["c"], dtype=torch.float64, device=x.device)
    carry = torch.zeros_like(state)
    for t in reversed(range(case["l"])):
        gh = g[..., t] + carry
        at, mt, rt, it = a[..., t], m[..., t], gate_r[..., t], gate_i[..., t]
        dx[..., t] = gh * mt * it
        di[..., t] = gh * mt * x[..., t] * it * (1 - it)
        dl = gh * before[..., t] * at - gh * it * x[..., t] * at ** 2 / mt
        dr[..., t] = -k[:, 0] * dl * rt * (1 - rt)
        dk -= (dl * rt).sum(0)
        carry = at * gh
    return {"y": h, "dx": dx, "dr": dr, "di": di, "ddecay": dk * SHARP / (1 + torch.exp(-decay))}


def _exact_norm(s):
    case = s["case"]
    v = s["x"].double() + s["residual"].double()
    w = s["w"].double()
    root = torch.sqrt((v ** 2).sum(1) / case["c"] + EPS)[:, None]
    y = w * v / root
    if "gy" in s:
        g = s["gy"].double()
        unit = v / root
        inner = (g * w * unit).sum(1)[:, None] / case["c"]
        return {"residual": v, "y": y, "dx": s["gresidual"].double() + (g * w - unit * inner) / root, "dw": (g * unit).sum(0)}
    if not case["f8"]:
        return {"residual": v, "y": y}
    width = case["group"] or case["c"]
    top = torch.stack([p.abs().amax(1) for p in y.split(width, 1)], 1)
    return {"residual": v, "y": y * (F8_MAX / top).repeat_interleave(width, 1), "scales": top / F8_MAX}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adapters":
        y, index = s["base"].double(), s["index"].tolist()
        for e in set(index) - {-1}:
            rows = [j for j, v in enumerate(index) if v == e]
            x = s["x"][rows].double() if s["x_scales"] is None else s["x"].float()[rows].double() * s["x_scales"][rows].double()
            y[rows] += s["scaling"][e].double() * (x @ s["a"][e].double().T) @ s["b"][e].double().T
        return y
    if op.startswith("norm"):
        return _exact_norm(s)
    if op == "gated_token":
        one = {v: s[v][..., None] for v in ("x", "r", "i")}
        r = _exact_gated(dict(s, **one, offsets=None, case=dict(case, l=1)))
        return {"y": r["y"][..., 0], "state": r["state"]}
    return _exact_gated(s)
