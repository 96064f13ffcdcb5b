"""Cases of the sequence operators: the short causal convolution, the selective
state space scan (prompts, training steps, single tokens) and products with
4-bit weights.

``own`` selects what ``run`` calls: the operators' plain form in elementary
torch operations (32-bit arithmetic, one rounding at the end), or the library.

Logical layouts follow the convolution library: activations are [N, C, L],
stored channels-last (L rows of C channels); a packed batch of sequences is
[1, C, T] with ``offsets`` (int32, one more than sequences), sequence s being
the rows offsets[s] .. offsets[s+1]-1.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One decoding step of the convolution for a batch of running requests.
        dict(name="conv token bf16", op="conv_token", dtype="bf16", n=16, c=4096, k=4, act="silu", bias=True),
        # A prompt batch of equal lengths, ending with the state that decoding starts from.
        dict(name="conv prompt bf16", op="conv", dtype="bf16", n=4, l=2048, c=4096, k=4, act="silu", bias=True,
             packed=False, start=False),
        # Requests of unlike lengths packed in one row of tokens, continuing from cached states; odd sizes.
        dict(name="conv packed f16", op="conv", dtype="f16", n=13, l=5003, c=1160, k=3, act="none", bias=False,
             packed=True, start=True),
        # A training step: output and every gradient.
        dict(name="conv train bf16", op="conv_train", dtype="bf16", n=8, l=2048, c=2048, k=4, act="silu", bias=True),
        # One decoding step of the scan for a batch of running requests.
        dict(name="scan token bf16", op="scan_token", dtype="bf16", n=32, c=4096, s=16, g=1),
        # A prompt batch.
        dict(name="scan prompt bf16", op="scan", dtype="bf16", n=8, l=1024, c=2048, s=16, g=1, packed=False, start=False),
        # One long document: few rows, a long axis.
        dict(name="scan long bf16", op="scan", dtype="bf16", n=1, l=32768, c=1536, s=16, g=1, packed=False, start=False),
        # Packed prompts of unlike lengths with cached states, two groups of B and C, odd sizes, 32 bits.
        dict(name="scan packed f32", op="scan", dtype="f32", n=7, l=1931, c=720, s=12, g=2, packed=True, start=True),
        # A training step: output and every gradient.
        dict(name="scan train bf16", op="scan_train", dtype="bf16", n=8, l=2048, c=2048, s=16, g=1),
        # One token through a projection.
        dict(name="mv4 token bf16", op="mv4", dtype="bf16", m=1, k=4096, n=8192, group=128, zeros=False, bias=False),
        # A few requests at once, asymmetric weights, an odd number of outputs.
        dict(name="mv4 batch f16", op="mv4", dtype="f16", m=11, k=5120, n=2501, group=64, zeros=True, bias=True),
        # The widest product of a step, the output head.
        dict(name="mv4 head bf16", op="mv4", dtype="bf16", m=4, k=8192, n=65536, group=128, zeros=False, bias=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in lo .. hi (lo itself need not be one), even over the logarithm; 3072 is left out."""
    v = -(-int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // step) * step
    v = min(v, hi // step * step)
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["conv_token", "conv", "conv_train", "scan_token", "scan", "scan_train", "mv4", "mv4"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    step = rng.choice([1, 8, 64])  # channels: any number, whole vectors, whole blocks
    if op == "conv_token":
        return dict(op=op, dtype=dtype, n=_log(rng, 1, 256), c=_log(rng, 256, 8192, step), k=rng.randint(2, 4),
                    act=rng.choice(["silu", "none"]), bias=rng.random() < 0.7)
    if op == "scan_token":
        return dict(op=op, dtype=dtype, n=_log(rng, 1, 256), c=_log(rng, 256, 8192, 8 * step), s=rng.choice([8, 12, 16, 16, 32]),
                    g=rng.choice([1, 1, 2, 4]))
    if op == "mv4":
        group = rng.choice([32, 64, 128])
        n = _log(rng, 512, 65536)
        return dict(op=op, dtype=dtype, m=_log(rng, 1, 24), k=_log(rng, 1024, min(16384, 2 ** 29 // n), group), n=n, group=group,
                    zeros=rng.random() < 0.4, bias=rng.random() < 0.4)
    c = _log(rng, 192, 4096, max(8, step) if op.startswith("scan") else step)
    if op == "conv" or op == "conv_train":
        tokens = _log(rng, 200, 2 ** 25 // c)
        case = dict(op=op, dtype=dtype, c=c, k=rng.randint(2, 4), act=rng.choice(["silu", "none"]), bias=rng.random() < 0.7)
    else:
        s = rng.choice([8, 12, 16, 16, 32])
        tokens = _log(rng, 100, 2 ** (29 if op == "scan" else 28) // (c * s))
        case = dict(op=op, dtype=dtype, c=c, s=s, g=rng.choice([1, 1, 2, 4]))
    n = _log(rng, 1, min(32, tokens))
    if op in ("conv", "scan"):
        case["start"] = rng.random() < 0.5
        case["packed"] = rng.random() < 0.4
        return dict(case, n=n, l=tokens if case["packed"] else tokens // n)
    return dict(case, n=n, l=tokens // n)


def _tokens(case):
    return case["l"] if case.get("packed") else case["n"] * case["l"]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "mv4":
        m, k, n = case["m"], case["k"], case["n"]
        scales = n * (k // case["group"]) * e * (2 if case["zeros"] else 1)
        return {"bytes": n * k // 2 + scales + (m * k + m * n + (n if case["bias"] else 0)) * e, "flops": 2 * m * n * k}
    n, c = case["n"], case["c"]
    if op.startswith("conv"):
        k = case["k"]
        act = 4 if case["act"] == "silu" else 0
        par = c * (k + (1 if case["bias"] else 0)) * e
        st = n * c * (k - 1) * e
        if op == "conv_token":
            return {"bytes": 2 * n * c * e + 2 * st + par, "flops": n * c * (2 * k + act)}
        t = _tokens(case) * c
        if op == "conv":
            return {"bytes": 2 * t * e + st * (2 if case["start"] else 1) + par, "flops": t * (2 * k + act)}
        return {"bytes": 4 * t * e + 2 * par, "flops": t * (8 * k + 3 * act)}
    s, g = case["s"], case["g"]
    par = c * s * 4 + 2 * c * 4
    st = n * c * s * 4
    if op == "scan_token":
        return {"bytes": 4 * n * c * e + 2 * n * g * s * e + 2 * st + par, "flops": n * c * (7 * s + 16)}
    t = _tokens(case)
    if op == "scan":
        return {"bytes": (4 * c + 2 * g * s) * t * e + st * (2 if case["start"] else 1) + par, "flops": t * c * (7 * s + 16)}
    return {"bytes": (8 * c + 4 * g * s) * t * e + 2 * par, "flops": t * c * (20 * s + 40)}


# ------------------------------------------------------------------ inputs --

def _offsets(n, total, gen):
    """Cuts 0 .. total into n sequences of unlike lengths (now and then empty ones)."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=gen).sort().values
    lens = torch.cat([cuts, torch.tensor([total])]) - torch.cat([torch.tensor([0]), cuts])
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = lens.cumsum(0)
    return off.to(DEV), int(lens.max())


def _rows(gen, dt, n, l, *c):
    """Normal values [n, *c, l], stored with l rows of c channels."""
    v = torch.randn((n, l) + c, generator=gen, device=DEV).to(dt)
    return v.movedim(1, -1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    if op == "mv4":
        m, k, n, groups = case["m"], case["k"], case["n"], case["k"] // case["group"]
        s["x"] = rand(m, k).to(dt)
        s["packed"] = torch.randint(0, 256, (n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((n, groups), generator=gen, device=DEV)) / (4 * math.sqrt(k))).to(dt)
        s["zeros"] = torch.randint(5, 12, (n, groups), generator=gen, device=DEV).to(dt) if case["zeros"] else None
        s["bias"] = (0.1 * rand(n)).to(dt) if case["bias"] else None
        if own:  # a serving program keeps the plan of its weight's shape
            from depthwise_stencil_implicit_amd import lm
            s["plan"] = lm.PreparedMatvec4(s["x"], s["packed"], s["scales"], s["zeros"], s["bias"])
        return s
    n, c = case["n"], case["c"]
    packed = case.get("packed", False)
    s["offsets"], s["max_len"] = _offsets(n, case["l"], host) if packed else (None, None)
    rows, l = (1 if packed else n), case.get("l", 1)
    if op.startswith("conv"):
        k = case["k"]
        s["w"] = (rand(c, k) / math.sqrt(k)).to(dt)
        s["b"] = (0.1 * rand(c)).to(dt) if case["bias"] else None
        start = (torch.randn((n, k - 1, c), generator=gen, device=DEV).to(dt)).movedim(1, -1)
        if op == "conv_token":
            s["x"], s["state"] = rand(n, c).to(dt), start
            if own:  # a decoding loop keeps the plan of its step
                from depthwise_stencil_implicit_amd import lm
                s["plan"] = lm.PreparedCausalConvStep(s["x"], s["w"], s["b"], s["state"], activation=case["act"])
            return s
        s["x"] = _rows(gen, dt, rows, l, c)
        s["state"] = start if case.get("start") else None
        if op == "conv_train":
            s["gy"] = _rows(gen, dt, rows, l, c)
        return s
    st, g = case["s"], case["g"]
    # Decay rates spread over the states, step sizes log-uniform in 1e-3 .. 1e-1 before the input's part.
    s["A"] = -torch.arange(1, st + 1, device=DEV) * torch.exp(0.1 * rand(c, st))
    step = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(c, generator=gen, device=DEV))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1 + 0.1 * rand(c)
    start = rand(n, c, st)
    if op == "scan_token":
        s["x"], s["z"], s["dt"] = rand(n, c).to(dt), rand(n, c).to(dt), (0.5 * rand(n, c)).to(dt)
        s["B"], s["C"], s["state"] = rand(n, g, st).to(dt), rand(n, g, st).to(dt), start
        if own:  # a decoding loop keeps the plan of its step
            from depthwise_stencil_implicit_amd import lm
            s["plan"] = lm.PreparedSelectiveScanStep(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                                                     z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
        return s
    s["x"], s["z"] = _rows(gen, dt, rows, l, c), _rows(gen, dt, rows, l, c)
    s["dt"] = _rows(gen, dt, rows, l, c).mul_(0.5)
    s["B"], s["C"] = _rows(gen, dt, rows, l, g, st), _rows(gen, dt, rows, l, g, st)
    s["state"] = start if case.get("start") else None
    if op == "scan_train":
        s["gy"] = _rows(gen, dt, rows, l, c)
    return s


# -------------------------------------------------------------- plain forms --

def _silu(p):
    return p * torch.sigmoid(p)


def _silu_slope(p):
    q = torch.sigmoid(p)
    return q * (1 + p * (1 - q))


def _plain_conv(x, w, b, act, state, offsets, gy=None):
    """x [N, C, L] (or [1, C, T] with offsets); output, last state, and for gy the gradients of x, w and b."""
    dt = x.dtype
    k = w.shape[1]
    if offsets is None:
        n, c, l = x.shape
        front = torch.zeros(n, c, k - 1, device=x.device) if state is None else state.float()
        xp = torch.cat([front, x.float()], 2)
        last = xp[:, :, l:]
        win = xp.unfold(2, k, 1)  # [N, C, L, k]
    else:  # the sequences one after the other, each behind its k - 1 values of state
        c, t = x.shape[1:]
        n = offsets.numel() - 1
        off = offsets.long()
        row = torch.arange(t, device=x.device)
        seq = torch.searchsorted(off[1:], row, right=True)
        j = torch.arange(k - 1, device=x.device)
        s = torch.arange(n, device=x.device)[:, None] * (k - 1)
        xp = torch.zeros(c, t + n * (k - 1), device=x.device)
        xp[:, row + (seq + 1) * (k - 1)] = x[0].float()
        if state is not None:
            xp[:, (off[:-1, None] + s + j).reshape(-1)] = state.float().movedim(0, 1).reshape(c, -1)
        last = xp[:, off[1:, None] + s + j].movedim(0, 1)
        win = xp.unfold(1, k, 1)[None, :, row + seq * (k - 1)]
    p = (win * w.float()[None, :, None]).sum(3)
    if b is not None:
        p = p + b.float()[None, :, None]
    y = _silu(p) if act == "silu" else p
    if gy is None:
        return {"y": y.to(dt), "state": last.to(dt)}
    gp = gy.float() * (_silu_slope(p) if act == "silu" else 1)
    gpp = torch.nn.functional.pad(gp, (0, k - 1))
    dx = (gpp.unfold(2, k, 1) * w.float().flip(1)[None, :, None]).sum(3)
    dw = (win * gp[..., None]).sum((0, 2))
    out = {"y": y.to(dt), "dx": dx.to(dt), "dw": dw.to(dt)}
    if b is not None:
        out["db"] = gp.sum((0, 2)).to(dt)
    return out


def _scan(a, h, span):
    """h[t] += a[t] h[t-1] along dim 1, by doubling: log2(span) passes over whole tensors."""
    d = 1
    while d < span:
        h = torch.cat([h[:, :d], torch.addcmul(h[:, d:], a[:, d:], h[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return h


def _per_channel(v, c):
    """[N, G, S, L] of groups -> [N, L, C, S]."""
    return v.float().permute(0, 3, 1, 2).repeat_interleave(c // v.shape[1], 2)


def _plain_scan(s, gy=None):
    x, dt = s["x"], s["x"].dtype
    n, c, l = x.shape
    offsets, span = s["offsets"], s["max_len"] or l
    rows = lambda v: v.float().movedim(2, 1)[..., None]  # noqa: E731  [N, L, C, 1]
    xs, z = rows(x), rows(s["z"])
    raw = rows(s["dt"]) + s["dt_bias"][:, None]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    A, B, C = s["A"], _per_channel(s["B"], c), _per_channel(s["C"], c)
    a = torch.exp(delta * A)
    u = delta * xs * B
    first = torch.zeros(n, dtype=torch.long, device=x.device) if offsets is None else offsets.long()[:-1]
    if offsets is None:
        if s["state"] is not None:
            u[:, 0] += a[:, 0] * s["state"]
        h = _scan(a, u, span)
        last = h[:, -1]
    else:
        full = offsets.long().diff() > 0
        start = s["state"] if s["state"] is not None else torch.zeros(full.numel(), c, A.shape[1], device=x.device)
        at = first[full]
        u[0, at] += a[0, at] * start[full]
        cut = a.clone()
        cut[0, at] = 0
        h = _scan(cut, u, span)
        last = torch.where(full[:, None, None], h[0, (offsets.long()[1:] - 1).clamp(min=0)], start)
    y = (h * C).sum(3) + s["D"] * xs[..., 0]
    gate = _silu(z[..., 0])
    out = {"y": (y * gate).movedim(1, 2).to(dt)}
    if gy is None:
        return dict(out, state=last)
    g = rows(gy)[..., 0]
    sy = g * gate
    dh = C * sy[..., None]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    dh = _scan(after.flip(1), dh.flip(1), l).flip(1)
    del after
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1) * a  # a[t] h[t-1]
    del a
    fold = lambda v: v.reshape(n, l, s["B"].shape[1], -1, A.shape[1]).sum(3).permute(0, 2, 3, 1).to(dt)  # noqa: E731
    out["dC"] = fold(h * sy[..., None])
    del h
    du = (dh * B).sum(3)
    out["dB"] = fold(dh * (delta * xs))
    dh *= before
    del before
    ddelta = (dh * A).sum(3) + du * xs[..., 0]
    draw_ = ddelta * torch.sigmoid(raw[..., 0])
    back = lambda v: v.movedim(1, 2).to(dt)  # noqa: E731
    out["dx"] = back(du * delta[..., 0] + s["D"] * sy)
    out["ddt"] = back(draw_)
    out["dz"] = back(g * y * _silu_slope(z[..., 0]))
    out["dA"] = (dh * delta).sum((0, 1))
    out["dD"] = (sy * xs[..., 0]).sum((0, 1))
    out["ddt_bias"] = draw_.sum((0, 1))
    return out


def _plain_conv_token(s):
    x, st = s["x"], s["state"]
    win = torch.cat([st.float(), x.float()[..., None]], 2)
    p = (win * s["w"].float()).sum(2)
    if s["b"] is not None:
        p = p + s["b"].float()
    st.copy_(win[..., 1:])
    return {"y": (_silu(p) if s["case"]["act"] == "silu" else p).to(x.dtype), "state": st}


def _plain_scan_token(s):
    x, st = s["x"].float(), s["state"]
    raw = s["dt"].float() + s["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    per = x.shape[1] // s["B"].shape[1]
    B, C = s["B"].float().repeat_interleave(per, 1), s["C"].float().repeat_interleave(per, 1)
    st.copy_(torch.exp(delta[..., None] * s["A"]) * st + (delta * x)[..., None] * B)
    y = (st * C).sum(2) + s["D"] * x
    return {"y": (y * _silu(s["z"].float())).to(s["x"].dtype), "state": st}


def _plain_mv4(s):
    case, q = s["case"], s["packed"]
    w = torch.stack([q & 15, q >> 4], 2).reshape(case["n"], -1, case["group"]).float()
    w = w - (8 if s["zeros"] is None else s["zeros"].float()[..., None])
    w = (w * s["scales"].float()[..., None]).reshape(case["n"], -1)
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


# --------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "mv4":
            return _plain_mv4(s)
        if op == "conv_token":
            return _plain_conv_token(s)
        if op == "scan_token":
            return _plain_scan_token(s)
        if op.startswith("conv"):
            return _plain_conv(s["x"], s["w"], s["b"], case["act"], s["state"], s["offsets"], s.get("gy"))
        return _plain_scan(s, s.get("gy"))

    if op == "mv4":
        return s["plan"].run(s["x"], s["packed"], s["scales"], s["zeros"], s["bias"])
    if op == "conv_token":
        return {"y": s["plan"].run(s["x"], s["w"], s["b"], s["state"]), "state": s["state"]}
    if op == "scan_token":
        y = s["plan"].run(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        return {"y": y, "state": s["state"]}
    from depthwise_stencil_implicit_amd import lm
    if op == "conv":
        r = lm.causal_conv(s["x"], s["w"], s["b"], activation=case["act"], state=s["state"], offsets=s["offsets"],
                           max_len=s["max_len"], return_state=True)
        return {"y": r.y, "state": r.state}
    if op == "conv_train":
        y = lm.causal_conv(s["x"], s["w"], s["b"], activation=case["act"]).y
        r = lm.causal_conv_backward(s["gy"], s["x"], s["w"], s["b"], activation=case["act"])
        out = {"y": y, "dx": r.dx, "dw": r.dw}
        return dict(out, db=r.db) if s["b"] is not None else out
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if op == "scan":
        r = lm.selective_scan(*args, **kw, state=s["state"], offsets=s["offsets"], max_len=s["max_len"], return_state=True)
        return {"y": r.y, "state": r.state}
    f = lm.selective_scan(*args, **kw, save=True)
    r = lm.selective_scan_backward(s["gy"], *args, **kw, saved=f.saved)
    return {"y": f.y, "dx": r.dx, "ddt": r.ddt, "dA": r.dA, "dB": r.dB, "dC": r.dC, "dD": r.dD, "dz": r.dz,
            "ddt_bias": r.ddt_bias}


# ------------------------------------------------------- definition, 64 bits --

def _segments(s):
    """(row of the tensors, first, end, state's index) of each sequence."""
    case = s["case"]
    if s["offsets"] is None:
        return [(i, 0, case["l"], i) for i in range(case["n"])]
    off = s["offsets"].tolist()
    return [(0, off[i], off[i + 1], i) for i in range(case["n"])]


def _exact_conv(s):
    case = s["case"]
    k = case["k"]
    x, w = s["x"].double(), s["w"].double()
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dw, db = torch.zeros_like(w), torch.zeros(case["c"], dtype=torch.float64, device=x.device)
    last = torch.zeros((case["n"], case["c"], k - 1), dtype=torch.float64, device=x.device)
    for r, lo, hi, i in _segments(s):
        m = hi - lo
        ext = torch.zeros(case["c"], m + k - 1, dtype=torch.float64, device=x.device)
        if s["state"] is not None:
            ext[:, : k - 1] = s["state"][i].double()
        ext[:, k - 1:] = x[r, :, lo:hi]
        last[i] = ext[:, m:]
        pre = torch.zeros(case["c"], m, dtype=torch.float64, device=x.device)
        if s["b"] is not None:
            pre += s["b"].double()[:, None]
        for j in range(k):
            pre += w[:, j: j + 1] * ext[:, j: j + m]
        sig = 1 / (1 + torch.exp(-pre))
        y[r, :, lo:hi] = pre * sig if case["act"] == "silu" else pre
        if "gy" in s:
            gp = s["gy"][r, :, lo:hi].double()
            if case["act"] == "silu":
                gp = gp * (sig + pre * sig * (1 - sig))
            gext = torch.zeros_like(ext)
            for j in range(k):
                gext[:, j: j + m] += w[:, j: j + 1] * gp
                dw[:, j] += (gp * ext[:, j: j + m]).sum(1)
            dx[r, :, lo:hi] = gext[:, k - 1:]
            db += gp.sum(1)
    if "gy" not in s:
        return {"y": y, "state": last}
    out = {"y": y, "dx": dx, "dw": dw}
    return dict(out, db=db) if s["b"] is not None else out


def _exact_scan(s):
    """Token by token; every batch row at once, or the packed sequences one after the other."""
    x = s["x"].double()
    n, c, l = x.shape
    A, D = s["A"].double(), s["D"].double()
    per = c // s["B"].shape[1]
    raw = s["dt"].double() + s["dt_bias"].double()[:, None]
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw)))
    z, g = s["z"].double(), s["gy"].double() if "gy" in s else None
    sig = 1 / (1 + torch.exp(-z))
    state = s["state"].double() if s["state"] is not None else torch.zeros((s["case"]["n"], c, A.shape[1]), dtype=torch.float64, device=x.device)
    at = lambda v, t: v[..., t].double().repeat_interleave(per, 1)  # noqa: E731
    if s["offsets"] is None:
        h = state
        hs = [h]
        y = torch.empty_like(x)
        for t in range(l):
            d = delta[..., t, None]
            h = torch.exp(d * A) * h + d * x[..., t, None] * at(s["B"], t)
            y[..., t] = (h * at(s["C"], t)).sum(2) + D * x[..., t]
            if g is not None:
                hs.append(h)
        last = h
    else:
        y, last = torch.empty_like(x), state.clone()
        for r, lo, hi, i in _segments(s):
            h = state[i: i + 1]
            for t in range(lo, hi):
                d = delta[..., t, None]
                h = torch.exp(d * A) * h + d * x[..., t, None] * at(s["B"], t)
                y[..., t] = (h * at(s["C"], t)).sum(2) + D * x[..., t]
            last[i] = h[0]
    out = {"y": y * z * sig}
    if g is None:
        return dict(out, state=last)
    sy = g * z * sig
    dx, ddelta = torch.empty_like(x), torch.empty_like(x)
    dB = torch.empty(s["B"].shape, dtype=torch.float64, device=x.device)
    dC = torch.empty_like(dB)
    dA = torch.zeros_like(A)
    dh = torch.zeros_like(hs[0])
    sums = lambda v: v.reshape(n, -1, per, A.shape[1]).sum(2)  # noqa: E731
    for t in reversed(range(l)):
        d, v, B = delta[..., t, None], x[..., t, None], at(s["B"], t)
        dh = dh + sy[..., t, None] * at(s["C"], t)
        a = torch.exp(d * A)
        dC[..., t] = sums(sy[..., t, None] * hs[t + 1])
        dB[..., t] = sums(dh * d * v)
        dx[..., t] = (dh * B * d).sum(2) + D * sy[..., t]
        ga = dh * hs[t] * a
        ddelta[..., t] = (ga * A + dh * B * v).sum(2)
        dA += (ga * d).sum(0)
        dh = dh * a
    ddt = ddelta / (1 + torch.exp(-raw))
    return dict(out, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(sy * x).sum((0, 2)),
                dz=g * y * (sig + z * sig * (1 - sig)), ddt_bias=ddt.sum((0, 2)))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mv4":
        q = s["packed"].long()
        w = torch.empty(case["n"], case["k"], dtype=torch.float64, device=q.device)
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
        grp = torch.arange(case["k"], device=q.device) // case["group"]
        w -= 8 if s["zeros"] is None else s["zeros"].double()[:, grp]
        w *= s["scales"].double()[:, grp]
        y = s["x"].double() @ w.T
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "conv_token":
        ext = torch.cat([s["state"], s["x"][..., None]], 2).double()
        pre = torch.einsum("nck,ck->nc", ext, s["w"].double())
        if s["b"] is not None:
            pre = pre + s["b"].double()
        y = pre / (1 + torch.exp(-pre)) if case["act"] == "silu" else pre
        return {"y": y, "state": ext[..., 1:]}
    if op == "scan_token":
        s = {k: v[..., None] if k in ("x", "z", "dt", "B", "C") else v for k, v in s.items() if k != "plan"}
        s["offsets"], s["case"] = None, dict(case, l=1)
        r = _exact_scan(s)
        return {"y": r["y"][..., 0], "state": r["state"]}
    return _exact_conv(s) if op.startswith("conv") else _exact_scan(s)
