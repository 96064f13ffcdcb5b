"""The gated recurrence, the RMS norm and the adapters in 64 bits, from their
formulas (torch on the CPU), and the sums over absolute terms that their f32
kernels' bounds count in (lm_reference.py says how).

Roundings that a term passes, in units of 2^-24.  Recurrence: the factor a of
one step is off by 1 to 2 units from its exponential and by |log2 a| ln 2 times
what its exponent is off by, about 20 units (the softplus, the sigmoid with
gates up to 6, three products), so 24 per step for |log2 a| up to 1.5, with the
step's own multiply-add; sqrt(1 - a^2) by 32 where 1 - a^2 is 1/16 and less on
both sides.  Norm: a thread adds up to 64 squares, 10 levels join them, and the
root, its reciprocal and three products follow.  Adapters: one per term of
either sum."""
import torch

from lm_reference import f64, sigmoid, softplus, spans

F8 = torch.float8_e4m3fn


def gated(x, r, i, decay, sharpness=8.0, state=None, offsets=None, gy=None, gstate=None, bound=False):
    """dict of y and state or, with gy, of the gradients."""
    x, r, i, decay, state, gy, gstate = map(f64, (x, r, i, decay, state, gy, gstate))
    ab = (lambda v: v.abs()) if bound else (lambda v: v)
    C = x.shape[1]
    segs = spans(x, offsets)
    k = (sharpness * softplus(decay))[:, None]
    rho, iota = sigmoid(r), sigmoid(i)
    a, comp = torch.exp(-k * rho), -torch.expm1(-2 * k * rho)
    m = comp.sqrt()
    over = torch.where(m > 0, a * a / m, 0.0)      # the limit counts where nothing is left to divide by
    u = ab(m * iota * x)
    o = {"y": torch.zeros_like(x), "state": torch.zeros(len(segs), C, dtype=torch.float64)}
    g = {n: torch.zeros_like(x) for n in ("dx", "dr", "di")}
    g |= {"ddecay": torch.zeros(C, dtype=torch.float64), "dstate": torch.zeros_like(o["state"])}
    for s, (b, lo, hi) in enumerate(segs):
        h = ab(state[s]) if state is not None else torch.zeros(C, dtype=torch.float64)
        before = []
        for t in range(lo, hi):
            before.append(h)
            h = a[b, :, t] * h + u[b, :, t]
            o["y"][b, :, t] = h
        o["state"][s] = h
        if gy is None:
            continue
        q = ab(gstate[s]) if gstate is not None else torch.zeros(C, dtype=torch.float64)
        for t in reversed(range(lo, hi)):
            at = lambda v: v[b, :, t]  # noqa: E731
            gh = ab(at(gy)) + q
            g["dx"][b, :, t] = gh * at(m) * at(iota)
            g["di"][b, :, t] = gh * at(m) * ab(at(x)) * at(iota) * (1 - at(iota))
            second = at(iota) * ab(at(x)) * at(over)
            dl = gh * (at(a) * before[t - lo] + (second if bound else -second))
            g["dr"][b, :, t] = (k[:, 0] if bound else -k[:, 0]) * dl * at(rho) * (1 - at(rho))
            g["ddecay"] += dl * at(rho)
            q = at(a) * gh
        g["dstate"][s] = q
    if gy is None:
        return o
    g["ddecay"] *= (sharpness if bound else -sharpness) * sigmoid(decay)
    return g


def norm(x, w, residual=None, eps=1e-6):
    """(y, v, rstd) with channels in dim 1."""
    v = f64(x) + (f64(residual) if residual is not None else 0)
    rstd = 1 / torch.sqrt((v * v).mean(1) + eps)
    shape = (-1,) + (1,) * (v.dim() - 2)
    return v * rstd.unsqueeze(1) * f64(w).view(shape), v, rstd


def norm_backward(gy, v, w, rstd, gresidual=None):
    """((dx, dw), their bounds)."""
    gy, v, w, rstd = f64(gy), f64(v), f64(w), f64(rstd).unsqueeze(1)
    u, wg = v * rstd, gy * w.view((-1,) + (1,) * (v.dim() - 2))
    gs = f64(gresidual) if gresidual is not None else torch.zeros_like(v)
    rest = [d for d in range(v.dim()) if d != 1]
    dx = gs + rstd * (wg - u * (wg * u).mean(1, keepdim=True))
    bx = gs.abs() + rstd * (wg.abs() + u.abs() * (wg * u).abs().mean(1, keepdim=True))
    return (dx, (gy * u).sum(rest)), (bx, (gy * u).abs().sum(rest))


def check_f8(q, scales, y, what="", units=128):
    """q (e4m3) times scales against y, channels in dim 1: each scale is its
    group's largest |y| / 448 and each value within half a step (2^-4 of itself,
    2^-10 below 2^-6) of y / scale, whose f32 steps are `units`."""
    G = scales.shape[1]
    s, v = f64(scales), f64(q)
    top = y.abs().unflatten(1, (G, -1)).amax(2)
    want = torch.where(top == 0, 448.0, top) / 448
    assert bool(((s - want).abs() <= units * 2.0 ** -24 * want).all()), f"{what}: scales"
    ideal = y / want.repeat_interleave(y.shape[1] // G, 1)
    allowed = (2.0 ** -4 + units * 2.0 ** -24) * ideal.abs() + 2.0 ** -10
    bad = (v - ideal).abs() > allowed
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values outside"


def adapters(x, a, b, index, base=None, scaling=None, x_scales=None):
    """(y, bound) of rows [M, K] or [N, K, L]."""
    rows = (lambda v: v) if x.dim() == 2 else (lambda v: v.movedim(1, 2).flatten(0, 1))
    xr = rows(x.float() if x.dtype == F8 else x)
    xr, a, b = f64(xr), f64(a), f64(b)
    if x_scales is not None:
        xr = xr * f64(rows(x_scales))
    y = f64(rows(base)).clone() if base is not None else torch.zeros(xr.shape[0], b.shape[1], dtype=torch.float64)
    bound = y.abs()
    for m, e in enumerate(index.cpu().flatten().tolist()):
        if 0 <= e < a.shape[0]:
            s = float(scaling[e]) if scaling is not None else 1.0
            y[m] += s * (b[e] @ (a[e] @ xr[m]))
            bound[m] += abs(s) * (b[e].abs() @ (a[e].abs() @ xr[m].abs()))
    if x.dim() == 3:
        y, bound = (v.unflatten(0, (x.shape[0], x.shape[2])).movedim(2, 1) for v in (y, bound))
    return y, bound
