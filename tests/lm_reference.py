"""The sequence operators in 64 bits, written from their formulas position by
position (torch on the CPU), and the bounds their f32 kernels are held to.

Every reference can be run a second time with ``bound=True``: the same sums
over the absolute values of their terms.  A kernel's result may differ from the
reference by

    u * |result|  +  n * 2^-24 * (sum of absolute terms)  +  tiny,

u the half spacing of the output type, n the number of f32 roundings a term
can pass through: its own products and exponentials (64 allows for the
arguments of exp and log, whose rounding grows with their size, up to 20 here),
one or two per addition of a sum, and four per step of a recurrence.
"""
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def assert_close(got, ref, bound, n, what=""):
    """got within u |ref| + n 2^-24 bound of ref, NaN and infinities equal."""
    g = f64(got)
    assert tuple(g.shape) == tuple(ref.shape), (what, g.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities differ"
    err = (g - ref).abs()
    tol = U[got.dtype] * 1.01 * ref.abs() + n * 2.0 ** -24 * bound + TINY[got.dtype]
    bad = fine & ~(err <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got {g[i]:.9g}, reference "
                             f"{ref[i]:.9g}, allowed {tol[i]:.3g}; largest error / allowed {(err / tol)[fine].max():.3g}")


def spans(x, offsets):
    """(row of x, first, end) of each sequence."""
    if offsets is None:
        return [(i, 0, x.shape[2]) for i in range(x.shape[0])]
    o = offsets.cpu().tolist()
    return [(0, o[i], o[i + 1]) for i in range(len(o) - 1)]


def sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def conv(x, w, b=None, act=None, state=None, offsets=None, gy=None, gstate=None, bound=False):
    """(y, state) or, with gy, (dx, dw, db, dstate) of the causal convolution."""
    x, w, b, state, gy, gstate = map(f64, (x, w, b, state, gy, gstate))
    C, K = w.shape
    segs = spans(x, offsets)
    y, last = torch.zeros_like(x), torch.zeros(len(segs), C, K - 1, dtype=torch.float64)
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(C, dtype=torch.float64)
    ds = torch.zeros_like(last)
    ab = (lambda v: v.abs()) if bound else (lambda v: v)
    for i, (r, lo, hi) in enumerate(segs):
        n = hi - lo
        xx = torch.zeros(C, n + K - 1, dtype=torch.float64)
        if state is not None:
            xx[:, : K - 1] = state[i]
        xx[:, K - 1:] = x[r, :, lo:hi]
        last[i] = xx[:, n:]
        gg = torch.zeros_like(xx)
        if gstate is not None:
            gg[:, n:] += ab(gstate[i])
        for t in range(n):
            p = (w * xx[:, t:t + K]).sum(1) + (b if b is not None else 0)
            pa = (w * xx[:, t:t + K]).abs().sum(1) + (b.abs() if b is not None else 0)
            q = sigmoid(p)
            # With |act'| <= 1.1 an error of p reaches y and act' at most 1.1 times.
            y[r, :, lo + t] = (1.1 * pa if bound else p * q) if act else (pa if bound else p)
            if gy is not None:
                g = ab(gy[r, :, lo + t])
                if act:
                    g = g * (1.1 + pa) if bound else g * (q * (1 + p * (1 - q)))
                gg[:, t:t + K] += g[:, None] * ab(w)
                dw += g[:, None] * ab(xx[:, t:t + K])
                db += g
        dx[r, :, lo:hi] = gg[:, K - 1:]
        ds[i] = gg[:, : K - 1]
    return (y, last) if gy is None else (dx, dw, db, ds)


def softplus(v):
    return torch.where(v > 40, v, torch.log1p(torch.exp(v.clamp(max=40))))


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus_dt=False, state=None, offsets=None, gy=None, gstate=None,
         bound=False):
    """dict of y and state or, with gy, of the gradients of the selective scan."""
    x, dt, A, B, C, D, z, dt_bias, state, gy, gstate = map(f64, (x, dt, A, B, C, D, z, dt_bias, state, gy, gstate))
    N, Ch, L = x.shape
    S, G = A.shape[1], B.shape[1]
    segs = spans(x, offsets)
    ab = (lambda v: v.abs()) if bound else (lambda v: v)
    raw = dt + (dt_bias[:, None] if dt_bias is not None else 0)
    d = softplus(raw) if softplus_dt else raw
    gate, slope = torch.ones_like(x), torch.zeros_like(x)
    if z is not None:
        q = sigmoid(z)
        gate, slope = z * q, q * (1 + z * (1 - q))
    per = Ch // G
    at = lambda v, r, t: v[r, :, :, t].repeat_interleave(per, 0)  # noqa: E731
    o = {"y": torch.zeros_like(x), "state": torch.zeros(len(segs), Ch, S, dtype=torch.float64)}
    g = {k: torch.zeros_like(v) for k, v in (("dx", x), ("ddt", x), ("dz", x), ("dA", A), ("dB", B), ("dC", C))}
    g |= {"dD": torch.zeros(Ch, dtype=torch.float64), "ddt_bias": torch.zeros(Ch, dtype=torch.float64),
          "dstate": torch.zeros_like(o["state"])}
    Dv = D if D is not None else torch.zeros(Ch, dtype=torch.float64)
    for i, (r, lo, hi) in enumerate(segs):
        h = ab(state[i]) if state is not None else torch.zeros(Ch, S, dtype=torch.float64)
        hs = [h]
        for t in range(lo, hi):
            dd, v = d[r, :, t], x[r, :, t]
            h = torch.exp(dd[:, None] * A) * h + ab((dd * v)[:, None] * at(B, r, t))
            hs.append(h)
            y = (ab(at(C, r, t)) * h).sum(1) + ab(Dv * v)
            o["y"][r, :, t] = y * ab(gate[r, :, t])
            if gy is not None:
                g["dz"][r, :, t] = ab(gy[r, :, t]) * y * (1.1 + z[r, :, t].abs() if bound else slope[r, :, t]) if z is not None else 0
        o["state"][i] = h
        if gy is None:
            continue
        rr = ab(gstate[i]) if gstate is not None else torch.zeros(Ch, S, dtype=torch.float64)
        for t in reversed(range(lo, hi)):
            dd, v, b, c = d[r, :, t], ab(x[r, :, t]), ab(at(B, r, t)), ab(at(C, r, t))
            s = ab(gy[r, :, t] * gate[r, :, t])
            if bound:
                dd_f = dd.abs()
            else:
                dd_f = dd
            rr = rr + s[:, None] * c
            a = torch.exp(dd[:, None] * A)
            k = t - lo
            g["dC"][r, :, :, t] = (s[:, None] * hs[k + 1]).reshape(G, per, S).sum(1)
            g["dB"][r, :, :, t] = (rr * (dd_f * v)[:, None]).reshape(G, per, S).sum(1)
            rb = (rr * b).sum(1)
            g["dx"][r, :, t] = dd_f * rb + ab(Dv) * s
            w = rr * a * hs[k]
            gd = (w * ab(A)).sum(1) + v * rb
            if softplus_dt:
                gd = gd * sigmoid(raw[r, :, t])
            g["ddt"][r, :, t] = gd
            g["dA"] += w * dd_f[:, None]
            g["dD"] += s * v
            g["ddt_bias"] += gd
            rr = rr * a
        g["dstate"][i] = rr
    return o if gy is None else g


def matvec4(x, packed, scales, zeros=None, bias=None, bound=False):
    packed_excess = x.dtype == torch.bfloat16
    x, scales, zeros, bias = map(f64, (x, scales, zeros, bias))
    p = packed.cpu().long()
    n, k = p.shape[0], 2 * p.shape[1]
    q = torch.zeros(n, k, dtype=torch.float64)
    q[:, 0::2], q[:, 1::2] = (p & 15).double(), (p >> 4).double()
    per = k // scales.shape[1]
    zz = zeros.repeat_interleave(per, 1) if zeros is not None else torch.full_like(q, 8)
    s = scales.repeat_interleave(per, 1)
    if bound:  # bf16 rows: the kernel sums (128 + q) x and (128 + z) x apart; else (q - 8) x and (z - 8) x
        m = 288 if packed_excess else 24
        return x.abs() @ ((m + zz.abs()) * s.abs()).T + (bias.abs() if bias is not None else 0)
    y = x @ (s * (q - zz)).T
    return y + bias if bias is not None else y
