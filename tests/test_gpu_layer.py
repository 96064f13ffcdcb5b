"""The gated recurrence, the RMS norm and the adapters on the GPU against the
64-bit reference: types, layouts, odd sizes, lengths from zero, packed
sequences, chunked axes, states, gradients, single tokens."""
import pytest
import torch

import layer_reference as Y
import lm_reference as R
from depthwise_stencil_implicit_amd import lm
from test_gpu_lm import gen, offsets_of, rnd, to_layout

pytestmark = pytest.mark.gpu

BF, HF, F, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------- recurrence --

GATED = [
    # dtype, N, C, L, state, layout, lens (packed), chunk
    (F, 2, 16, 40, False, "nlc", None, None),
    (BF, 1, 64, 130, True, "nlc", None, 128),
    (BF, 2, 130, 300, True, "nlc", None, 128),
    (HF, 3, 17, 1, True, "nlc", None, None),
    (F, 2, 65, 257, True, "nlc", None, 128),
    (BF, 1, 1, 70, True, "nlc", None, None),
    (HF, 2, 2, 129, False, "nlc", None, None),
    (F, 1, 1, 7, False, "nlc", None, None),
    (BF, 2, 40, 150, True, "ncl", None, 128),
    (HF, 2, 41, 150, True, "wide", None, 128),
    (F, 2, 24, 140, True, "every", None, 128),
    (BF, 1, 72, 700, True, "nlc", [0, 1, 2, 128, 0, 129, 440, 0], 128),
    (F, 1, 70, 501, True, "wide", [133, 0, 331, 37], None),
    (HF, 1, 9, 64, False, "nlc", [64], 128),
    (BF, 2, 16, 0, True, "nlc", None, None),
    (BF, 1, 16, 0, True, "nlc", [0, 0], None),
]


def gated_case(i):
    dt, N, C, L, st, layout, lens, chunk = GATED[i]
    g = gen(900 + i)
    n = len(lens) if lens else N
    lay = lambda scale: to_layout(rnd(g, N, C, L, dtype=dt, scale=scale), layout)  # noqa: E731
    args = (lay(1.0), lay(1.5), lay(1.5), (rnd(g, C, scale=1.5) - 4).cuda())
    off = offsets_of(lens).cuda() if lens else None
    kw = dict(sharpness=(8.0, 1.0, 3.5)[i % 3], state=rnd(g, n, C).cuda() if st else None, offsets=off)
    return args, kw, dict(max_len=max(lens) // 2 if lens else None, chunk=chunk), g, n


def steps_of(i):
    return 24 * GATED[i][3] + 192


@pytest.mark.parametrize("i", range(len(GATED)))
def test_gated_recurrence(i):
    args, kw, split, _, _ = gated_case(i)
    print(f"gated {GATED[i]}", flush=True)
    got = lm.gated_recurrence(*args, **kw, **split, return_state=True)
    o, b = Y.gated(*args, **kw), Y.gated(*args, **kw, bound=True)
    R.assert_close(got.state, o["state"], b["state"], steps_of(i), "state")
    R.assert_close(got.y, o["y"], b["y"], steps_of(i), "y")


@pytest.mark.parametrize("i", range(len(GATED)))
def test_gated_recurrence_backward(i):
    args, kw, split, g, n = gated_case(i)
    dt, N, C, L, layout = (GATED[i][k] for k in (0, 1, 2, 3, 5))
    gy = to_layout(rnd(g, N, C, L, dtype=dt), layout)
    gs = rnd(g, n, C).cuda() if i % 2 else None
    print(f"gated backward {GATED[i]}", flush=True)
    saved = lm.gated_recurrence(*args, **kw, **split, save=True).saved if i % 3 else None
    got = lm.gated_recurrence_backward(gy, *args, **kw, **split, gstate=gs, saved=saved)
    o, b = (Y.gated(*args, **kw, gy=gy, gstate=gs, bound=k) for k in (False, True))
    for k in ("dx", "dr", "di", "ddecay", "dstate"):
        v = getattr(got, k)
        if v is not None:
            R.assert_close(v, o[k], b[k], 2 * steps_of(i) + (N * L if k == "ddecay" else 0), k)
    assert (got.dstate is None) == (kw["state"] is None)


def test_gated_gradients_against_differences():
    """d<y, gy> + d<state, gstate> along random directions, by central
    differences of the 64-bit formula."""
    g = gen(9)
    N, C, L = 2, 5, 12
    v = dict(x=rnd(g, N, C, L), r=rnd(g, N, C, L), i=rnd(g, N, C, L), decay=rnd(g, C) - 3, state=rnd(g, N, C))
    gy, gs = rnd(g, N, C, L), rnd(g, N, C)
    c = {k: t.cuda() for k, t in v.items()}
    got = lm.gated_recurrence_backward(gy.cuda(), c["x"], c["r"], c["i"], c["decay"], state=c["state"], gstate=gs.cuda())
    grads = dict(x=got.dx, r=got.dr, i=got.di, decay=got.ddecay, state=got.dstate)

    def value(w):
        o = Y.gated(w["x"], w["r"], w["i"], w["decay"], state=w["state"])
        return float((o["y"] * gy.double()).sum() + (o["state"] * gs.double()).sum())

    for k in v:
        d = torch.randn(v[k].shape, generator=g).double()
        e = 1e-5
        up, down = ({**{n: t.double() for n, t in v.items()}, k: v[k].double() + s * e * d} for s in (1, -1))
        diff, terms = (value(up) - value(down)) / (2 * e), grads[k].cpu().double() * d
        # Differences of order e^2; f32 gradients of at most a few hundred terms.
        assert abs(diff - float(terms.sum())) <= 1e-4 * (1 + float(terms.abs().sum())), (k, diff, float(terms.sum()))


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("C", [1, 6, 7, 64, 130])
def test_gated_step_continues_the_prompt(dt, C):
    g = gen(C)
    N, L = 3, 6
    x, r, i = (to_layout(rnd(g, N, C, L, dtype=dt), "nlc") for _ in range(3))
    decay = (rnd(g, C) - 4).cuda()
    whole = lm.gated_recurrence(x, r, i, decay, return_state=True)
    first = lm.gated_recurrence(x[:, :, :2], r[:, :, :2], i[:, :, :2], decay, return_state=True)
    table = torch.full((5, C), 3.0, device="cuda")
    rows = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    table[rows.long()] = first.state
    for t in range(2, L):
        y = lm.gated_recurrence_step(x[:, :, t], r[:, :, t], i[:, :, t], decay, table, rows=rows)
        one = Y.gated(x[:, :, :t + 1], r[:, :, :t + 1], i[:, :, :t + 1], decay)["y"][:, :, t]
        R.assert_close(y, one, Y.gated(x[:, :, :t + 1], r[:, :, :t + 1], i[:, :, :t + 1], decay, bound=True)["y"][:, :, t], 24 * L + 192, "step")
    R.assert_close(table[rows.long()], f64 := whole.state.double().cpu(), f64.abs() + 1, 48 * L + 384, "state")
    assert bool((table[[1, 3]] == 3).all())
    out = torch.tensor([-1, 0, 9], dtype=torch.int32, device="cuda")
    before = table.clone()
    y = lm.gated_recurrence_step(x[:, :, 0], r[:, :, 0], i[:, :, 0], decay, table, rows=out)
    assert bool((y[[0, 2]] == 0).all()) and torch.equal(table[1:], before[1:])


@pytest.mark.parametrize("dt", [BF, F])
def test_gated_limits(dt):
    """Closed and open gates, rates of nothing and of everything: the state
    stays, goes, or takes the input as it is; gradients stay finite."""
    N, C, L = 1, 8, 140
    g = gen(3)
    x, r, i, gy = (to_layout(rnd(g, N, C, L, dtype=dt), "nlc") for _ in range(4))
    decay = torch.full((C,), -3.0, device="cuda")
    low = torch.finfo(dt).min
    r[:, 0], r[:, 1], i[:, 2], i[:, 3], r[:, 6] = -torch.inf, low, -torch.inf, torch.inf, 40.0
    decay[4], decay[5] = -torch.inf, 60.0
    st = rnd(g, N, C).cuda()
    got = lm.gated_recurrence(x, r, i, decay, state=st, return_state=True)
    assert torch.equal(got.state[:, [0, 1, 4]], st[:, [0, 1, 4]])   # a is 1, nothing comes in
    o, b = (Y.gated(x, r, i, decay, state=st, bound=k) for k in (False, True))
    R.assert_close(got.y, o["y"], b["y"], 40 * L + 192, "y")
    back = lm.gated_recurrence_backward(gy, x, r, i, decay, state=st)
    o, b = (Y.gated(x, r, i, decay, state=st, gy=gy, bound=k) for k in (False, True))
    for k in ("dx", "dr", "di", "dstate"):
        R.assert_close(getattr(back, k), o[k], b[k], 80 * L + 384, k)
    R.assert_close(back.ddecay, o["ddecay"], b["ddecay"], 81 * L + 384, "ddecay")
    x[:, 7, 130] = torch.nan   # stays in its channel, from its step on
    y = lm.gated_recurrence(x, r, i, decay, state=st).y
    assert bool(torch.isnan(y[:, 7, 130:]).all()) and not bool(torch.isnan(y[:, 7, :130]).any()) and not bool(torch.isnan(y[:, :7]).any())


def test_gated_far_rows():
    """Rows further apart than 32 bits of elements reach."""
    g = gen(4)
    C, L, step = 6, 20, 2 ** 28
    big = torch.empty(step * L, dtype=BF, device="cuda")
    far = big.as_strided((1, C, L), (step * L, 1, step))
    x, r, i, gy = (to_layout(rnd(g, 1, C, L, dtype=BF), "nlc") for _ in range(4))
    decay = (rnd(g, C) - 4).cuda()
    want = lm.gated_recurrence(x, r, i, decay).y
    back = lm.gated_recurrence_backward(gy, x, r, i, decay)
    for k in range(3):
        args = [x, r, i]
        far.copy_(args[k])
        args[k] = far
        assert torch.equal(lm.gated_recurrence(*args, decay).y, want)
        saved = lm._new_gated_saved(x, None)
        lm._call(lm.A.LM_GATED, [(lm._X, args[0]), (lm._A, args[1]), (lm._B, args[2]), (lm._D, decay)], [(lm._SAVED, saved)], value=8.0)
        dx = torch.empty_like(x)
        rest = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(decay)]
        lm._call(lm.A.LM_GATED_BWD, [(lm._GY, gy), (lm._X, args[0]), (lm._A, args[1]), (lm._B, args[2]), (lm._D, decay), (lm._SAVED, saved)],
                 [(lm._DX, dx), (lm._DA, rest[0]), (lm._DB, rest[1]), (lm._DD, rest[2])], value=8.0)
        assert torch.equal(dx, back.dx) and torch.equal(rest[0], back.dr) and torch.equal(rest[2], back.ddecay)


# ------------------------------------------------------------------- norm --

NORM = [
    # dtype, N, C, L (0: rows [N, C]), residual, layout
    (BF, 5, 64, 0, True, "nlc"),
    (HF, 3, 1, 0, False, "nlc"),
    (F, 2, 7, 0, True, "nlc"),
    (BF, 1, 513, 0, True, "nlc"),
    (BF, 3, 4099, 0, True, "nlc"),
    (F, 2, 20000, 0, False, "nlc"),
    (HF, 1, 65536, 0, True, "nlc"),
    (BF, 2, 2056, 9, True, "nlc"),
    (HF, 2, 40, 33, True, "ncl"),
    (F, 2, 129, 5, True, "wide"),
    (BF, 2, 300, 7, False, "every"),
    (BF, 2100, 130, 0, True, "nlc"),
    (F, 2100, 2049, 0, True, "nlc"),
    (BF, 2050, 520, 0, False, "nlc"),
    (HF, 0, 64, 0, True, "nlc"),
]


def norm_case(i):
    dt, N, C, L, res, layout = NORM[i]
    g = gen(1200 + i)
    lay = lambda scale: to_layout(rnd(g, N, C, L or 1, dtype=dt, scale=scale), layout)  # noqa: E731
    v = [lay(1.0), lay(2.0) if res else None, lay(1.0), lay(1.0)]
    if not L:
        v = [t if t is None else t[:, :, 0] for t in v]
    return *v, (1 + 0.2 * rnd(g, C)).to(dt).cuda()


@pytest.mark.parametrize("i", range(len(NORM)))
def test_rms_norm(i):
    x, res, gy, gr, w = norm_case(i)
    print(f"norm {NORM[i]}", flush=True)
    got = lm.rms_norm(x, w, residual=res, eps=1e-5, save=True)
    y, v, rstd = Y.norm(x, w, res, 1e-5)
    R.assert_close(got.y, y, y.abs(), 128, "y")
    R.assert_close(got.rstd, rstd, rstd, 128, "rstd")
    if res is not None:
        R.assert_close(got.residual, v, f64_sum(x, res), 1, "residual")
    else:
        assert got.residual is None
    total = got.residual if res is not None else x
    back = lm.rms_norm_backward(gy, total, w, got.rstd, gresidual=gr if i % 2 else None)
    (dx, dw), (bx, bw) = Y.norm_backward(gy, total, w, got.rstd, gr if i % 2 else None)
    R.assert_close(back.dx, dx, bx, 160, "dx")
    R.assert_close(back.dw, dw, bw, NORM[i][1] * max(1, NORM[i][3]) + 160, "dw")
    only = lm.rms_norm_backward(gy, total, w, got.rstd, need_dx=False)
    assert only.dx is None and torch.equal(only.dw, back.dw)
    only = lm.rms_norm_backward(gy, total, w, got.rstd, gresidual=gr if i % 2 else None, need_dw=False)
    assert only.dw is None and torch.equal(only.dx, back.dx)


def f64_sum(x, res):
    return x.cpu().double().abs() + res.cpu().double().abs()


@pytest.mark.parametrize("i", range(len(NORM)))
@pytest.mark.parametrize("group", [None, 32, 64, 128])
def test_rms_norm_in_8_bits(i, group):
    x, res, _, _, w = norm_case(i)
    C = x.shape[1]
    if group and C % group:
        with pytest.raises(ValueError, match="groups of"):
            lm.rms_norm(x, w, residual=res, out_dtype=F8, group=group)
        return
    print(f"norm in 8 bits {NORM[i]} {group}", flush=True)
    if C > 2 and x.shape[0]:
        x[0, : min(C, group or C)] = 0   # a group of zeros, where there is no residual
    got = lm.rms_norm(x, w, residual=res, out_dtype=F8, group=group, save=True)
    y, v, rstd = Y.norm(x, w, res)
    assert got.y.dtype == F8 and got.scales.shape[:2] == (x.shape[0], C // group if group else 1)
    Y.check_f8(got.y.float(), got.scales, y)
    R.assert_close(got.rstd, rstd, rstd, 128, "rstd")
    plain = lm.rms_norm(x, w, residual=res)
    if res is not None:
        assert torch.equal(got.residual, plain.residual)


def test_rms_norm_of_extremes():
    """Rows of zeros, of tiny and of large values, of an infinity and of a NaN:
    each row by itself."""
    g = gen(5)
    x, w = rnd(g, 8, 256, dtype=F).cuda(), torch.ones(256, device="cuda")
    x[0], x[1], x[2], x[3, 7], x[4, 9] = 0, x[1] * 1e-30, x[2] * 1e18, torch.inf, torch.nan
    x[5] *= 1e-38
    for group in (None, 32):
        got = lm.rms_norm(x, w, eps=1e-6)
        y, _, _ = Y.norm(x, w)
        fine = [0, 1, 2, 5, 6, 7]
        R.assert_close(got.y[fine], y[fine], y[fine].abs(), 160, "y")
        assert bool(torch.isnan(got.y[4]).all()) and bool(torch.isnan(got.y[3, 7]))
        q = lm.rms_norm(x, w, eps=1e-6, out_dtype=F8, group=group)
        back = q.y.float() * q.scales.repeat_interleave(256 // q.scales.shape[1], 1)
        assert bool((back[0] == 0).all()) and bool((q.scales[0] == 1).all())
        assert bool(torch.isnan(back[4]).all()) and bool(torch.isfinite(back[fine]).all())
        # Half a step of e4m3 and, below 2^-6 of a scale, half its smallest step.
        lim = 2.0 ** -4 * y[fine].abs() * 1.001 + 2.0 ** -10 * q.scales[fine].cpu().double().repeat_interleave(256 // q.scales.shape[1], 1)
        assert bool(((back[fine].cpu().double() - y[fine]).abs() <= lim).all())


def test_norm_of_many_rows():
    """More rows than a launch of 1024 threads for each would hold."""
    rows, C = (1 << 22) + 5, 8
    x = torch.randn(rows, C, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(BF)
    w = torch.arange(1, 9, device="cuda").to(BF)
    got = lm.rms_norm(x, w, save=True)
    v = x.float()
    want = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.float()
    # One rounding to bf16, and f32's on both sides.
    assert bool(((got.y.float() - want).abs() <= (2 ** -8 + 2 ** -19) * want.abs()).all())
    back = lm.rms_norm_backward(x, x, w, got.rstd)
    u = v.double() * got.rstd.double()[:, None]
    dw = (v.double() * u).sum(0)
    assert bool(((back.dw.double() - dw).abs() <= 2 ** -7 * dw).all())
    assert torch.equal(back.dx[-3:], lm.rms_norm_backward(x[-3:], x[-3:], w, got.rstd[-3:]).dx)


def test_norm_gradients_against_differences():
    g = gen(6)
    x, w, gy, gr = rnd(g, 3, 10), rnd(g, 10), rnd(g, 3, 10), rnd(g, 3, 10)
    f = lm.rms_norm(x.cuda(), w.cuda(), residual=torch.zeros(3, 10, device="cuda"), eps=1e-3, save=True)
    got = lm.rms_norm_backward(gy.cuda(), f.residual, w.cuda(), f.rstd, gresidual=gr.cuda())

    def value(u):
        y, v, _ = Y.norm(u["x"], u["w"], eps=1e-3)
        return float((y * gy.double()).sum() + (v * gr.double()).sum())

    for k, grad in (("x", got.dx), ("w", got.dw)):
        base = dict(x=x.double(), w=w.double())
        d = torch.randn(base[k].shape, generator=g).double()
        diff = (value({**base, k: base[k] + 1e-5 * d}) - value({**base, k: base[k] - 1e-5 * d})) / 2e-5
        terms = grad.cpu().double() * d
        assert abs(diff - float(terms.sum())) <= 1e-4 * (1 + float(terms.abs().sum())), k


# --------------------------------------------------------------- adapters --

ADAPTERS = [
    # dtype, rows (M or (N, L)), K, N', R, E, index ("each" its own, "runs", "mixed", "none"), base, scaling, 8-bit x, layout
    (BF, 1, 64, 64, 16, 1, "each", True, True, False, "nlc"),
    (BF, 3, 256, 300, 8, 4, "mixed", True, True, False, "nlc"),
    (HF, 17, 1000, 129, 24, 5, "mixed", True, False, False, "nlc"),
    (F, 33, 96, 70, 16, 40, "each", False, True, False, "nlc"),
    (BF, 16, 31, 5, 4, 3, "mixed", True, True, False, "nlc"),
    (HF, 5, 1, 1, 1, 2, "each", True, True, False, "nlc"),
    (BF, 40, 520, 513, 64, 6, "none", True, True, False, "nlc"),
    (BF, 600, 264, 320, 32, 5, "runs", True, True, False, "nlc"),
    (HF, 515, 200, 260, 40, 3, "mixed", True, True, False, "nlc"),
    (F, 700, 130, 140, 16, 70, "mixed", True, False, False, "nlc"),
    (BF, 130, 320, 90, 256, 3, "mixed", True, True, False, "nlc"),
    (F, 520, 70, 66, 200, 2, "runs", True, True, False, "nlc"),
    (BF, 20, 384, 264, 16, 4, "mixed", True, True, True, "nlc"),
    (HF, 530, 333, 136, 72, 4, "runs", True, True, True, "nlc"),
    (F, 9, 100, 40, 12, 2, "mixed", False, False, True, "nlc"),
    (BF, (2, 9), 72, 80, 8, 3, "mixed", True, True, False, "nlc"),
    (HF, (3, 200), 136, 72, 16, 4, "runs", True, True, False, "nlc"),
    (BF, (2, 30), 64, 40, 8, 3, "mixed", True, True, False, "ncl"),
    (F, (2, 11), 50, 24, 6, 3, "mixed", True, True, False, "every"),
    (BF, (2, 11), 56, 25, 16, 3, "mixed", True, True, True, "wide"),
    (BF, 0, 64, 64, 8, 2, "each", True, True, False, "nlc"),
    (BF, 6, 0, 64, 8, 2, "each", True, True, False, "nlc"),
    (BF, 6, 64, 64, 8, 0, "none", True, False, False, "nlc"),
    (BF, 300, 2100, 1500, 16, 3, "mixed", True, True, False, "nlc"),
    (HF, (2, 250), 2304, 600, 40, 31, "mixed", True, True, True, "nlc"),
    (BF, 6, 64, 64, 8, 0, "none", False, False, False, "nlc"),
    (HF, 600, 64, 66, 12, 0, "none", False, True, False, "nlc"),
    (F, 600, 64, 66, 16, 3, "none", False, True, False, "nlc"),
]


def adapters_case(i):
    dt, rows, K, N, rank, E, how, base, scaling, f8, layout = ADAPTERS[i]
    g = gen(1500 + i)
    two = not isinstance(rows, tuple)
    n, l = (rows, 1) if two else rows
    M = n * l
    flat = (lambda v: v if v is None else v[:, :, 0]) if two else (lambda v: v)
    x = rnd(g, n, K, l)
    xs = None
    if f8:
        xs = (x.abs().amax(1, keepdim=True) / 448)
        x = (x / xs).to(F8)
        x, xs = to_layout(x.view(torch.uint8), layout).view(F8), flat(xs.cuda())
    else:
        x = to_layout(x.to(dt), layout)
    if how == "each":
        index = torch.arange(M) % max(E, 1)
    elif how == "none":
        index = torch.tensor([-1, E, -(2 ** 31), 2 ** 31 - 1])[torch.arange(M) % 4]
    else:
        index = torch.randint(-1, E + 1, (M,), generator=g)
        index = index.sort().values if how == "runs" else index
    index = index.to(torch.int32).cuda() if two else index.to(torch.int32).view(n, l).cuda()
    kw = dict(base=flat(to_layout(rnd(g, n, N, l, dtype=dt), layout)) if base else None,
              scaling=(0.5 + torch.rand(E, generator=g)).cuda() if scaling else None, x_scales=xs)
    return (flat(x), rnd(g, E, rank, K, dtype=dt).cuda(), rnd(g, E, N, rank, dtype=dt).cuda(), index), kw


@pytest.mark.parametrize("i", range(len(ADAPTERS)))
def test_adapters(i):
    args, kw = adapters_case(i)
    print(f"adapters {ADAPTERS[i]}", flush=True)
    got = lm.adapters(*args, **kw)
    y, b = Y.adapters(*args, **kw)
    n = ADAPTERS[i][2] + ADAPTERS[i][4] + 64
    R.assert_close(got, y, b, n, "y")
    if kw["base"] is not None:   # onto the base itself
        inplace = kw["base"].clone(memory_format=torch.preserve_format)
        assert lm.adapters(*args, **{**kw, "base": inplace}, out=inplace) is inplace
        assert torch.equal(inplace, got)


@pytest.mark.parametrize("dt", [BF, HF, F])
def test_adapters_keep_rows_apart(dt):
    """What is not finite in one row, or in one adapter, reaches that row, or
    the rows that name it, alone; a zero times it is what it always is."""
    g = gen(8)
    x, a, b = rnd(g, 40, 96, dtype=dt).cuda(), rnd(g, 3, 16, 96, dtype=dt).cuda(), rnd(g, 3, 50, 16, dtype=dt).cuda()
    base = rnd(g, 40, 50, dtype=dt).cuda()
    index = torch.randint(-1, 2, (40,), generator=g).to(torch.int32).cuda()
    index[5], index[6], index[7] = 0, 2, -1
    want = lm.adapters(x, a, b, index, base=base)
    x[5], x[7], base[9, 3], a[2, 1], b[2, 4] = torch.nan, torch.inf, torch.nan, torch.inf, torch.nan
    got = lm.adapters(x, a, b, index, base=base)
    assert bool(torch.isnan(got[5]).all()) and bool(torch.isnan(got[6, 4])) and bool(torch.isnan(got[9, 3]))
    rest = [m for m in range(40) if m not in (5, 6, 9)]
    assert torch.equal(got[rest], want[rest])


def test_adapters_sums_stay_f32():
    """Inner sums that cancel to 2^-12 of their terms in the second product keep
    what 24 bits hold of them, far more than one rounding to the weights' type."""
    g = gen(10)
    for dt in (BF, HF, F):
        x, a = rnd(g, 20, 512, dtype=dt).cuda(), rnd(g, 1, 16, 512, dtype=dt).cuda()
        a[:, 8:] = a[:, :8]
        b = rnd(g, 1, 70, 16, dtype=dt).cuda()
        b[..., 8:] = -b[..., :8] * (1 + 2.0 ** -7)   # rounded to the type: differs by its last bits
        index = torch.zeros(20, dtype=torch.int32, device="cuda")
        y, bound = Y.adapters(x, a, b, index)
        R.assert_close(lm.adapters(x, a, b, index), y, bound, 512 + 16 + 64, "y")


def test_adapters_far_weights():
    """Adapters further apart than 32 bits of elements reach."""
    g = gen(11)
    x, a, b = rnd(g, 9, 72, dtype=BF).cuda(), rnd(g, 3, 8, 72, dtype=BF).cuda(), rnd(g, 3, 40, 8, dtype=BF).cuda()
    index = torch.tensor([0, 2, 1, 2, 2, 0, -1, 1, 2], dtype=torch.int32, device="cuda")
    want = lm.adapters(x, a, b, index)
    step = 2 ** 31 + 8
    big = torch.empty(2 * step + 1024, dtype=BF, device="cuda")
    far = big.as_strided((3, 8, 72), (step, 72, 1))
    far.copy_(a)
    assert torch.equal(lm.adapters(x, far, b, index), want)
    far = big.as_strided((3, 40, 8), (step, 8, 1))
    far.copy_(b)
    assert torch.equal(lm.adapters(x, a, far, index), want)
