"""The sequence operators on the GPU against the 64-bit reference: types,
layouts, odd sizes, lengths from zero, packed sequences, chunked axes, states,
gradients, single tokens, 4-bit products, streams."""
import math

import pytest
import torch

import lm_reference as R
from depthwise_stencil_implicit_amd import lm

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def to_layout(v, layout):
    """v [N, C, L] (or [N, G, S, L]) on the GPU in a memory order: 'nlc' rows of
    channels, 'ncl' contiguous, 'wide' rows inside wider ones at an odd offset,
    'every' every second channel."""
    if v is None:
        return None
    if layout == "ncl":
        return v.cuda().contiguous()
    rows = v.movedim(-1, 1).contiguous().cuda()
    if layout == "nlc":
        return rows.movedim(1, -1)
    if layout == "wide":
        big = torch.full(rows.shape[:-1] + (rows.shape[-1] + 5,), 7.0, dtype=v.dtype, device="cuda")
        big[..., 3:-2] = rows
        return big[..., 3:-2].movedim(1, -1)
    big = torch.full(rows.shape[:-1] + (2 * rows.shape[-1],), 7.0, dtype=v.dtype, device="cuda")
    big[..., ::2] = rows
    return big[..., ::2].movedim(1, -1)


def offsets_of(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32)


# ------------------------------------------------------ causal convolution --

CONV = [
    # dtype, N, C, L, K, act, bias, state, layout, lens (packed), chunk
    (BF, 2, 64, 33, 4, "silu", True, False, "nlc", None, None),
    (BF, 1, 8, 1, 4, "silu", True, True, "nlc", None, None),
    (HF, 3, 17, 2, 4, None, True, True, "nlc", None, None),
    (F, 2, 5, 40, 3, "silu", False, True, "nlc", None, 16),
    (F, 2, 3, 9, 2, None, True, False, "nlc", None, None),
    (BF, 2, 1, 70, 8, "silu", True, True, "nlc", None, 16),
    (HF, 1, 129, 65, 1, "silu", True, False, "nlc", None, 32),
    (BF, 2, 40, 50, 4, "silu", True, True, "ncl", None, None),
    (HF, 2, 40, 50, 4, "silu", True, True, "wide", None, 16),
    (F, 2, 12, 50, 5, None, True, True, "every", None, None),
    (BF, 1, 72, 90, 4, "silu", True, True, "nlc", [0, 1, 2, 40, 0, 47, 0], 16),
    (F, 1, 10, 60, 6, "silu", True, True, "wide", [3, 0, 5, 52], None),
    (HF, 1, 24, 31, 7, None, False, True, "nlc", [31], 16),
    (BF, 2, 16, 0, 4, "silu", True, True, "nlc", None, None),
]


def conv_case(i):
    dt, N, C, L, K, act, bias, state, layout, lens, chunk = CONV[i]
    g = gen(100 + i)
    n = len(lens) if lens else N
    c = dict(x=to_layout(rnd(g, N, C, L, dtype=dt), layout), w=rnd(g, C, K, dtype=dt, scale=0.6).cuda(),
             b=rnd(g, C, dtype=dt).cuda() if bias else None,
             state=rnd(g, n, C, K - 1, dtype=dt).cuda() if state else None,
             offsets=offsets_of(lens).cuda() if lens else None)
    kw = dict(activation=act, offsets=c["offsets"], max_len=max(lens) // 2 if lens else None, chunk=chunk)
    return c, kw, g, dt, act, layout


@pytest.mark.parametrize("i", range(len(CONV)))
def test_causal_conv(i):
    c, kw, g, dt, act, _ = conv_case(i)
    print(f"conv {CONV[i]}", flush=True)
    got = lm.causal_conv(c["x"], c["w"], c["b"], state=c["state"], return_state=True, **kw)
    args = (c["x"], c["w"], c["b"], act, c["state"], c["offsets"])
    (y, st), (yb, _) = R.conv(*args), R.conv(*args, bound=True)
    n = 2 * c["w"].shape[1] + 64
    R.assert_close(got.y, y, yb, n, "y")
    assert torch.equal(got.state.cpu().double(), st), "the state holds inputs exactly"


@pytest.mark.parametrize("i", range(len(CONV)))
def test_causal_conv_backward(i):
    c, kw, g, dt, act, layout = conv_case(i)
    N, C, L = c["x"].shape
    gy = to_layout(rnd(g, N, C, L, dtype=dt), layout)
    seqs = N if c["offsets"] is None else c["offsets"].numel() - 1
    gs = rnd(g, seqs, C, c["w"].shape[1] - 1, dtype=dt).cuda() if i % 2 else None
    print(f"conv backward {CONV[i]}", flush=True)
    got = lm.causal_conv_backward(gy, c["x"], c["w"], c["b"], state=c["state"], gstate=gs, **kw)
    args = (c["x"], c["w"], c["b"], act, c["state"], c["offsets"], gy, gs)
    ref, bound = R.conv(*args), R.conv(*args, bound=True)
    K = c["w"].shape[1]
    R.assert_close(got.dx, ref[0], bound[0], 4 * K + 64, "dx")
    R.assert_close(got.dw, ref[1], bound[1], N * L + 4 * K + 64, "dw")
    if c["b"] is not None:
        R.assert_close(got.db, ref[2], bound[2], N * L + 4 * K + 64, "db")
    if c["state"] is not None:
        R.assert_close(got.dstate, ref[3], bound[3], 4 * K + 64, "dstate")


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("C,K", [(1, 4), (7, 3), (64, 4), (130, 2), (33, 8)])
def test_causal_conv_step_continues_the_prompt(dt, C, K):
    g = gen(C * K)
    N, L = 3, 6
    x, w, b = to_layout(rnd(g, N, C, L, dtype=dt), "nlc"), rnd(g, C, K, dtype=dt).cuda(), rnd(g, C, dtype=dt).cuda()
    whole = lm.causal_conv(x, w, b, activation="silu", return_state=True)
    first = lm.causal_conv(x[:, :, :2], w, b, activation="silu", return_state=True)
    # The state in a table of more rows, at rows of its own.
    table = torch.full((5, K - 1, C), 3.0, dtype=dt, device="cuda").transpose(1, 2)
    rows = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    table[rows.long()] = first.state
    for t in range(2, L):
        y = lm.causal_conv_step(x[:, :, t], w, b, table, activation="silu", rows=rows)
        assert torch.equal(y, whole.y[:, :, t]), t
    assert torch.equal(table[rows.long()], whole.state)
    assert bool((table[[1, 3]] == 3).all())
    out = torch.tensor([-1, 0, 9], dtype=torch.int32, device="cuda")
    before = table.clone()
    y = lm.causal_conv_step(x[:, :, 0], w, b, table, activation="silu", rows=out)
    assert bool((y[[0, 2]] == 0).all()) and torch.equal(table[1:], before[1:])


# --------------------------------------------------------- selective scan --

SCAN = [
    # dtype, N, C, L, S, G, D, z, bias, softplus, state, layout, lens, chunk
    (F, 2, 16, 40, 16, 1, True, True, True, True, False, "nlc", None, None),
    (BF, 1, 64, 70, 16, 1, True, True, True, True, True, "nlc", None, 32),
    (HF, 2, 40, 33, 8, 2, True, False, True, True, True, "nlc", None, None),
    (F, 3, 6, 1, 4, 1, False, False, False, False, True, "nlc", None, None),
    (BF, 1, 130, 65, 12, 1, True, True, True, True, False, "nlc", None, 64),
    (F, 1, 66, 100, 1, 1, True, True, False, True, True, "nlc", None, 32),
    (F, 2, 5, 37, 3, 1, False, True, True, True, True, "nlc", None, 32),
    (BF, 1, 24, 35, 32, 3, True, True, True, True, True, "nlc", None, 32),
    (F, 1, 8, 66, 64, 2, True, True, True, True, True, "nlc", None, 32),
    (F, 2, 20, 33, 50, 1, True, False, False, True, False, "nlc", None, None),
    (BF, 2, 24, 40, 16, 1, True, True, True, True, True, "ncl", None, None),
    (HF, 2, 24, 40, 16, 1, True, True, True, True, True, "wide", None, 32),
    (F, 2, 24, 40, 7, 2, True, True, True, True, True, "every", None, None),
    (BF, 1, 72, 150, 16, 1, True, True, True, True, True, "nlc", [0, 1, 2, 97, 0, 50, 0], 32),
    (F, 1, 70, 101, 12, 2, True, True, True, True, True, "wide", [33, 0, 31, 37], None),
    (F, 1, 9, 64, 16, 1, True, True, True, True, False, "nlc", [64], 32),
    (BF, 2, 16, 0, 16, 1, True, True, True, True, True, "nlc", None, None),
]


def scan_case(i):
    dt, N, C, L, S, G, hasD, hasz, hasb, sp, st, layout, lens, chunk = SCAN[i]
    g = gen(500 + i)
    n = len(lens) if lens else N
    lay = lambda *s, scale=1.0: to_layout(rnd(g, *s, dtype=dt, scale=scale), layout)  # noqa: E731
    x, delta = lay(N, C, L), lay(N, C, L, scale=0.5)
    if not sp:
        delta = delta.abs() * 0.2
    A = -torch.exp(rnd(g, C, S, scale=0.5)).cuda()
    B, Cm = lay(N, G, S, L), lay(N, G, S, L)
    kw = dict(D=rnd(g, C).cuda() if hasD else None, z=lay(N, C, L) if hasz else None,
              dt_bias=(rnd(g, C) - 2).cuda() if hasb else None)
    state = rnd(g, n, C, S).cuda() if st else None
    off = offsets_of(lens).cuda() if lens else None
    extra = dict(dt_softplus=sp, state=state, offsets=off, max_len=max(lens) // 2 if lens else None, chunk=chunk)
    ref = dict(kw, softplus_dt=sp, state=state, offsets=off)
    return (x, delta, A, B, Cm), kw, extra, ref, g


def steps_of(i):
    return 4 * SCAN[i][3] + 2 * SCAN[i][4] + 64


@pytest.mark.parametrize("i", range(len(SCAN)))
def test_selective_scan(i):
    args, kw, extra, ref, g = scan_case(i)
    print(f"scan {SCAN[i]}", flush=True)
    got = lm.selective_scan(*args, **kw, **extra, return_state=True)
    o, b = R.scan(*args, **ref), R.scan(*args, **ref, bound=True)
    R.assert_close(got.state, o["state"], b["state"], steps_of(i), "state")
    R.assert_close(got.y, o["y"], b["y"], steps_of(i), "y")


@pytest.mark.parametrize("i", range(len(SCAN)))
def test_selective_scan_backward(i):
    args, kw, extra, ref, g = scan_case(i)
    dt, N, C, L, S, G, layout, lens = (SCAN[i][k] for k in (0, 1, 2, 3, 4, 5, 11, 12))
    gy = to_layout(rnd(g, N, C, L, dtype=dt), layout)
    n = len(lens) if lens else N
    gs = rnd(g, n, C, S).cuda() if i % 2 else None
    print(f"scan backward {SCAN[i]}", flush=True)
    saved = lm.selective_scan(*args, **kw, **extra, save=True).saved if i % 3 else None
    got = lm.selective_scan_backward(gy, *args, **kw, **extra, gstate=gs, saved=saved)
    o, b = R.scan(*args, **ref, gy=gy, gstate=gs), R.scan(*args, **ref, gy=gy, gstate=gs, bound=True)
    many = steps_of(i) * 2
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate"):
        v = getattr(got, k)
        if v is None:
            continue
        more = N * L if k in ("dA", "dD", "ddt_bias") else C if k in ("dB", "dC") else 0
        R.assert_close(v, o[k], b[k], many + more, k)
    assert (got.dz is None) == (kw["z"] is None) and (got.dstate is None) == (extra["state"] is None)


def test_scan_gradients_against_differences():
    """d<y, gy> along random directions, by central differences of the 64-bit
    forward formula."""
    g = gen(9)
    N, C, L, S = 1, 4, 12, 5
    x, dt, z, gy = (rnd(g, N, C, L) for _ in range(4))
    A, B, Cm, D, bias, st = -torch.exp(rnd(g, C, S)), rnd(g, N, 1, S, L), rnd(g, N, 1, S, L), rnd(g, C), rnd(g, C), rnd(g, N, C, S)
    v = dict(x=x, dt=dt, A=A, B=B, C=Cm, D=D, z=z, dt_bias=bias, state=st)
    c = {k: t.cuda() for k, t in v.items()}
    got = lm.selective_scan_backward(gy.cuda(), c["x"], c["dt"], c["A"], c["B"], c["C"], D=c["D"], z=c["z"], dt_bias=c["dt_bias"],
                                     dt_softplus=True, state=c["state"])
    grads = dict(x=got.dx, dt=got.ddt, A=got.dA, B=got.dB, C=got.dC, D=got.dD, z=got.dz, dt_bias=got.ddt_bias, state=got.dstate)

    def value(w):
        o = R.scan(w["x"], w["dt"], w["A"], w["B"], w["C"], w["D"], w["z"], w["dt_bias"], True, w["state"])
        return float((o["y"] * gy.double()).sum())

    for k in v:
        d = torch.randn(v[k].shape, generator=g).double()
        e = 1e-5
        up, down = ({**{n: t.double() for n, t in v.items()}, k: v[k].double() + s * e * d} for s in (1, -1))
        diff = (value(up) - value(down)) / (2 * e)
        mine = float((grads[k].cpu().double() * d).sum())
        # Differences of order e^2; f32 gradients of at most a few hundred terms.
        assert abs(diff - mine) <= 1e-4 * (1 + float((grads[k].cpu().double() * d).abs().sum())), (k, diff, mine)


def test_conv_gradients_against_differences():
    g = gen(10)
    x, w, b, st, gy = rnd(g, 2, 3, 9), rnd(g, 3, 4), rnd(g, 3), rnd(g, 2, 3, 3), rnd(g, 2, 3, 9)
    got = lm.causal_conv_backward(gy.cuda(), x.cuda(), w.cuda(), b.cuda(), activation="silu", state=st.cuda())
    v, grads = dict(x=x, w=w, b=b, state=st), dict(x=got.dx, w=got.dw, b=got.db, state=got.dstate)
    value = lambda u: float((R.conv(u["x"], u["w"], u["b"], "silu", u["state"])[0] * gy.double()).sum())  # noqa: E731
    for k in v:
        d = torch.randn(v[k].shape, generator=g).double()
        up, down = ({**{n: t.double() for n, t in v.items()}, k: v[k].double() + s * 1e-5 * d} for s in (1, -1))
        diff = (value(up) - value(down)) / 2e-5
        mine = float((grads[k].cpu().double() * d).sum())
        assert abs(diff - mine) <= 1e-4 * (1 + float((grads[k].cpu().double() * d).abs().sum())), (k, diff, mine)


def test_scan_masked_positions():
    """dt of the type's lowest value (softplus gives 0) leaves the state as it
    is; steps of a large dt forget it entirely; a NaN stays in its channel."""
    g = gen(11)
    N, C, L, S = 1, 70, 40, 16
    for dtype in (F, BF):
        x, dt = to_layout(rnd(g, N, C, L, dtype=dtype), "nlc"), to_layout(rnd(g, N, C, L, dtype=dtype), "nlc")
        B, Cm = to_layout(rnd(g, N, 1, S, L, dtype=dtype), "nlc"), to_layout(rnd(g, N, 1, S, L, dtype=dtype), "nlc")
        A, st = -torch.exp(rnd(g, C, S)).cuda(), rnd(g, N, C, S).cuda()
        dt[:, :, 5:20] = torch.finfo(dtype).min
        dt[:, 3] = torch.finfo(dtype).min
        dt[:, 4] = -math.inf
        dt[:, 7, 30] = 1e4
        x[:, 9, 12] = math.nan
        got = lm.selective_scan(x, dt, A, B, Cm, dt_softplus=True, state=st, return_state=True)
        o = R.scan(x, dt, A, B, Cm, softplus_dt=True, state=st)
        b = R.scan(torch.nan_to_num(x), dt, A, B, Cm, softplus_dt=True, state=st, bound=True)
        assert torch.equal(got.state[:, 3:5], st[:, 3:5])
        R.assert_close(got.state, o["state"], b["state"], 4 * L + 96, "state")
        R.assert_close(got.y, o["y"], b["y"], 4 * L + 96, "y")
        clean = lm.selective_scan(torch.nan_to_num(x), dt, A, B, Cm, dt_softplus=True, state=st).y
        others = [c for c in range(C) if c != 9]
        assert torch.equal(got.y[:, others], clean[:, others])


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("C,S,G", [(4, 16, 1), (30, 5, 2), (65, 64, 1), (12, 2, 3), (8, 32, 1)])
def test_selective_scan_step(dt, C, S, G):
    g = gen(C + S)
    N = 3
    x, d, z = (rnd(g, N, C, dtype=dt).cuda() for _ in range(3))
    B, Cm = rnd(g, N, G, S, dtype=dt).cuda(), rnd(g, N, G, S, dtype=dt).cuda()
    A, D, bias, st = -torch.exp(rnd(g, C, S)).cuda(), rnd(g, C).cuda(), rnd(g, C).cuda(), rnd(g, N, C, S).cuda()
    ref = dict(D=D, z=z[..., None], dt_bias=bias, softplus_dt=True, state=st)
    args = (x[..., None], d[..., None], A, B[..., None], Cm[..., None])
    o, b = R.scan(*args, **ref), R.scan(*args, **ref, bound=True)
    # In a table with other rows, through row numbers; one batch row is left out.
    table = torch.full((6, C, S), 2.0, device="cuda")
    rows = torch.tensor([5, 1, 3], dtype=torch.int32, device="cuda")
    table[rows.long()] = st
    y = lm.selective_scan_step(x, d, A, B, Cm, table, D=D, z=z, dt_bias=bias, dt_softplus=True, rows=rows)
    R.assert_close(y, o["y"][..., 0], b["y"][..., 0], 2 * S + 68, "y")
    R.assert_close(table[rows.long()], o["state"], b["state"], 68, "state")
    assert bool((table[[0, 2, 4]] == 2).all())
    # The state at other strides, states not contiguous.
    other = st.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(lm.selective_scan_step(x, d, A, B, Cm, other, D=D, z=z, dt_bias=bias, dt_softplus=True), y)
    assert torch.equal(other, table[rows.long()])
    before = table.clone()
    out = torch.tensor([6, -1, 1], dtype=torch.int32, device="cuda")
    y = lm.selective_scan_step(x, d, A, B, Cm, table, D=D, z=z, dt_bias=bias, dt_softplus=True, rows=out)
    assert bool((y[:2] == 0).all()) and torch.equal(table[[0, 2, 3, 4, 5]], before[[0, 2, 3, 4, 5]])


# ---------------------------------------------------------- 4-bit products --

@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("M,K,N,group,zeros,bias", [
    (1, 128, 16, 128, False, False), (1, 32, 1, 32, True, True), (16, 256, 33, 64, True, False), (17, 160, 40, 32, False, True),
    (3, 1152, 50, 128, True, True), (5, 1152, 70, 384, False, False), (40, 96, 19, 96, True, True), (2, 4096, 17, 4096, False, True),
    (0, 64, 8, 32, False, False), (7, 2080, 31, 32, True, False), (2, 192, 35, 64, True, True), (3, 224, 20, 32, False, False),
    (1, 1120, 50, 224, True, False)])
def test_matvec4(dt, M, K, N, group, zeros, bias):
    g = gen(M + K + N)
    x = rnd(g, M, K, dtype=dt).cuda()
    packed = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (torch.rand((N, K // group), generator=g) / 8).to(dt).cuda()
    zz = torch.randint(0, 16, (N, K // group), generator=g).to(dt).cuda() if zeros else None
    bb = rnd(g, N, dtype=dt).cuda() if bias else None
    y = lm.matvec4(x, packed, scales, zz, bb)
    # Sums inside a block of 128 columns, then one rounding per group and wave.
    n = 128 + 2 * (K // min(group, 128)) + 16
    R.assert_close(y, R.matvec4(x, packed, scales, zz, bb), R.matvec4(x, packed, scales, zz, bb, bound=True), n, "y")
    if M > 1:
        # Rows of another tensor: strided, off 16 bytes, columns apart.
        wide = torch.zeros(M, K + 3, dtype=dt, device="cuda")
        wide[:, 1:K + 1] = x
        assert torch.equal(lm.matvec4(wide[:, 1:K + 1], packed, scales, zz, bb), y)
        apart = torch.zeros(K, M, dtype=dt, device="cuda").t()
        apart.copy_(x)
        assert torch.equal(lm.matvec4(apart, packed, scales, zz, bb), y)
        assert torch.equal(lm.matvec4(x[1:2], packed, scales, zz, bb), y[1:2])


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("M,K,N,group,zeros", [(2, 8320, 37, 128, False), (17, 16384, 16, 64, True), (1, 9088, 40, 32, False),
                                               (3, 10240, 20, 2560, True), (2, 8224, 33, 32, True), (5, 4160, 18, 64, False)])
def test_matvec4_long_rows(dt, M, K, N, group, zeros):
    """Rows split over several workgroups."""
    g = gen(M + K + N)
    x = rnd(g, M, K, dtype=dt).cuda()
    packed = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (torch.rand((N, K // group), generator=g) / 8).to(dt).cuda()
    zz = torch.randint(0, 16, (N, K // group), generator=g).to(dt).cuda() if zeros else None
    y = lm.matvec4(x, packed, scales, zz)
    n = 128 + 2 * (K // min(group, 128)) + 16
    R.assert_close(y, R.matvec4(x, packed, scales, zz), R.matvec4(x, packed, scales, zz, bound=True), n, "y")
    apart = torch.zeros(K, M, dtype=dt, device="cuda").t()
    apart.copy_(x)
    assert torch.equal(lm.matvec4(apart, packed, scales, zz), y)


def test_matvec4_counts_every_weight_exactly():
    """Powers of two pick single weights: the product is exact."""
    for dt in (BF, HF, F):
        K, N = 256, 16
        packed = torch.randint(0, 256, (N, K // 2), generator=gen(3), dtype=torch.uint8)
        q = torch.stack([packed & 15, packed >> 4], 2).reshape(N, K).double() - 8
        x = torch.eye(K).to(dt)
        for group in (32, 128):
            y = lm.matvec4(x.cuda(), packed.cuda(), torch.ones(N, K // group, dtype=dt, device="cuda"))
            assert torch.equal(y.cpu().double(), q.t())


def test_quantize4_round_trip():
    w = torch.randn(40, 256, generator=gen(4)).cuda()
    w[3, :64] = 0
    for symmetric in (True, False):
        packed, scales, zeros = lm.quantize4(w, 64, symmetric=symmetric, dtype=F)
        back = lm.matvec4(torch.eye(256, device="cuda"), packed, scales, zeros).t()
        step = scales.repeat_interleave(64, 1)
        assert bool(((back - w).abs() <= step * 0.5001 + (0 if symmetric else step * 0.5)).all())


# ------------------------------------------------------------ whole calls --

def test_results_repeat_bit_for_bit():
    args, kw, extra, _, g = scan_case(1)
    gy = to_layout(rnd(g, 1, 64, 70, dtype=BF), "nlc")
    a, b = (lm.selective_scan_backward(gy, *args, **kw, **extra) for _ in range(2))
    for u, v in zip(a, b):
        assert u is None or torch.equal(u, v)


def test_another_stream():
    args, kw, extra, _, _ = scan_case(1)
    want = lm.selective_scan(*args, **kw, **extra, return_state=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lm.selective_scan(*args, **kw, **extra, return_state=True)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got.y, want.y) and torch.equal(got.state, want.state)


def test_parts_of_the_gradients():
    """Selected gradients, a depthwise [C, 1, K] weight, one group without its
    dim, a broadcast output gradient."""
    g = gen(21)
    x, w, b = to_layout(rnd(g, 2, 20, 33), "nlc"), rnd(g, 20, 4).cuda(), rnd(g, 20).cuda()
    gy = rnd(g, 2, 20, 1).cuda().expand(2, 20, 33)
    whole = lm.causal_conv_backward(gy, x, w[:, None], b, activation="silu")
    assert whole.dw.shape == (20, 1, 4)
    one = lm.causal_conv_backward(gy.contiguous(), x, w, b, activation="silu", need_dx=False)
    two = lm.causal_conv_backward(gy, x, w, b, activation="silu", need_dw=False)
    assert one.dx is None and two.dw is None and two.db is None
    assert torch.equal(one.dw, whole.dw[:, 0]) and torch.equal(one.db, whole.db) and torch.equal(two.dx, whole.dx)
    dt, A = to_layout(rnd(g, 2, 20, 33), "nlc"), -torch.exp(rnd(g, 20, 6)).cuda()
    B, C = to_layout(rnd(g, 2, 1, 6, 33), "nlc"), to_layout(rnd(g, 2, 1, 6, 33), "nlc")
    D = torch.ones(1, device="cuda").expand(20)
    args = dict(D=D, dt_softplus=True)
    a = lm.selective_scan_backward(gy, x, dt, A, B, C, **args)
    c = lm.selective_scan_backward(gy, x, dt, A, B[:, 0], C[:, 0], **args)
    assert c.dB.shape == (2, 6, 33) and torch.equal(c.dB, a.dB[:, 0]) and torch.equal(c.dx, a.dx)
    assert a.dD.shape == (20,) and torch.equal(a.dD, c.dD)


def test_decoding_in_a_graph():
    """One token through convolution, scan and projection in a captured graph,
    replayed with eager work and synchronisation between."""
    g = gen(22)
    n, c, s = 3, 64, 16
    w, b, A = rnd(g, c, 4, dtype=BF).cuda(), rnd(g, c, dtype=BF).cuda(), -torch.exp(rnd(g, c, s)).cuda()
    B, C = rnd(g, n, 1, s, dtype=BF).cuda(), rnd(g, n, 1, s, dtype=BF).cuda()
    packed = torch.randint(0, 256, (40, c // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (torch.rand((40, 2), generator=g) / 8).to(BF).cuda()
    xs = [rnd(g, n, c, dtype=BF).cuda() for _ in range(4)]
    start = rnd(g, n, c, 3, dtype=BF).cuda(), rnd(g, n, c, s).cuda()

    def step(x, conv, ssm):
        u = lm.causal_conv_step(x, w, b, conv, activation="silu")
        y = lm.selective_scan_step(u, u, A, B, C, ssm, dt_softplus=True)
        return lm.matvec4(y, packed, scales)

    eager = tuple(t.clone() for t in start)
    want = [step(x, *eager) for x in xs]
    state, x = tuple(t.clone() for t in start), xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, *(t.clone() for t in start))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, *state)
    for t, v in zip(state, start):
        t.copy_(v)
    for k, v in enumerate(xs):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k]), k
        torch.empty(1 << 20, device="cuda").fill_(float(k))
    assert all(torch.equal(t, v) for t, v in zip(state, eager))


def test_refuses_tensors_elsewhere():
    x = torch.zeros(1, 8, 4, device="cuda")
    with pytest.raises(ValueError, match="GPU only"):
        lm.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(RuntimeError, match="element type"):
        lm.causal_conv(x, torch.zeros(8, 4, device="cuda", dtype=HF))
