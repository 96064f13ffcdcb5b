"""Calls of the sequence operators as programs make them: prepared steps with
an output and a stream of the caller's, steps by name, extreme values, packed
batches, products that are exact."""
import pytest
import torch

import lm_reference as R
from depthwise_stencil_implicit_amd import lm

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def pool_of(t):
    """The stream whose memory holds t."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's memory")


def prepared(kind, dt=BF):
    """(run(**kw), state or None, its start, y of the plain call, that call's state)."""
    g = gen(31)
    if kind == "conv":
        x, w, b, st = rnd(g, 3, 70, dtype=dt), rnd(g, 70, 4, dtype=dt), rnd(g, 70, dtype=dt), rnd(g, 3, 70, 3, dtype=dt)
        p = lm.PreparedCausalConvStep(x, w, b, st, activation="silu")
        run = lambda s, **kw: p.run(x, w, b, s, **kw)  # noqa: E731
        plain = lambda s: lm.causal_conv_step(x, w, b, s, activation="silu")  # noqa: E731
    elif kind == "scan":
        x, d, z, B, C = rnd(g, 3, 70, dtype=dt), rnd(g, 3, 70, dtype=dt), rnd(g, 3, 70, dtype=dt), rnd(g, 3, 1, 16, dtype=dt), rnd(g, 3, 1, 16, dtype=dt)
        A, D, st = -torch.exp(rnd(g, 70, 16)), rnd(g, 70), rnd(g, 3, 70, 16)
        p = lm.PreparedSelectiveScanStep(x, d, A, B, C, st, D=D, z=z, dt_softplus=True)
        run = lambda s, **kw: p.run(x, d, A, B, C, s, D=D, z=z, **kw)  # noqa: E731
        plain = lambda s: lm.selective_scan_step(x, d, A, B, C, s, D=D, z=z, dt_softplus=True)  # noqa: E731
    else:
        # More columns than one workgroup takes, and in "apart" an x to be gathered first.
        k = 8448 if kind == "split" else 256
        x = rnd(g, 3, k, dtype=dt) if kind == "split" else rnd(g, k, 3, dtype=dt).t()
        packed = torch.randint(0, 256, (50, k // 2), generator=g, dtype=torch.uint8).cuda()
        scales, st = (torch.rand((50, k // 32), generator=g) / 8).to(dt).cuda(), None
        p = lm.PreparedMatvec4(x, packed, scales)
        assert p.plan.workspace_bytes > 0
        run = lambda s, **kw: p.run(x, packed, scales, **kw)  # noqa: E731
        plain = lambda s: lm.matvec4(x, packed, scales)  # noqa: E731
    copy = lambda: st.clone() if st is not None else None  # noqa: E731
    after = copy()
    return run, copy, plain(after), after


@pytest.mark.parametrize("kind", ["conv", "scan", "split", "apart"])
def test_prepared_run_on_a_given_stream(kind):
    """With and without an output of the caller's, on the current stream, on
    another one that is busy while the current one allocates, and on the default
    stream from within another."""
    run, copy, want, after = prepared(kind)
    s = torch.cuda.Stream()
    for stream in (None, torch.cuda.current_stream().cuda_stream, s.cuda_stream):
        for given in (False, True):
            state = copy()
            y = torch.full_like(want, 5.0) if given else None
            big = torch.zeros(1 << 26, device="cuda")
            torch.cuda.synchronize()
            if stream == s.cuda_stream:
                with torch.cuda.stream(s):
                    for _ in range(8):
                        big.add_(1.0)
            out = run(state, y=y, stream=stream)
            for size in (want.numel() * want.element_size(), 50 * 3 * 2 * 4, 3 * 256 * 2, 1 << 16):
                torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            assert not given or out is y
            assert given or pool_of(out) == (s.cuda_stream if stream == s.cuda_stream else torch.cuda.current_stream().cuda_stream)
            assert torch.equal(out, want), (stream, given)
            assert state is None or torch.equal(state, after)
    state = copy()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = run(state, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and pool_of(out) == 0


@pytest.mark.parametrize("dt,C,S,L,chunk", [(F, 20, 16, 37, None), (BF, 70, 12, 100, 32), (HF, 8, 40, 21, None), (F, 5, 64, 70, 32)])
def test_scan_of_rates_that_forget_at_once(dt, C, S, L, chunk):
    """A = -inf: exp(d A) is 0 for every d > 0, also where the axis ends inside
    a block of steps; the gradients of A and d through that factor are 0."""
    g = gen(C + L)
    lay = lambda *s: rnd(g, *s, dtype=dt).movedim(-1, 1).contiguous().movedim(1, -1)  # noqa: E731
    x, d, z, gy, B, Cm = lay(1, C, L), lay(1, C, L), lay(1, C, L), lay(1, C, L), lay(1, 1, S, L), lay(1, 1, S, L)
    A, D, st, gs = -torch.exp(rnd(g, C, S, scale=0.5)), rnd(g, C), rnd(g, 1, C, S), rnd(g, 1, C, S)
    A[::3, 1::2] = -torch.inf
    kw = dict(D=D, z=z, state=st)
    ref = lambda **k: R.scan(x, d, A.clamp(min=-1e30), B, Cm, softplus_dt=True, **kw, **k)  # noqa: E731  exp(-1e30 d) is 0 in 64 bits too
    n = 8 * L + 4 * S + 128
    got = lm.selective_scan(x, d, A, B, Cm, dt_softplus=True, return_state=True, chunk=chunk, **kw)
    o, b = ref(), ref(bound=True)
    R.assert_close(got.state, o["state"], b["state"], n, "state")
    R.assert_close(got.y, o["y"], b["y"], n, "y")
    grads = lm.selective_scan_backward(gy, x, d, A, B, Cm, dt_softplus=True, gstate=gs, chunk=chunk, **kw)
    o, b = ref(gy=gy, gstate=gs), ref(gy=gy, gstate=gs, bound=True)
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dstate"):
        R.assert_close(getattr(grads, k), o[k], b[k], n + (L if k in ("dA", "dD") else C), k)
    h = st.clone()
    y = lm.selective_scan_step(x[:, :, 0], d[:, :, 0], A, B[..., 0], Cm[..., 0], h, D=D, z=z[:, :, 0], dt_softplus=True)
    one = [v[..., :1] for v in (x, d, B, Cm, z)]
    args = (one[0], one[1], A.clamp(min=-1e30), one[2], one[3])
    o, b = R.scan(*args, D=D, z=one[4], softplus_dt=True, state=st), R.scan(*args, D=D, z=one[4], softplus_dt=True, state=st, bound=True)
    R.assert_close(y, o["y"][..., 0], b["y"][..., 0], n, "step's y")
    R.assert_close(h, o["state"], b["state"], n, "step's state")


@pytest.mark.parametrize("lens", [None, [3, 0, 4]])
def test_scan_gradients_without_channels(lens):
    """dB and dC are sums over the channels: zeros when there are none."""
    from depthwise_stencil_implicit_amd import _abi as A
    N, G, S, L = (1, 2, 5, 7) if lens else (2, 1, 5, 7)
    x, B, rate = torch.zeros(N, 0, L, device="cuda"), rnd(gen(1), N, G, S, L), torch.zeros(0, S, device="cuda")
    off = torch.tensor([0, 3, 3, 7], dtype=torch.int32, device="cuda") if lens else None
    dB, dC = torch.full_like(B, 5.0), torch.full_like(B, 5.0)
    ins = [(lm._GY, x), (lm._X, x), (lm._DT, x), (lm._A, rate), (lm._B, B), (lm._C, B), (lm._OFF, off),
           (lm._SAVED, lm._new_saved(x, rate, off))]
    lm._call(A.LM_SCAN_BWD, ins, [(lm._DX, x.clone()), (lm._DDT, x.clone()), (lm._DA, rate.clone()), (lm._DB, dB), (lm._DC, dC)])
    assert bool((dB == 0).all()) and bool((dC == 0).all())
    got = lm.selective_scan_backward(x, x, x, rate, B, B, offsets=off)
    assert got.dx.shape == x.shape and bool((got.dB == 0).all()) and bool((got.dC == 0).all())
    out = lm.selective_scan(x, x, rate, B, B, offsets=off, return_state=True)
    assert out.y.shape == x.shape and out.state.shape == (len(lens) if lens else N, 0, S)


def lengths(g, n, total, most_empty=False):
    """n lengths that add up to total, many of them zero with most_empty."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=g).sort().values
    if most_empty:
        cuts = cuts[torch.randint(0, 4, (n - 1,), generator=g).sort().values] if n > 4 else cuts
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([total])]).to(torch.int32)


PACKED = [
    # dtype, sequences, rows, channels, chunk, max_len, most of them empty
    (F, 5, 130, 24, 32, None, False),
    (BF, 13, 300, 1, 32, None, False),       # a wave spans many chunks
    (F, 70, 400, 3, 32, None, True),         # more than one wave of sequences
    (HF, 200, 260, 66, 32, 7, False),        # max_len far below the longest
    (F, 4200, 4500, 2, 32, None, False),     # more than a wave of waves
    (BF, 1, 200, 130, 64, None, False),
    (F, 3, 96, 40, 32, 1, True),
]


def packed_case(i):
    dt, n, t, c, chunk, max_len, empty = PACKED[i]
    g = gen(700 + i)
    off = lengths(g, n, t, empty)
    rows = lambda *s: rnd(g, t, *s, dtype=dt).movedim(0, -1)[None]  # noqa: E731
    return g, dt, n, t, c, off.cuda(), dict(offsets=off.cuda(), chunk=chunk, max_len=max_len), rows


@pytest.mark.parametrize("i", range(len(PACKED)))
def test_packed_convolutions_of_any_lengths(i):
    """Chunks of unlike sequences beside each other, in one piece and in many;
    every sequence, the empty ones too, hands its state on."""
    g, dt, n, t, c, off, kw, rows = packed_case(i)
    print(f"packed conv {PACKED[i]}", flush=True)
    K = 4
    x, gy, w, b = rows(c), rows(c), rnd(g, c, K, dtype=dt, scale=0.6), rnd(g, c, dtype=dt)
    st, gs = rnd(g, n, c, K - 1, dtype=dt), rnd(g, n, c, K - 1, dtype=dt)
    args = (x, w, b, "silu", st, off)
    (y, last), (yb, _) = R.conv(*args), R.conv(*args, bound=True)
    ref, bound = R.conv(*args, gy, gs), R.conv(*args, gy, gs, bound=True)
    for chunk in (kw["chunk"], 3, None):
        kw["chunk"] = chunk
        got = lm.causal_conv(x, w, b, activation="silu", state=st, return_state=True, **kw)
        back = lm.causal_conv_backward(gy, x, w, b, activation="silu", state=st, gstate=gs, **kw)
        R.assert_close(got.y, y, yb, 2 * K + 64, "y")
        assert torch.equal(got.state.cpu().double(), last)
        for name, v, r, e in zip(("dx", "dw", "db", "dstate"), back, ref, bound):
            R.assert_close(v, r, e, (t if name in ("dw", "db") else 0) + 4 * K + 64, name)


@pytest.mark.parametrize("i", range(len(PACKED)))
def test_packed_scans_of_any_lengths(i):
    g, dt, n, t, c, off, kw, rows = packed_case(i)
    print(f"packed scan {PACKED[i]}", flush=True)
    S = 6
    x, d, z, gy, B, Cm = rows(c), rows(c), rows(c), rows(c), rows(1, S), rows(1, S)
    A, D, st, gs = -torch.exp(rnd(g, c, S, scale=0.5)), rnd(g, c), rnd(g, n, c, S), rnd(g, n, c, S)
    par = dict(D=D, z=z, state=st)
    got = lm.selective_scan(x, d, A, B, Cm, dt_softplus=True, return_state=True, **par, **kw)
    o, b = (R.scan(x, d, A, B, Cm, softplus_dt=True, offsets=off, **par, bound=k) for k in (False, True))
    n_f = 4 * t + 2 * S + 64
    R.assert_close(got.state, o["state"], b["state"], n_f, "state")
    R.assert_close(got.y, o["y"], b["y"], n_f, "y")
    back = lm.selective_scan_backward(gy, x, d, A, B, Cm, dt_softplus=True, gstate=gs, **par, **kw)
    o, b = (R.scan(x, d, A, B, Cm, softplus_dt=True, offsets=off, **par, gy=gy, gstate=gs, bound=k) for k in (False, True))
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dstate"):
        R.assert_close(getattr(back, k), o[k], b[k], 2 * n_f + (t if k in ("dA", "dD") else c), k)


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("K,group,zeros", [
    (192, 64, True), (224, 32, False), (160, 32, True), (1120, 224, True), (1152, 96, False), (2080, 32, True), (4160, 64, False),
    (8224, 32, True), (9088, 32, False), (8320, 128, False), (16384, 64, True), (10240, 2560, True)])
def test_matvec4_weighs_every_group_exactly(dt, K, group, zeros):
    """Rows with one power of two each, one in every 32 columns and in each of
    the last 64: rows cut short, split rows and every size of group leave no
    column out, take its own scale and zero, and round nothing."""
    g = gen(K)
    N = 21
    cols = sorted({c + (7 * c // 32) % 32 for c in range(0, K, 32)} | set(range(K - 64, K)))
    x = torch.zeros(len(cols), K, dtype=torch.float64)
    x[range(len(cols)), cols] = 2.0 ** (torch.arange(len(cols)) % 5 - 2).double()
    packed = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = 2.0 ** torch.randint(-4, 3, (N, K // group), generator=g).double()
    zz = torch.randint(0, 16, (N, K // group), generator=g).double() if zeros else None
    q = torch.stack([packed & 15, packed >> 4], 2).reshape(N, K).double()
    w = scales.repeat_interleave(group, 1) * (q - (zz.repeat_interleave(group, 1) if zeros else 8))
    on = lambda v: v.to(dt).cuda() if v is not None else None  # noqa: E731
    y = lm.matvec4(on(x), packed.cuda(), on(scales), on(zz))
    assert torch.equal(y.cpu().double(), x @ w.t())


def test_steps_of_zero_keep_the_state():
    """dt of the type's lowest value under softplus is d = 0: prompt and step
    leave the state bit for bit, whatever A is, and a NaN in A stays one."""
    g = gen(77)
    C, S, L = 12, 16, 5
    x, B = rnd(g, 1, C, L), rnd(g, 1, 1, S, L)
    d = torch.full_like(x, torch.finfo(F).min)
    A, st = -torch.exp(rnd(g, C, S)), rnd(g, 1, C, S)
    A[::2, ::3], A[1, 1] = -torch.inf, torch.inf
    got = lm.selective_scan(x, d, A, B, B, dt_softplus=True, state=st, return_state=True)
    assert torch.equal(got.state, st)
    h = st.clone()
    lm.selective_scan_step(x[:, :, 0], d[:, :, 0], A, B[..., 0], B[..., 0], h, dt_softplus=True)
    assert torch.equal(h, st)
    A[3, 4] = torch.nan
    got = lm.selective_scan(x, x, A, B, B, dt_softplus=True, state=st, return_state=True)
    assert torch.equal(torch.isnan(got.state).nonzero().cpu(), torch.tensor([[0, 3, 4]]))
