"""Calls of the recurrence, the norm and the adapters as programs make them:
packed batches of any lengths and long ones, prepared calls with a stream and an
output of the caller's, captured steps, large batches in any order."""
import pytest
import torch

import layer_reference as Y
import lm_reference as R
from depthwise_stencil_implicit_amd import lm
from test_gpu_layer import BF, F, F8, HF
from test_gpu_lm_calls import PACKED, gen, packed_case, pool_of, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("i", range(len(PACKED)))
def test_packed_recurrences_of_any_lengths(i):
    """Chunks of unlike sequences beside each other, in one piece and in many;
    every sequence, the empty ones too, hands its state on."""
    g, dt, n, t, c, off, kw, rows = packed_case(i)
    print(f"packed gated {PACKED[i]}", flush=True)
    x, r, i_, gy, decay, st, gs = rows(c), rows(c), rows(c), rows(c), rnd(g, c) - 4, rnd(g, n, c), rnd(g, n, c)
    args, ref = (x, r, i_, decay), dict(state=st, offsets=off)
    o, b = (Y.gated(*args, **ref, bound=k) for k in (False, True))
    go, gb = (Y.gated(*args, **ref, gy=gy, gstate=gs, bound=k) for k in (False, True))
    steps = 24 * t + 192
    for chunk in (128, None):
        got = lm.gated_recurrence(*args, state=st, offsets=off, max_len=kw["max_len"], chunk=chunk, return_state=True, save=True)
        R.assert_close(got.y, o["y"], b["y"], steps, "y")
        R.assert_close(got.state, o["state"], b["state"], steps, "state")
        back = lm.gated_recurrence_backward(gy, *args, state=st, offsets=off, max_len=kw["max_len"], chunk=chunk, gstate=gs, saved=got.saved)
        for k in ("dx", "dr", "di", "ddecay", "dstate"):
            R.assert_close(getattr(back, k), go[k], gb[k], 2 * steps + (t if k == "ddecay" else 0), k)


@pytest.mark.parametrize("dt,c,lens", [(BF, 66, [7000]), (F, 3, [5200, 0, 40, 2500]), (HF, 257, [130, 4000, 1])])
def test_long_recurrences(dt, c, lens):
    """Tiles that look further back than sixteen others, on slow decays."""
    g = gen(c)
    t = sum(lens)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    rows = lambda: rnd(g, t, c, dtype=dt).t()[None]  # noqa: E731
    x, r, i, gy, decay, st = rows(), rows(), rows(), rows(), rnd(g, c) - 9, rnd(g, len(lens), c)
    o, b = (Y.gated(x, r, i, decay, state=st, offsets=off, bound=k) for k in (False, True))
    for kw in (dict(chunk=128), dict(chunk=256), dict()):
        got = lm.gated_recurrence(x, r, i, decay, state=st, offsets=off, return_state=True, save=True, **kw)
        # Rounding errors of factors next to 1 add up over the axis, two a step.
        R.assert_close(got.y, o["y"], b["y"], 4 * t + 192, "y")
        R.assert_close(got.state, o["state"], b["state"], 4 * t + 192, "state")
        for _ in range(3):   # however far its tiles had to look
            again = lm.gated_recurrence(x, r, i, decay, state=st, offsets=off, return_state=True, save=True, **kw)
            assert torch.equal(got.y, again.y) and torch.equal(got.state, again.state)
    o, b = (Y.gated(x, r, i, decay, state=st, offsets=off, gy=gy, bound=k) for k in (False, True))
    back = lm.gated_recurrence_backward(gy, x, r, i, decay, state=st, offsets=off, saved=got.saved)
    for k in ("dx", "dr", "di", "ddecay", "dstate"):
        R.assert_close(getattr(back, k), o[k], b[k], 8 * t + 384 + (t if k == "ddecay" else 0), k)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("l", [1, 2, 4, 5, 8, 9, 33, 60, 64, 65, 120, 121, 128])
def test_short_recurrences(dt, l):
    """Workgroups of fewer waves, the last of them with a row or all of its rows;
    the same tokens packed into unlike sequences."""
    g = gen(l)
    n, c = 3, 70
    decay, st, gs = rnd(g, c) - 4, rnd(g, n, c), rnd(g, n, c)
    x, r, i, gy = (rnd(g, n, l, c, dtype=dt).transpose(1, 2) for _ in range(4))
    packed = [rnd(g, 1, l, c, dtype=dt).transpose(1, 2) for _ in range(4)]
    off = torch.tensor([0, l // 3, l // 3, l], dtype=torch.int32, device="cuda")
    for (x, r, i, gy), off in (((x, r, i, gy), None), (packed, off)):
        o, b = (Y.gated(x, r, i, decay, state=st, offsets=off, bound=k) for k in (False, True))
        go, gb = (Y.gated(x, r, i, decay, state=st, offsets=off, gy=gy, gstate=gs, bound=k) for k in (False, True))
        steps = 24 * l + 192
        got = lm.gated_recurrence(x, r, i, decay, state=st, offsets=off, return_state=True, save=True)
        R.assert_close(got.y, o["y"], b["y"], steps, "y")
        R.assert_close(got.state, o["state"], b["state"], steps, "state")
        back = lm.gated_recurrence_backward(gy, x, r, i, decay, state=st, offsets=off, gstate=gs, saved=got.saved)
        for k in ("dx", "dr", "di", "ddecay", "dstate"):
            R.assert_close(getattr(back, k), go[k], gb[k], 2 * steps + (n * l if k == "ddecay" else 0), k)


# -------------------------------------------------- prepared calls, streams --

def prepared(kind):
    """(run(**kw) -> outputs, the plain call's)."""
    g = gen(41)
    if kind == "step":
        x, r, i, decay, st = rnd(g, 5, 70, dtype=BF), rnd(g, 5, 70, dtype=BF), rnd(g, 5, 70, dtype=BF), rnd(g, 70) - 4, rnd(g, 5, 70)
        p = lm.PreparedGatedRecurrenceStep(x, r, i, decay, st)
        after = st.clone()
        return lambda **kw: (p.run(x, r, i, decay, s := st.clone(), **kw), s), (lm.gated_recurrence_step(x, r, i, decay, after), after)
    if kind.startswith("norm"):
        x, res, w = rnd(g, 9, 320, dtype=HF), rnd(g, 9, 320, dtype=HF), rnd(g, 320, dtype=HF)
        kw0 = dict(out_dtype=F8, group=64) if kind == "norm8" else dict(save=True)
        p = lm.PreparedRmsNorm(x, w, res, **kw0)
        return lambda stream=None: p.run(x, w, res, stream=stream), lm.rms_norm(x, w, residual=res, **kw0)
    m, e = {"adapters": (30, 6), "adapters found": (700, 6), "adapters sorted": (700, 70)}[kind]
    x, a, b, base = rnd(g, m, 200, dtype=BF), rnd(g, e, 24, 200, dtype=BF), rnd(g, e, 90, 24, dtype=BF), rnd(g, m, 90, dtype=BF)
    index = torch.randint(-1, e, (m,), generator=g).to(torch.int32).cuda()
    p = lm.PreparedAdapters(x, a, b, index, base=base)
    assert p.plan.workspace_bytes > 0
    return lambda **kw: (p.run(x, a, b, index, base=base, **kw),), (lm.adapters(x, a, b, index, base=base),)


@pytest.mark.parametrize("kind", ["step", "norm", "norm8", "adapters", "adapters found", "adapters sorted"])
def test_prepared_run_on_a_given_stream(kind):
    """On the current stream, on another one that is busy while the current one
    allocates, and on the default stream from within another."""
    run, want = prepared(kind)
    s = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream
    for stream in (None, here, s.cuda_stream, 0):
        big = torch.zeros(1 << 26, device="cuda")
        torch.cuda.synchronize()
        if stream == s.cuda_stream:
            with torch.cuda.stream(s):
                for _ in range(8):
                    big.add_(1.0)
        if kind == "step" and stream is not None:
            torch.cuda.synchronize()   # its copy of the state is made on the current stream
        with torch.cuda.stream(s if stream == 0 else torch.cuda.current_stream()):
            out = run(stream=stream)
        for size in (1 << 12, 1 << 14, 1 << 16):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for k, (got, exp) in enumerate(zip(out, want)):
            if exp is None:
                assert got is None
                continue
            if kind != "step" or k == 0:
                assert pool_of(got) == (s.cuda_stream if stream == s.cuda_stream else 0 if stream == 0 else here)
            view = (lambda t: t.view(torch.uint8)) if exp.dtype == F8 else (lambda t: t)
            assert torch.equal(view(got), view(exp)), (stream, k)


def test_prepared_adapters_onto_the_base():
    g = gen(42)
    x, a, b, base = rnd(g, 8, 64, dtype=BF), rnd(g, 2, 8, 64, dtype=BF), rnd(g, 2, 40, 8, dtype=BF), rnd(g, 8, 40, dtype=BF)
    index = torch.tensor([0, 1, -1, 1, 0, 0, 2, 1], dtype=torch.int32, device="cuda")
    want = lm.adapters(x, a, b, index, base=base)
    p = lm.PreparedAdapters(x, a, b, index, base=base)
    assert p.run(x, a, b, index, base=base, y=base) is base and torch.equal(base, want)


@pytest.mark.parametrize("m,e", [(40, 3), (600, 3), (600, 70)])
def test_a_layer_in_a_graph(m, e):
    """Norm, adapters and recurrence of a token and of a prompt in one captured
    graph, replayed with other inputs and eager work between."""
    g = gen(43)
    c, l = 96, 300
    w, decay = rnd(g, c, dtype=BF), rnd(g, c) - 4
    a, b = rnd(g, e, 16, c, dtype=BF), rnd(g, e, c, 16, dtype=BF)
    ins = [(rnd(g, m, c, dtype=BF), rnd(g, m, c, dtype=BF), torch.randint(-1, e, (m,), generator=g).to(torch.int32).cuda(),
            rnd(g, 1, l, c, dtype=BF).transpose(1, 2)) for _ in range(4)]
    start = rnd(g, m, c)

    def layer(x, res, index, rows, state):
        n = lm.rms_norm(x, w, residual=res)
        q = lm.rms_norm(x, w, residual=res, out_dtype=F8)
        u = lm.adapters(n.y, a, b, index, base=n.y)
        v = lm.adapters(q.y, a, b, index, base=n.y, x_scales=q.scales)
        h = lm.gated_recurrence_step(u, u, v, decay, state)
        p = lm.gated_recurrence(rows, rows, rows, decay, return_state=True, save=True)
        back = lm.gated_recurrence_backward(rows, rows, rows, rows, decay, saved=p.saved)
        f = lm.rms_norm(x, w, save=True)
        return [n.residual, u, v, h, p.y, p.state, back.dx, back.ddecay, lm.rms_norm_backward(u, x, w, f.rstd).dw]

    eager, want = start.clone(), []
    for v in ins:
        want.append([t.clone() for t in layer(*v, eager)])
    state, live = start.clone(), [t.clone() for t in ins[0]]
    live[3] = ins[0][3].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*live, start.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(*live, state)
    state.copy_(start)
    for k, v in enumerate(ins):
        for t, u in zip(live, v):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(out, want[k])), k
        torch.empty(1 << 20, device="cuda").fill_(float(k))
    assert torch.equal(state, eager)


@pytest.mark.parametrize("e", [5, 80])
def test_two_streams_at_once(e):
    """Long recurrences and adapters of many rows on two streams beside each other."""
    g = gen(44)
    x = rnd(g, 1, 20000, 192, dtype=BF).transpose(1, 2)
    decay, index = rnd(g, 192) - 5, torch.randint(-1, e, (3000,), generator=g).to(torch.int32).cuda()
    rows, a, b = rnd(g, 3000, 256, dtype=BF), rnd(g, e, 16, 256, dtype=BF), rnd(g, e, 300, 16, dtype=BF)
    want = lm.gated_recurrence(x, x, x, decay).y, lm.adapters(rows, a, b, index)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                out.append((lm.gated_recurrence(x, x, x, decay).y, lm.adapters(rows, a, b, index)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in out for p, q in zip(o, want))


# ---------------------------------------------------------- any order, many --

@pytest.mark.parametrize("dt,m,e,rank", [(BF, 1500, 300, 8), (HF, 520, 3, 20), (F, 1300, 1100, 6), (BF, 4000, 5, 100),
                                            (BF, 2000, 63, 8), (HF, 1000, 64, 8), (F, 8192, 10, 4), (BF, 8193, 10, 4), (HF, 600, 1, 16)])
def test_adapters_of_many_rows_in_any_order(dt, m, e, rank):
    """More adapters than one turn of the sort holds, many rows of one adapter,
    many adapters of one row: rows in any order get what each alone would."""
    g = gen(m)
    x, a, b = rnd(g, m, 40, dtype=dt), rnd(g, e, rank, 40, dtype=dt), rnd(g, e, 30, rank, dtype=dt)
    base, scaling = rnd(g, m, 30, dtype=dt), torch.rand(e, generator=g).cuda()
    index = torch.randint(-2, e + 2, (m,), generator=g)
    index[::7] = e // 2
    index = index.to(torch.int32).cuda()
    got = lm.adapters(x, a, b, index, base=base, scaling=scaling)
    y, bound = Y.adapters(x, a, b, index, base=base, scaling=scaling)
    R.assert_close(got, y, bound, 40 + rank + 64, "y")
    some = torch.randperm(m, generator=g)[:500].cuda()   # the same rows by the other way to find them
    R.assert_close(lm.adapters(x[some], a, b, index[some], base=base[some], scaling=scaling), y[some.cpu()], bound[some.cpu()], 40 + rank + 64, "some")
    assert torch.equal(got, lm.adapters(x, a, b, index, base=base, scaling=scaling))


def test_views_and_broadcasts():
    """Slices of one projection, gates shared by the batch, gradients of a
    broadcast output, norms of slices."""
    g = gen(45)
    n, c, l = 2, 24, 140
    big = rnd(g, n, l, 3 * c + 5, dtype=BF).transpose(1, 2)
    x, r, i = big[:, 1:c + 1], big[:, c + 2:2 * c + 2], big[:, 2 * c + 3:3 * c + 3]
    decay = torch.full((1,), -4.0, device="cuda").expand(c)
    dense = [v.clone(memory_format=torch.contiguous_format) for v in (x, r, i)]
    got, want = lm.gated_recurrence(x, r, i, decay, return_state=True), lm.gated_recurrence(*dense, decay.contiguous(), return_state=True)
    assert torch.equal(got.y, want.y) and torch.equal(got.state, want.state)
    gy = rnd(g, n, c, 1, dtype=BF).expand(n, c, l)
    shared = rnd(g, 1, c, l, dtype=BF).expand(n, c, l)
    one, two = lm.gated_recurrence_backward(gy, x, shared, i, decay), lm.gated_recurrence_backward(gy.contiguous(), dense[0], shared.contiguous(), dense[2], decay)
    assert all(torch.equal(a, b) for a, b in zip(one[:4], two[:4])) and one.ddecay.shape == (c,)
    w = rnd(g, c, dtype=BF)
    a, b = lm.rms_norm(x, w, residual=shared, save=True), lm.rms_norm(dense[0], w, residual=shared.contiguous(), save=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.residual, b.residual)
    for k, (u, v) in enumerate(zip(lm.rms_norm_backward(gy, a.residual, w, a.rstd), lm.rms_norm_backward(gy.contiguous(), b.residual, w, b.rstd))):
        R.assert_close(u, v.double().cpu(), v.double().abs().cpu() + (gy.abs().sum().double().cpu() if k else 0), 600, "gradients")
    cut = rnd(g, 6, 50, dtype=BF)
    assert torch.equal(lm.rms_norm(cut[:, 3:40], w[:1].expand(37)).y, lm.rms_norm(cut[:, 3:40].contiguous(), w[:1].expand(37).contiguous()).y)


def test_rows_behind_the_last_sequence_stay():
    """Offsets that end before the rows do: what lies behind is not written."""
    g = gen(46)
    x = rnd(g, 1, 300, 40, dtype=BF).transpose(1, 2)
    decay, off = rnd(g, 40) - 4, torch.tensor([0, 30, 170], dtype=torch.int32, device="cuda")
    for chunk in (None, 128):
        y = torch.full_like(x, 9.0)
        lm._call(lm.A.LM_GATED, [(lm._X, x), (lm._A, x), (lm._B, x), (lm._D, decay), (lm._OFF, off)], [(lm._Y, y)], 0, None, chunk, 8.0)
        assert bool((y[:, :, 170:] == 9).all())
        assert torch.equal(y[:, :, :170], lm.gated_recurrence(x[:, :, :170], x[:, :, :170], x[:, :, :170], decay, offsets=off, chunk=chunk).y)


def test_refusals_on_the_device():
    x = torch.zeros(1, 8, 4, device="cuda")
    with pytest.raises(ValueError, match="GPU only"):
        lm.gated_recurrence(x, x, x, torch.zeros(8))
    with pytest.raises(RuntimeError, match="element type"):
        lm.rms_norm(x, torch.zeros(8, device="cuda", dtype=HF))
    with pytest.raises(RuntimeError, match="rank 300"):
        lm.adapters(x, torch.zeros(2, 300, 8, device="cuda"), torch.zeros(2, 5, 300, device="cuda"), torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):   # a base that is y in another order
        y = torch.zeros(4, 4, device="cuda")
        lm.adapters(torch.zeros(4, 8, device="cuda"), torch.zeros(2, 8, 8, device="cuda"), torch.zeros(2, 4, 8, device="cuda"),
                    torch.zeros(4, dtype=torch.int32, device="cuda"), base=y.t(), out=y)
