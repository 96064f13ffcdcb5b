"""Host logic of the gated recurrence, the RMS norm and the adapters, on the
CPU: what lm_plan accepts and refuses, lm_run's own checks, and what the binding
allocates and hands over.  ``calls`` stands in for the launch."""
import ctypes

import pytest
import torch

from depthwise_stencil_implicit_amd import _abi as A
from depthwise_stencil_implicit_amd import lm
from test_lm_boundary import status
from test_lm_calls import calls, default_dtype  # noqa: F401  fixtures

BF, HF, F, F8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32


def e(*shape, d=BF):
    return torch.empty(shape, dtype=d)


def gated(n=2, c=8, l=10, dtype=BF, step=False):
    s = (n, c) if step else (n, c, l)
    t = {lm._X: e(*s, d=dtype), lm._A: e(*s, d=dtype), lm._B: e(*s, d=dtype), lm._D: e(c, d=F), lm._Y: e(*s, d=dtype)}
    return {**t, lm._S1 if step else lm._S0: e(n, c, d=F)}


def gated_bwd(n=2, c=8, l=10, dtype=BF):
    t = gated(n, c, l, dtype)
    x = t[lm._X]
    return {lm._X: x, lm._A: x, lm._B: x, lm._D: t[lm._D], lm._GY: x, lm._DX: x, lm._DA: x, lm._DB: x, lm._DD: e(c, d=F),
            lm._SAVED: lm._new_gated_saved(x, None)}


def norm(n=3, c=64, l=5, dtype=BF, f8=False, g=1):
    t = {lm._X: e(n, c, l, d=dtype), lm._W: e(c, d=dtype), lm._S0: e(n, c, l, d=dtype), lm._S1: e(n, c, l, d=dtype),
         lm._Y: e(n, c, l, d=F8 if f8 else dtype), lm._SAVED: e(n, l, d=F)}
    return {**t, lm._SCALES: e(n, g, l, d=F)} if f8 else t


def norm_bwd(n=3, c=64, dtype=BF):
    return {lm._X: e(n, c, d=dtype), lm._GY: e(n, c, d=dtype), lm._W: e(c, d=dtype), lm._SAVED: e(n, d=F), lm._GS: e(n, c, d=dtype),
            lm._DX: e(n, c, d=dtype), lm._DW: e(c, d=dtype)}


def adapt(m=4, k=64, n=48, r=8, a=3, dtype=BF, f8=False):
    t = {lm._X: e(m, k, d=F8 if f8 else dtype), lm._A: e(a, r, k, d=dtype), lm._B: e(a, n, r, d=dtype), lm._ROWS: e(m, d=I32),
         lm._Z: e(m, n, d=dtype), lm._D: e(a, d=F), lm._Y: e(m, n, d=dtype)}
    return {**t, lm._SCALES: e(m, 1, d=F)} if f8 else t


def test_plans_of_plain_calls():
    for dt in (BF, HF, F):
        assert status(A.LM_GATED, gated(dtype=dt), value=8.0) == A.OK
        assert status(A.LM_GATED_BWD, gated_bwd(dtype=dt), value=8.0) == A.OK
        assert status(A.LM_GATED_STEP, gated(dtype=dt, step=True), value=8.0) == A.OK
        for f8 in (False, True):
            assert status(A.LM_NORM, norm(dtype=dt, f8=f8), value=1e-6) == A.OK
            assert status(A.LM_ADAPTERS, adapt(dtype=dt, f8=f8)) == A.OK
        assert status(A.LM_NORM_BWD, norm_bwd(dtype=dt)) == A.OK
    # A long row with few channels is split, a wide batch is not.
    assert lm._make_plan(A.LM_GATED, gated(n=1, c=64, l=9000), value=8.0).chunks > 8
    assert lm._make_plan(A.LM_GATED, gated(n=32, c=2048, l=200), value=8.0).chunks == 1
    # What gated_recurrence allocates for saved states is what the plan asks for.
    for n, l, lens in ((2, 65, None), (1, 500, [0, 17, 300]), (1, 64, [64]), (3, 1, None), (1, 0, [0])):
        t = gated(n=n, l=l)
        t.pop(lm._S0)
        t[lm._OFF] = e(len(lens) + 1, d=I32) if lens else None
        t[lm._SAVED] = lm._new_gated_saved(t[lm._X], t[lm._OFF])
        assert status(A.LM_GATED, t, value=8.0) == A.OK


def x10(d=BF):
    return e(2, 8, 10, d=d)


BAD = [
    (A.LM_GATED, gated, {}, {lm._X: e(2, 8)}, A.EINVAL),                        # rank
    (A.LM_GATED, gated, {}, {lm._X: x10(torch.uint8)}, A.EINVAL),
    (A.LM_GATED, gated, {}, {lm._A: x10(F)}, A.EINVAL),                         # mixed types
    (A.LM_GATED, gated, {}, {lm._B: None}, A.EINVAL),
    (A.LM_GATED, gated, {}, {lm._D: e(8)}, A.EINVAL),                           # decay is f32
    (A.LM_GATED, gated, {}, {lm._D: e(7, d=F)}, A.EINVAL),
    (A.LM_GATED, gated, {}, {lm._S0: e(3, 8, d=F)}, A.EINVAL),
    (A.LM_GATED, gated, {}, {lm._S0: e(2, 8)}, A.EINVAL),                       # states are f32
    (A.LM_GATED, gated, {}, {lm._SAVED: e(5, d=F)}, A.EINVAL),
    (A.LM_GATED, gated, {}, {lm._OFF: e(3, d=I32)}, A.EINVAL),                  # packed needs one row
    (A.LM_GATED, gated, {}, {lm._Y: e(2, 8, 1).expand(2, 8, 10)}, A.EINVAL),    # output in one place
    (A.LM_GATED, gated, {}, {lm._W: e(8)}, A.EINVAL),                           # no tensor of this operator
    (A.LM_GATED, gated, dict(value=-1.0), {}, A.EINVAL),
    (A.LM_GATED, gated, dict(value=float("nan")), {}, A.EINVAL),
    (A.LM_GATED, gated, dict(value=float("inf")), {}, A.EINVAL),
    (A.LM_GATED, gated, dict(flags=A.LM_SILU), {}, A.EINVAL),
    (A.LM_GATED, gated, dict(chunk=-1), {}, A.EINVAL),
    (A.LM_GATED_BWD, gated_bwd, {}, {lm._SAVED: None}, A.EINVAL),
    (A.LM_GATED_BWD, gated_bwd, {}, {lm._DX: None}, A.EINVAL),
    (A.LM_GATED_BWD, gated_bwd, {}, {lm._DD: None}, A.EINVAL),
    (A.LM_NORM, norm, {}, {lm._S1: None}, A.EINVAL),                            # a residual in without one out
    (A.LM_NORM, norm, {}, {lm._S0: None}, A.EINVAL),
    (A.LM_NORM, norm, {}, {lm._W: e(64, d=F)}, A.EINVAL),
    (A.LM_NORM, norm, {}, {lm._SCALES: e(3, 1, 5, d=F)}, A.EINVAL),             # scales of a y that has none
    (A.LM_NORM, norm, {}, {lm._Y: e(3, 64, 5, d=F)}, A.EINVAL),
    (A.LM_NORM, norm, {}, {lm._X: e(3, 64, 5, 1)}, A.EINVAL),
    (A.LM_NORM, norm, dict(value=-1.0), {}, A.EINVAL),
    (A.LM_NORM, norm, dict(chunk=4), {}, A.EINVAL),
    (A.LM_NORM, lambda: norm(f8=True), {}, {lm._SCALES: None}, A.EINVAL),
    (A.LM_NORM, lambda: norm(f8=True, g=3), {}, {}, A.EINVAL),                  # 64 / 3
    (A.LM_NORM, lambda: norm(f8=True, g=4), {}, {}, A.EUNSUPPORTED),            # groups of 16
    (A.LM_NORM, lambda: norm(n=1, c=65537, l=1), {}, {}, A.EUNSUPPORTED),
    (A.LM_NORM, lambda: norm(c=0), {}, {}, A.EINVAL),
    (A.LM_NORM_BWD, norm_bwd, {}, {lm._SAVED: None}, A.EINVAL),
    (A.LM_NORM_BWD, norm_bwd, {}, {lm._DX: None, lm._DW: None, lm._GS: None}, A.EINVAL),
    (A.LM_NORM_BWD, norm_bwd, {}, {lm._DX: None}, A.EINVAL),                    # gstate without dx
    (A.LM_ADAPTERS, adapt, {}, {lm._ROWS: e(4, d=F)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._ROWS: e(8, d=I32)[::2]}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._ROWS: e(5, d=I32)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._A: e(3, 8, 60)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._B: e(2, 48, 8)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._B: e(3, 48, 8, d=F)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._D: e(3)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._Z: e(4, 47)}, A.EINVAL),
    (A.LM_ADAPTERS, adapt, {}, {lm._SCALES: e(4, 1, d=F)}, A.EINVAL),           # scales of an x that has none
    (A.LM_ADAPTERS, lambda: adapt(f8=True), {}, {lm._SCALES: None}, A.EINVAL),
    (A.LM_ADAPTERS, lambda: adapt(f8=True), {}, {lm._SCALES: e(4, 2, d=F)}, A.EINVAL),
    (A.LM_ADAPTERS, lambda: adapt(r=257), {}, {}, A.EUNSUPPORTED),
    (A.LM_ADAPTERS, lambda: adapt(r=0), {}, {}, A.EUNSUPPORTED),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    op, make, kw, change, want = BAD[i]
    assert status(op, {**make(), **change}, **{"value": 1.0, **kw}) == want


@pytest.mark.parametrize("op,make", [
    (A.LM_GATED, lambda v: {**gated(1, 1, 1), **{k: v(1 << 22, 8192, 1) for k in (lm._X, lm._A, lm._B, lm._Y)}, lm._D: v(8192, d=F), lm._S0: None}),
    (A.LM_GATED_STEP, lambda v: {**{k: v(1 << 20, 16384) for k in (lm._X, lm._A, lm._B, lm._Y)}, lm._D: v(16384, d=F), lm._S1: v(1 << 20, 16384, d=F)}),
    (A.LM_NORM, lambda v: {lm._X: v(1 << 26, 64), lm._W: v(64), lm._Y: v(1 << 26, 64)}),
    (A.LM_ADAPTERS, lambda v: {lm._X: v(1 << 31, 64), lm._A: v(2, 8, 64), lm._B: v(2, 8, 8), lm._ROWS: v(1 << 31, d=I32), lm._Y: v(1 << 31, 8)}),
    (A.LM_ADAPTERS, lambda v: {lm._X: v(1 << 30, 64), lm._A: v(2, 8, 64), lm._B: v(2, 16, 8), lm._ROWS: v(1 << 30, d=I32), lm._Y: v(1 << 30, 16)}),
])
def test_refuses_what_one_launch_cannot_hold(op, make):
    t = make(lambda *s, d=BF: torch.empty(s, dtype=d, device="meta"))
    with pytest.raises(lm.ConvError, match="one launch") as r:
        lm._make_plan(op, t, value=1.0)
    assert r.value.status == A.EUNSUPPORTED


@pytest.mark.parametrize("rows,C", [(1 << 23, 64), (1 << 25, 2048), (16 << 20, 4096)])
def test_norms_of_many_rows(rows, C):
    """As many as a launch of their threads holds."""
    m = lambda *s: torch.empty(s, dtype=BF, device="meta")  # noqa: E731
    lm._make_plan(A.LM_NORM, {lm._X: m(rows - 1, C), lm._W: m(C), lm._Y: m(rows - 1, C)}, value=1.0)


@pytest.mark.parametrize("chunk", [101, 1 << 40, (1 << 63) - 40, (1 << 63) - 1])
def test_a_chunk_longer_than_the_axis(chunk):
    p = lm._make_plan(A.LM_GATED, gated(l=100), chunk=chunk, value=8.0)
    assert p.chunks == 1 and 100 <= p.chunk <= 128 and p.workspace_bytes == 0
    assert lm._make_plan(A.LM_GATED, gated(n=1, l=0), chunk=chunk, value=8.0).chunks == 1


@pytest.mark.parametrize("seqs,t,c,max_len", [(256, 16384, 4096, 0), (2000, 32768, 512, 30000), (64, 65536, 4096, 32768)])
def test_packed_workspace_follows_the_rows(seqs, t, c, max_len):
    m = lambda *s, d=BF: torch.empty(s, dtype=d, device="meta")  # noqa: E731
    x = m(1, c, t)
    ins = {lm._X: x, lm._A: x, lm._B: x, lm._D: m(c, d=F), lm._OFF: m(seqs + 1, d=I32)}
    p = lm._make_plan(A.LM_GATED, {**ins, lm._Y: x}, max_len=max_len, value=8.0)
    assert p.workspace_bytes <= (t // p.chunk + seqs) * 16 * c + 2 * c
    p = lm._make_plan(A.LM_GATED_BWD, {**ins, lm._GY: x, lm._DX: x, lm._DA: x, lm._DB: x, lm._DD: m(c, d=F),
                                       lm._SAVED: m((t // 64 + seqs + 1) * c, d=F)}, max_len=max_len, value=8.0)
    assert p.workspace_bytes <= (t // p.chunk + seqs) * 12 * c


def test_run_checks_pointers_before_any_device_call():
    for op, t in ((A.LM_GATED, gated()), (A.LM_NORM, norm(f8=True)), (A.LM_ADAPTERS, adapt())):
        p = lm._make_plan(op, t, value=1.0)
        q = lm._Ptrs()
        run = lambda ws=None, n=0: A.lib().lm_run(ctypes.byref(p), q, ws, n, None)  # noqa: E731
        assert run() == A.EINVAL
        for k, v in t.items():
            q[k] = v.data_ptr()
        q[lm._X] = t[lm._X].data_ptr() + 1
        assert run() == A.EALIGN
        q[lm._X] = t[lm._X].data_ptr()
        q[lm._GY] = t[lm._X].data_ptr()
        assert run() == A.EINVAL                                                # a pointer for an absent tensor
        q[lm._GY] = None
        if p.workspace_bytes:
            assert run() == A.EINVAL
    # A base that is y itself has y's strides.
    y = e(8, 48)
    t = {**adapt(), lm._Y: y[:4], lm._Z: y[::2]}
    p, q, ws = lm._make_plan(A.LM_ADAPTERS, t), lm._Ptrs(), torch.empty(1 << 20, dtype=torch.uint8)
    for k, v in t.items():
        q[k] = v.data_ptr()
    at = -(-ws.data_ptr() // 256) * 256
    assert p.workspace_bytes < (1 << 20) - 256
    assert A.lib().lm_run(ctypes.byref(p), q, at, p.workspace_bytes, None) == A.EINVAL


def test_outputs_of_calls(calls, default_dtype):  # noqa: F811
    """Shapes, types and memory order of what the calls allocate, under any
    default type."""
    default_dtype(torch.float64)
    x = e(2, 100, 64).transpose(1, 2)                                           # 100 rows of 64 channels
    r = lm.rms_norm(x, e(64), residual=x, out_dtype=F8, group=32, save=True)
    assert r.y.dtype == F8 and r.y.stride() == x.stride() and r.residual.dtype == BF and r.residual.stride() == x.stride()
    assert r.scales.shape == (2, 2, 100) and r.scales.stride() == (200, 1, 2) and r.scales.dtype == F
    assert r.rstd.shape == (2, 100) and r.rstd.dtype == F
    r = lm.rms_norm(e(3, 64), e(64))
    assert r.y.shape == (3, 64) and r.residual is r.scales is r.rstd is None
    y = lm.adapters(e(2, 100, 64, d=F8).transpose(1, 2), e(3, 8, 64), e(3, 40, 8), e(2, 100, d=I32), x_scales=e(2, 1, 100, d=F))
    assert y.shape == (2, 40, 100) and y.stride() == (4000, 1, 40) and y.dtype == BF
    out = lm.gated_recurrence(x, x, x, e(64, d=F), return_state=True, save=True)
    assert out.y.stride() == x.stride() and out.state.dtype == out.saved.dtype == F and out.state.shape == (2, 64)
    g = lm.gated_recurrence_backward(x, x, x, x, e(64, d=F), state=e(2, 64, d=F))
    assert g.dstate.shape == (2, 64) and g.ddecay.dtype == F
    assert lm.gated_recurrence_step(e(3, 8), e(3, 8), e(3, 8), e(8, d=F), e(3, 8, d=F)).shape == (3, 8)


def test_values_are_part_of_the_plan(calls):  # noqa: F811
    x, w = e(3, 64), e(64)
    for eps in (1e-6, 1e-5, 1e-6):
        lm.rms_norm(x, w, eps=eps)
    assert [round(c[0].args.value * 1e6) for c in calls] == [1, 10, 1] and len(lm._plans) == 2


def test_arguments(calls):  # noqa: F811
    with pytest.raises(ValueError, match="out_dtype"):
        lm.rms_norm(e(3, 64), e(64), out_dtype=torch.int8)
    with pytest.raises(ValueError, match="groups of"):
        lm.rms_norm(e(3, 64), e(64), group=32)
    with pytest.raises(ValueError, match="groups of"):
        lm.rms_norm(e(3, 64), e(64), out_dtype=F8, group=48)
    with pytest.raises(ValueError, match="dims"):
        lm.rms_norm(e(64), e(64))
    with pytest.raises(TypeError, match="unsupported dtype"):
        lm.adapters(e(4, 64), e(3, 8, 64), e(3, 40, 8), e(4, d=torch.int64))
    for x, a in ((e(64), e(3, 8, 64)), (e(4, 64), e(8, 64))):
        with pytest.raises(lm.ConvError, match="dims"):
            lm.adapters(x, a, e(3, 40, 8), e(4, d=I32))
    with pytest.raises(lm.ConvError, match="rows"):
        lm.gated_recurrence_step(e(3, 8), e(3, 8), e(3, 8), e(8, d=F), e(5, 8, d=F))
    assert not calls


def test_every_call_refuses_host_memory():
    x, d, st = torch.zeros(2, 8, 5), torch.zeros(8), torch.zeros(2, 8)
    one = (x[:, :, 0], x[:, :, 0], x[:, :, 0], d, st)
    ad = (torch.zeros(2, 8), torch.zeros(3, 4, 8), torch.zeros(3, 6, 4), torch.zeros(2, dtype=I32))
    for call in (lambda: lm.gated_recurrence(x, x, x, d, save=True), lambda: lm.gated_recurrence_backward(x, x, x, x, d),
                 lambda: lm.gated_recurrence_step(*one), lambda: lm.PreparedGatedRecurrenceStep(*one), lambda: lm.rms_norm(x, d),
                 lambda: lm.rms_norm_backward(x, x, d, torch.zeros(2, 5)), lambda: lm.PreparedRmsNorm(x, d),
                 lambda: lm.adapters(*ad), lambda: lm.PreparedAdapters(*ad)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


def test_norm_gradients_take_the_calls_residual(calls):  # noqa: F811
    t = norm_bwd()
    assert status(A.LM_NORM_BWD, {**t, lm._S0: e(3, 64)}, value=1e-6) == A.OK
    for bad in (e(3, 64, d=F), e(3, 63), e(2, 64), e(3, 64, 1)):
        assert status(A.LM_NORM_BWD, {**t, lm._S0: bad}, value=1e-6) == A.EINVAL
    x, w, rstd = e(3, 64), e(64), e(3, d=F)
    lm.rms_norm_backward(x, x, w, rstd, residual=e(3, 128)[:, ::2])
    lm.rms_norm_backward(x, x, w, rstd)
    assert [c[0].t[lm._S0].rank for c in calls] == [2, 0] and calls[0][0].t[lm._S0].strides[1] == 2


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("n,c,fits", [(1 << 20, 8191, False), (1 << 20, 8193, False), ((1 << 20) + 1, 8192, False), ((1 << 20) - 1, 8192, True),
                                      (1 << 19, 8191, True), (1 << 30, 3, True), (1 << 30, 5, False)])
def test_steps_that_one_launch_holds(dtype, n, c, fits):
    """An even number of channels takes two a thread, an odd number one, of any
    type and memory order: fewer than 2^32 threads either way."""
    v = lambda *s, d=dtype: torch.empty(s, dtype=d, device="meta")  # noqa: E731
    for x in (v(n, c), v(c, n).t()):
        t = {**{k: x for k in (lm._X, lm._A, lm._B, lm._Y)}, lm._D: v(c, d=F), lm._S1: v(n, c, d=F)}
        if fits:
            lm._make_plan(A.LM_GATED_STEP, t, value=1.0)
        else:
            with pytest.raises(lm.ConvError, match="one launch") as r:
                lm._make_plan(A.LM_GATED_STEP, t, value=1.0)
            assert r.value.status == A.EUNSUPPORTED


@pytest.mark.parametrize("m,e,parts", [(513, 1000, 4), (1024, 1000, 4), (2048, 2000, 2), (513, 6, 16), (8192, 6, 2), (8192, 1000, 2), (512, 1000, 1)])
def test_many_adapters_count_as_workgroups(m, e, parts):
    """Tiles of a row or two each are many workgroups: their columns are not
    split further, as those of few tiles are, and the sums in the workspace stay few."""
    v = lambda *s, d=BF: torch.empty(s, dtype=d, device="meta")  # noqa: E731
    p = lm._make_plan(A.LM_ADAPTERS, {lm._X: v(m, 4096), lm._A: v(e, 16, 4096), lm._B: v(e, 4096, 16), lm._ROWS: v(m, d=I32), lm._Y: v(m, 4096)})
    assert p.chunks <= parts and p.chunks >= parts // 2
    tiles = m // 64 + min(m, e + 1)   # listed with a place, an adapter and 64 rows each
    assert p.workspace_bytes <= 4 * m * parts * 32 + tiles * (16 + 64 * 4) + 1024
