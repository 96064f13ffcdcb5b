"""What the binding of the sequence operators hands to the library, on the CPU:
the outputs it allocates and the plans it keeps.  ``calls`` stands in for the
launch and records each call's plan and tensors."""
import contextlib
import ctypes

import pytest
import torch

from depthwise_stencil_implicit_amd import _abi as A
from depthwise_stencil_implicit_amd import lm

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """A list that receives (plan, {place: pointer}) of every call; CPU tensors
    count as ones of device 0."""
    made = []
    monkeypatch.setattr(lm, "_plans", {})
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(lm, "_run", lambda p, q, *rest: made.append((p, {i: v for i, v in enumerate(q) if v})))
    return made


@pytest.fixture
def default_dtype():
    before = torch.get_default_dtype()
    yield torch.set_default_dtype
    torch.set_default_dtype(before)


def scan_args(n=2, c=8, l=20, s=16, dtype=F):
    e = lambda *v: torch.zeros(v, dtype=dtype)  # noqa: E731
    return e(n, c, l), e(n, c, l), torch.zeros(c, s, dtype=F), e(n, 1, s, l), e(n, 1, s, l)


@pytest.mark.parametrize("other", [BF, HF, torch.float64])
def test_states_are_f32_under_any_default_type(calls, default_dtype, other):
    """The kernels write f32 states; their memory must not follow torch's
    default type, neither with a new plan nor with a kept one."""
    args = scan_args()
    for kind in (F, other, other):
        default_dtype(kind)
        out = lm.selective_scan(*args, return_state=True, save=True)
        assert out.state.dtype == F and out.saved.dtype == F
        lm.selective_scan_backward(args[0], *args)
    for s in (1, 12, 20, 64):
        x, _, a, _, _ = scan_args(s=s)
        assert lm._new_saved(x, a, None).dtype == F


def test_a_kept_plan_serves_only_its_own_outputs(calls, monkeypatch):
    """dstate has the state's type and layout: a state that the kept plan was
    not made for is checked anew, and one elsewhere is refused."""
    args, gy = scan_args(), torch.zeros(2, 8, 20)
    state = torch.zeros(2, 8, 16)
    lm.selective_scan_backward(gy, *args, state=state, saved=lm._new_saved(args[0], args[2], None))
    saved = lm._new_saved(args[0], args[2], None)
    for other in (BF, HF):
        with pytest.raises(lm.ConvError, match="element type"):
            lm.selective_scan_backward(gy, *args, state=state.to(other), saved=saved)
    turned = torch.zeros(2, 16, 8).transpose(1, 2)
    lm.selective_scan_backward(gy, *args, state=turned, saved=saved)
    assert list(calls[-1][0].t[lm._DS].strides[:3]) == [128, 1, 8]
    made = len(calls)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: -1 if self.dim() == 3 and self.shape[2] == 16 else 0)
    with pytest.raises(ValueError, match="GPU only"):
        lm.selective_scan_backward(gy, *args, state=state, saved=saved)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1 if self.dim() == 3 and self.shape[2] == 16 else 0)
    with pytest.raises(ValueError, match="cuda:0 and cuda:1"):
        lm.selective_scan_backward(gy, *args, state=state, saved=saved)
    assert len(calls) == made


def test_prepared_calls_allocate_on_the_stream_they_launch_on(monkeypatch):
    """The output and the workspace of ``run(stream=...)`` belong to that
    stream: the current one's next tensor could else take their memory while
    the kernels still use it."""
    here, log = [7], []

    @contextlib.contextmanager
    def stream(s):
        before, here[0] = here[0], s
        yield
        here[0] = before

    class Fake(lm._Step):
        def __init__(self):
            self.plan, self.device = None, torch.device("cuda", 0)

        def empty_output(self):
            log.append(("output", here[0]))
            return torch.zeros(1)

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: here[0], raising=False)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device: s)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: 0)
    monkeypatch.setattr(lm, "_run", lambda *a: log.append(("launch", here[0])))
    for given, used in ((None, 7), (7, 7), (9, 9), (0, 0)):
        log.clear()
        q, y = lm._Ptrs(), Fake()._launch
        out = y(q, None, given)
        assert log == [("output", used), ("launch", used)] and q[lm._Y] == out.data_ptr() and here == [7]
        log.clear()
        mine = torch.zeros(1)
        assert y(q, mine, given) is mine and q[lm._Y] == mine.data_ptr() and log == [("launch", used)]


def test_steps_by_name_plan_once(calls, monkeypatch):
    """A decoding loop calls them once per token and layer: only the first call
    of a shape checks and plans."""
    plans, make = [], lm._make_plan
    monkeypatch.setattr(lm, "_make_plan", lambda *a, **k: plans.append(a) or make(*a, **k))
    x, w, st = torch.zeros(3, 8), torch.zeros(8, 4), torch.zeros(3, 8, 3)
    dt, a, bc, h = torch.zeros(3, 8), torch.zeros(8, 16), torch.zeros(3, 16), torch.zeros(3, 8, 16)
    packed, scales, wide = torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(5, 2), torch.zeros(2, 3, 64)
    for call in (lambda: lm.causal_conv_step(x, w[:, None], None, st, activation="silu"),
                 lambda: lm.selective_scan_step(x, dt, a, bc, bc, h, dt_softplus=True),
                 lambda: lm.matvec4(wide, packed, scales)):
        plans.clear()
        out = [call() for _ in range(3)]
        assert len(plans) == 1 and len(calls) == 3, call
        assert all(o.shape == out[0].shape and o.is_contiguous() for o in out)
        assert calls[2][1][lm._Y] == out[2].data_ptr()
        calls.clear()
    assert out[0].shape == (2, 3, 5)
    # Other rows of the same table are another call, an absent bias too.
    lm.causal_conv_step(x, w, torch.zeros(8), st)
    lm.causal_conv_step(x, w, torch.zeros(8), st, rows=torch.zeros(3, dtype=torch.int32))
    assert lm._BIAS in calls[0][1] and lm._ROWS not in calls[0][1] and lm._ROWS in calls[1][1]


def test_steps_by_name_refuse(calls):
    x, w, st = torch.zeros(3, 8), torch.zeros(8, 4), torch.zeros(3, 8, 3)
    with pytest.raises(TypeError, match="unsupported dtype"):
        lm.causal_conv_step(x, w, None, st, rows=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(lm.ConvError, match="rows"):
        lm.causal_conv_step(x, w, None, torch.zeros(5, 8, 3))
    with pytest.raises(lm.ConvError, match="groups"):
        lm.matvec4(torch.zeros(1, 64), torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(5, 3))
    assert not calls


def packed(op, seqs, t, c, s=16, max_len=0):
    """The plan of a packed call of bf16 rows, with nothing behind its descriptors."""
    rows = lambda *v, d=BF: torch.empty(v, dtype=d, device="meta")  # noqa: E731
    x, off = rows(1, c, t), rows(seqs + 1, d=torch.int32)
    if op == A.LM_CONV_BWD:
        w = rows(c, 4)
        return lm._make_plan(op, {lm._X: x, lm._GY: x, lm._W: w, lm._BIAS: rows(c), lm._OFF: off, lm._DX: x, lm._DW: w, lm._DBIAS: rows(c)},
                             max_len=max_len)
    bc, a = rows(1, 1, s, t), rows(c, s, d=F)
    ins = {lm._X: x, lm._DT: x, lm._A: a, lm._B: bc, lm._C: bc, lm._OFF: off}
    if op == A.LM_SCAN:
        return lm._make_plan(op, {**ins, lm._Y: x}, max_len=max_len)
    ck, w = (16, 16) if s <= 16 else (8, 32)
    saved = rows((t // ck + seqs + 1) * c * w, d=F)
    return lm._make_plan(op, {**ins, lm._GY: x, lm._DX: x, lm._DDT: x, lm._DA: a, lm._DB: bc, lm._DC: bc, lm._SAVED: saved}, max_len=max_len)


@pytest.mark.parametrize("op,seqs,t,c,max_len", [
    (A.LM_CONV_BWD, 256, 16384, 4096, 0), (A.LM_CONV_BWD, 64, 65536, 4096, 32768), (A.LM_CONV_BWD, 1000, 65536, 1024, 65536),
    (A.LM_SCAN, 256, 16384, 1024, 0), (A.LM_SCAN, 2000, 32768, 512, 30000), (A.LM_SCAN_BWD, 256, 16384, 1024, 0)])
def test_packed_workspace_follows_the_rows(op, seqs, t, c, max_len):
    """However long the longest sequence may be, all of them have at most
    t / chunk + seqs chunks, and the workspace holds one part for each."""
    p = packed(op, seqs, t, c, max_len=max_len)
    places = t // p.chunk + seqs
    per = {A.LM_CONV_BWD: 5, A.LM_SCAN: 17, A.LM_SCAN_BWD: 18 + 17}[op] * c * 4
    whole = 4 * -(-c // 64) * t * 2 * 16 if op == A.LM_SCAN_BWD else 0   # dB and dC of each 64 channels
    assert p.workspace_bytes <= whole + places * per + 64


@pytest.mark.parametrize("op,shape", [
    # Rows x what each of them gets threads for, 2^32 of them or more in one dimension of a grid.
    ("scan", (1 << 17, 4096, 1, 16, 1)), ("scan", (1 << 23, 64, 1, 16, 1)), ("scan_bwd", (1 << 18, 64, 64, 64, 2)),
    ("scan_bwd", (1 << 17, 4096, 1, 16, 1)), ("scan_step", (1 << 20, 1024, 1, 16, 1)), ("conv_step", (1 << 20, 8192)),
    ("conv", (1 << 24, 16384, 1)), ("conv_bwd", (1 << 20, 8192, 1)), ("mv4", (1, 64, 1 << 28))])
def test_refuses_what_one_launch_cannot_hold(op, shape):
    """A grid counts its threads in 32 bits: such calls are refused when they
    are planned, before any kernel of theirs runs."""
    e = lambda *v, d=BF: torch.empty(v, dtype=d, device="meta")  # noqa: E731
    if op == "mv4":
        m, k, n = shape
        code, t = A.LM_MV4, {lm._X: e(m, k), lm._W: e(n, k // 2, d=torch.uint8), lm._SCALES: e(n, 2), lm._Y: e(m, n)}
    elif op.startswith("conv"):
        x, (n, c) = e(*shape), shape[:2]
        w = e(c, 4)
        code, t = {"conv": (A.LM_CONV, {lm._Y: x}), "conv_step": (A.LM_CONV_STEP, {lm._Y: x, lm._S1: e(n, c, 3)}),
                   "conv_bwd": (A.LM_CONV_BWD, {lm._GY: x, lm._DX: x, lm._DW: w})}[op]
        t |= {lm._X: x, lm._W: w}
    else:
        n, c, l, s, g = shape
        x = e(n, c) if op == "scan_step" else e(n, c, l)
        bc, a = e(n, g, s) if op == "scan_step" else e(n, g, s, l), e(c, s, d=F)
        code, t = {"scan": (A.LM_SCAN, {lm._Y: x}), "scan_step": (A.LM_SCAN_STEP, {lm._Y: x, lm._S1: e(n, c, s, d=F)}),
                   "scan_bwd": (A.LM_SCAN_BWD, {lm._GY: x, lm._DX: x, lm._DDT: x, lm._DA: a, lm._DB: bc, lm._DC: bc})}[op]
        t |= {lm._X: x, lm._DT: x, lm._A: a, lm._B: bc, lm._C: bc}
        if op == "scan_bwd":
            t[lm._SAVED] = e(n * -(-l // (16 if s <= 16 else 4)) * c * (16 if s <= 16 else 64), d=F)
    with pytest.raises(lm.ConvError, match="one launch") as r:
        lm._make_plan(code, t)
    assert r.value.status == A.EUNSUPPORTED


def conv_and_scan(n=2, c=8, l=100, s=16, offsets=None):
    x, w = torch.zeros(n, c, l), torch.zeros(c, 4)
    bc, a = torch.zeros(n, 1, s, l), torch.zeros(c, s)
    return ((A.LM_CONV, {lm._X: x, lm._W: w, lm._Y: x, lm._OFF: offsets}),
            (A.LM_CONV_BWD, {lm._X: x, lm._GY: x, lm._W: w, lm._DX: x, lm._DW: w, lm._OFF: offsets}),
            (A.LM_SCAN, {lm._X: x, lm._DT: x, lm._A: a, lm._B: bc, lm._C: bc, lm._Y: x, lm._OFF: offsets}))


@pytest.mark.parametrize("chunk", [101, 1 << 40, (1 << 63) - 40, (1 << 63) - 1])
@pytest.mark.parametrize("offsets", [None, torch.zeros(4, dtype=torch.int32)])
def test_a_chunk_longer_than_the_axis(chunk, offsets):
    """One piece per sequence, whatever the forced length: none of the plan's
    numbers overflows."""
    for op, t in conv_and_scan(n=1 if offsets is not None else 2, offsets=offsets):
        p = lm._make_plan(op, t, chunk=chunk)
        assert p.chunks == 1 and 100 <= p.chunk <= 128 and 0 <= p.workspace_bytes < 4096
    for op, t in conv_and_scan(n=1, l=0):
        assert lm._make_plan(op, t, chunk=chunk).chunks == 1


def test_quantize4_takes_any_weight(calls):
    """Transposed and sliced weights of every type; columns that do not make
    pairs or groups are refused."""
    g = torch.Generator().manual_seed(1)
    w = torch.randn(64, 12, generator=g)
    wide = torch.randn(12, 100, generator=g)
    for v in (w.t(), wide[:, 10:74], w.t().to(BF), wide.to(HF)[:, ::1][:, 36:]):
        for symmetric in (True, False):
            got, want = (lm.quantize4(u, 32, symmetric=symmetric, dtype=F) for u in (v, v.contiguous()))
            assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
    for columns, group in ((21, 1), (21, 3), (21, 7), (21, 32), (64, 0), (64, -32), (64, 48), (64, 128)):
        with pytest.raises(ValueError, match=f"{columns} columns"):
            lm.quantize4(torch.zeros(4, columns), group)


def test_refuses_negative_sizes():
    """Through the C entry, where any descriptor may come."""
    d = (A.ConvTensor * A.LM_NSLOT)()
    for place, sizes in ((lm._X, (-2, 8, 10)), (lm._Y, (-2, 8, 10)), (lm._W, (8, 4))):
        d[place].rank, d[place].dtype = len(sizes), A.F32
        for i, s in enumerate(sizes):
            d[place].sizes[i], d[place].strides[i] = s, 1
    p, err = A.LmPlan(), ctypes.create_string_buffer(256)
    assert A.lib().lm_plan(A.LM_CONV, d, ctypes.byref(A.LmArgs()), ctypes.byref(p), err, len(err)) == A.EINVAL
    assert b"negative size" in err.value


def test_every_call_refuses_host_memory():
    """All tensors on the host, before a pointer of theirs goes anywhere."""
    x, w, st = torch.zeros(2, 8, 5), torch.zeros(8, 4), torch.zeros(2, 8, 3)
    dt, a, bc = torch.zeros(2, 8, 5), torch.zeros(8, 16), torch.zeros(2, 16, 5)
    packed, scales = torch.zeros(5, 32, dtype=torch.uint8), torch.zeros(5, 2)
    one = (x[:, :, 0], dt[:, :, 0], a, bc[..., 0], bc[..., 0], torch.zeros(2, 8, 16))
    for call in (lambda: lm.causal_conv(x, w, state=st, return_state=True), lambda: lm.causal_conv_backward(x, x, w, state=st),
                 lambda: lm.causal_conv_step(x[:, :, 0], w, None, st), lambda: lm.selective_scan(x, dt, a, bc, bc, save=True),
                 lambda: lm.selective_scan_backward(x, x, dt, a, bc, bc), lambda: lm.selective_scan_step(*one),
                 lambda: lm.matvec4(torch.zeros(2, 64), packed, scales),
                 lambda: lm.PreparedCausalConvStep(x[:, :, 0], w, None, st), lambda: lm.PreparedSelectiveScanStep(*one),
                 lambda: lm.PreparedMatvec4(torch.zeros(2, 64), packed, scales)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
