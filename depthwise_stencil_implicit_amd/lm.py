"""Sequence operators of language models on the GPU (binding of
include/miconv_lm.h): the short causal convolution, the selective state space
scan, and products with 4-bit weights.

Activations are logical [N, C, L] with any strides, like the convolution's;
channels-last storage (L rows of C channels) is the fast order.  A packed batch
is [1, C, T] with ``offsets`` (int32 on the device, ascending from 0 to T):
sequence s is the rows offsets[s] .. offsets[s+1]-1.  ``max_len`` with it, a
length that few sequences pass, helps to choose how the work is split (without
it they may be as long as T); results and the size of the workspace hold for any
value.

Each operator exists for prompts (``causal_conv``, ``selective_scan``), as its
gradients (``*_backward``) and for single tokens (``*_step``, which update the
state in place).  ``Prepared*`` objects keep the plan of fixed shapes, strides
and types for loops where a call's latency counts; like ``Prepared`` of the
convolution they take tensors of those descriptors and check no more.  Calls by
name keep their plans by the descriptors of all their tensors.

torch provides device memory and the current stream; all arithmetic is in the
library's kernels.  Nothing here records autograd history.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _abi as A
from .api import ConvError, _TORCH_DT

(_X, _W, _BIAS, _Y, _S0, _S1, _OFF, _GY, _GS, _DX, _DW, _DBIAS, _DS, _DT, _A, _B, _C, _D, _Z, _DTB, _DDT, _DA, _DB, _DC,
 _DD, _DZ, _DDTB, _SAVED, _ROWS, _SCALES, _ZEROS) = range(A.LM_NSLOT)
_TYPES = {**_TORCH_DT, torch.int32: A.LM_I32, torch.uint8: A.LM_U8}
_Ptrs = ctypes.c_void_p * A.LM_NSLOT


class ConvOut(NamedTuple):
    y: torch.Tensor
    state: Optional[torch.Tensor]


class ConvGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    db: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]


class ScanOut(NamedTuple):
    y: Optional[torch.Tensor]
    state: Optional[torch.Tensor]
    saved: Optional[torch.Tensor]


class ScanGrads(NamedTuple):
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]


# ------------------------------------------------------------------- plans --

def _make_plan(op, tensors, flags=0, max_len=0, chunk=0) -> A.LmPlan:
    """lm_plan for {place: tensor} (None: absent)."""
    d = (A.ConvTensor * A.LM_NSLOT)()
    for slot, t in tensors.items():
        if t is None:
            continue
        if t.dtype not in _TYPES:
            raise TypeError(f"{A.LM_SLOTS[slot].lower()}: unsupported dtype {t.dtype}")
        if t.dim() > A.MAX_RANK or t.dim() == 0:
            raise ValueError(f"{A.LM_SLOTS[slot].lower()}: 1 to {A.MAX_RANK} dims")
        e = d[slot]
        e.rank, e.dtype = t.dim(), _TYPES[t.dtype]
        for i, (s, st) in enumerate(zip(t.shape, t.stride())):
            e.sizes[i], e.strides[i] = s, st
    args = A.LmArgs(flags, 0, int(max_len or 0), int(chunk or 0))
    p = A.LmPlan()
    err = ctypes.create_string_buffer(256)
    st = A.lib().lm_plan(op, d, ctypes.byref(args), ctypes.byref(p), err, len(err))
    if st != A.OK:
        raise ConvError(st, err.value.decode())
    return p


# Plans by operator, arguments and every tensor's shape, strides and type (host structs only).
_plans: dict = {}


def _call(op, ins, outs, flags=0, max_len=None, chunk=None) -> None:
    """Plan (or its cached copy) and launch of a call on ``ins`` and ``outs``,
    lists of (place, tensor or None).  Outputs are part of the key too: not all
    of them follow from the inputs (dstate from a state that the call does not
    read), and lm_run sees pointers only."""
    key = [op, flags, max_len, chunk]
    dev, q, tensors = None, _Ptrs(), ins + outs
    for slot, t in tensors:
        if t is None:
            key.append(None)
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("the sequence operators run on the GPU only; move tensors to cuda")
            if dev is not None:
                raise ValueError(f"tensors on cuda:{dev} and cuda:{d}")
            dev = d
        key += (t.shape, t.stride(), t.dtype)
        q[slot] = t.data_ptr()
    key = tuple(key)
    p = _plans.get(key)
    if p is None:
        p = _make_plan(op, dict(tensors), flags, max_len, chunk)
        if len(_plans) >= 512:
            _plans.clear()
        _plans[key] = p
    _run(p, q, dev)


def _run(p: A.LmPlan, q, dev: int) -> None:
    """Launch on the device's current stream, which the workspace belongs to."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _run(p, q, dev)
    n = p.workspace_bytes
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    st = A.lib().lm_run(ctypes.byref(p), q, ws.data_ptr() if n else None, n, torch._C._cuda_getCurrentRawStream(dev))
    if st != A.OK:
        raise ConvError(st)


def _new(t) -> torch.Tensor:
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rows_like(n, c, l, ref):
    """[n, c, l] stored as l rows of c channels."""
    return torch.empty_strided((n, c, l), (l * c, 1, c), dtype=ref.dtype, device=ref.device)


def _act(activation) -> int:
    if activation in (None, "none"):
        return 0
    if activation == "silu":
        return A.LM_SILU
    raise ValueError(f"activation {activation!r}: None or 'silu'")


def _taps(w: torch.Tensor) -> torch.Tensor:
    """[C, K] of a depthwise weight [C, 1, K] or [C, K]."""
    return w.squeeze(1) if w.dim() == 3 and w.shape[1] == 1 else w


def _seqs(x, offsets) -> int:
    return x.shape[0] if offsets is None else offsets.shape[0] - 1


# ------------------------------------------------------ causal convolution --

def causal_conv(x, w, b=None, *, activation=None, state=None, offsets=None, max_len=None,
                return_state: bool = False, chunk=None) -> ConvOut:
    """act(bias + causal depthwise convolution of x with w [C, K] (or [C, 1, K])).

    ``state`` [sequences, C, K-1] holds the K-1 values in front of each
    sequence (zeros without it); ``return_state`` gives those in front of what
    follows it.  ``chunk`` forces the rows one thread walks."""
    w = _taps(w)
    y = torch.empty_like(x)
    last = _rows_like(_seqs(x, offsets), x.shape[1], w.shape[-1] - 1, x) if return_state else None
    _call(A.LM_CONV, [(_X, x), (_W, w), (_BIAS, b), (_S0, state), (_OFF, offsets)], [(_Y, y), (_S1, last)], _act(activation),
          max_len, chunk)
    return ConvOut(y, last)


def causal_conv_backward(gy, x, w, b=None, *, activation=None, state=None, offsets=None, max_len=None, gstate=None,
                         need_dx: bool = True, need_dw: bool = True, chunk=None) -> ConvGrads:
    """Gradients of ``causal_conv`` for gy, the gradient of y, and ``gstate``,
    that of the returned state.  db comes with a bias, dstate with a state;
    ``need_dw`` covers dw and db."""
    shape, w = w.shape, _taps(w)
    dx = torch.empty_like(x) if need_dx else None
    dw = _new(w) if need_dw else None
    db = _new(b) if need_dw and b is not None else None
    ds = torch.empty_like(state) if state is not None else None
    _call(A.LM_CONV_BWD, [(_GY, gy), (_X, x), (_W, w), (_BIAS, b), (_S0, state), (_OFF, offsets), (_GS, gstate)],
          [(_DX, dx), (_DW, dw), (_DBIAS, db), (_DS, ds)], _act(activation), max_len, chunk)
    return ConvGrads(dx, dw.view(shape) if dw is not None and len(shape) == 3 else dw, db, ds)


class _Step:
    """A plan whose output is a new contiguous tensor of the plan's shape.

    ``run`` launches on ``stream`` (a raw handle; the current stream without
    one).  A new output belongs to that stream, as if it had been made the
    current one for the call."""

    def __init__(self, op, tensors, shape, ref, flags=0):
        self.device = ref.device
        if any(t is not None and not t.is_cuda for t in tensors.values()):
            raise ValueError("the sequence operators run on the GPU only; move tensors to cuda")
        if any(t is not None and t.device != ref.device for t in tensors.values()):
            raise ValueError("tensors on several devices")
        self.shape, self.dtype = shape, ref.dtype
        self.plan = _make_plan(op, {**tensors, _Y: self.empty_output()}, flags)

    def empty_output(self) -> torch.Tensor:
        return torch.empty(self.shape, dtype=self.dtype, device=self.device)

    def _launch(self, q, y, stream) -> torch.Tensor:
        dev = self.device.index
        if stream is not None and stream != torch._C._cuda_getCurrentRawStream(dev):
            # Memory of the present stream's pool could be given out again
            # there while the kernels use it: allocate on the other stream.
            s = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            with torch.cuda.stream(s):
                return self._launch(q, y, None)
        if y is None:
            y = self.empty_output()
        q[_Y] = y.data_ptr()
        _run(self.plan, q, dev)
        return y


class PreparedCausalConvStep(_Step):
    """The step of ``causal_conv`` for fixed descriptors."""

    def __init__(self, x, w, b, state, *, activation=None, rows=None):
        super().__init__(A.LM_CONV_STEP, {_X: x, _W: _taps(w), _BIAS: b, _S1: state, _ROWS: rows}, tuple(x.shape), x,
                         _act(activation))

    def run(self, x, w, b, state, rows=None, y=None, stream: Optional[int] = None) -> torch.Tensor:
        q = _Ptrs()
        q[_X], q[_W], q[_S1] = x.data_ptr(), w.data_ptr(), state.data_ptr()
        if b is not None:
            q[_BIAS] = b.data_ptr()
        if rows is not None:
            q[_ROWS] = rows.data_ptr()
        return self._launch(q, y, stream)


def causal_conv_step(x, w, b, state, *, activation=None, rows=None) -> torch.Tensor:
    """One token: x [N, C], state [N, C, K-1] updated in place.  With ``rows``
    (int32 [N], distinct) batch row n uses state row rows[n]; a row outside
    the state is left out and its y is zero."""
    y = _new(x)
    _call(A.LM_CONV_STEP, [(_X, x), (_W, _taps(w)), (_BIAS, b), (_S1, state), (_ROWS, rows)], [(_Y, y)], _act(activation))
    return y


# --------------------------------------------------------- selective scan --

def _grouped(v, dims):
    """B or C with its group dim ([N, S, L] is one group)."""
    return v.unsqueeze(1) if v is not None and v.dim() == dims - 1 else v


def selective_scan(x, dt, A_, B, C, *, D=None, z=None, dt_bias=None, dt_softplus: bool = False, state=None, offsets=None,
                   max_len=None, return_state: bool = False, save: bool = False, want_y: bool = True,
                   chunk=None) -> ScanOut:
    """h <- exp(d A) h + d x B,  y = (sum_s C h + D x) silu(z),
    d = dt + dt_bias, or its softplus.

    x, dt, z [N, C, L]; A [C, S], D, dt_bias [C] in f32; B, C [N, G, S, L] (or
    [N, S, L]), channel c using group c // (C // G); ``state`` and the returned
    state f32 [sequences, C, S].  ``save`` returns what ``selective_scan_backward``
    takes as ``saved``.  ``chunk`` forces how many steps run in one piece."""
    B, C = _grouped(B, 4), _grouped(C, 4)
    y = torch.empty_like(x) if want_y else None
    # Their type is said: without it they would have torch's default one.
    last = x.new_empty((_seqs(x, offsets), x.shape[1], A_.shape[-1]), dtype=torch.float32) if return_state else None
    saved = _new_saved(x, A_, offsets) if save else None
    _call(A.LM_SCAN,
          [(_X, x), (_DT, dt), (_A, A_), (_B, B), (_C, C), (_D, D), (_Z, z), (_DTB, dt_bias), (_S0, state), (_OFF, offsets)],
          [(_Y, y), (_S1, last), (_SAVED, saved)], A.LM_SOFTPLUS if dt_softplus else 0, max_len, chunk)
    return ScanOut(y, last, saved)


def _new_saved(x, A_, offsets) -> torch.Tensor:
    """Room for the states before every 16th step (fewer steps above 16 states)."""
    s = A_.shape[-1]
    ns, rows = 1, 4 if s <= 16 else 8
    while rows * ns < s:
        ns *= 2
    ck = 16 if rows == 4 else max(1, 32 // ns)
    count = x.shape[0] * -(-x.shape[2] // ck) if offsets is None else x.shape[2] // ck + offsets.shape[0]
    return torch.empty(count * x.shape[1] * rows * ns, dtype=torch.float32, device=x.device)


def selective_scan_backward(gy, x, dt, A_, B, C, *, D=None, z=None, dt_bias=None, dt_softplus: bool = False, state=None,
                            offsets=None, max_len=None, gstate=None, saved=None, chunk=None) -> ScanGrads:
    """Gradients of ``selective_scan`` for gy, the gradient of y, and
    ``gstate``, that of the returned state.  ``saved`` comes from the forward
    call (``save=True``) on the same tensors; without it the states are computed
    again.  dD, dz, ddt_bias and dstate come with D, z, dt_bias and state."""
    if saved is None:
        saved = selective_scan(x, dt, A_, B, C, D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus, state=state,
                               offsets=offsets, max_len=max_len, save=True, want_y=False, chunk=chunk).saved
    b_shape, c_shape, B, C = B.shape, C.shape, _grouped(B, 4), _grouped(C, 4)
    new = lambda v: torch.empty_like(v) if v is not None else None  # noqa: E731
    dx, ddt, dA, dB, dC = (torch.empty_like(v) for v in (x, dt, A_, B, C))
    dD, dz, db, ds = new(D), new(z), new(dt_bias), new(state)
    _call(A.LM_SCAN_BWD,
          [(_GY, gy), (_X, x), (_DT, dt), (_A, A_), (_B, B), (_C, C), (_D, D), (_Z, z), (_DTB, dt_bias), (_OFF, offsets),
           (_GS, gstate), (_SAVED, saved)],
          [(_DX, dx), (_DDT, ddt), (_DA, dA), (_DB, dB), (_DC, dC), (_DD, dD), (_DZ, dz), (_DDTB, db), (_DS, ds)],
          A.LM_SOFTPLUS if dt_softplus else 0, max_len, chunk)
    return ScanGrads(dx, ddt, dA, dB if len(b_shape) == 4 else dB.view(b_shape), dC if len(c_shape) == 4 else dC.view(c_shape), dD,
                     dz, db, ds)


class PreparedSelectiveScanStep(_Step):
    """The step of ``selective_scan`` for fixed descriptors."""

    def __init__(self, x, dt, A_, B, C, state, *, D=None, z=None, dt_bias=None, dt_softplus: bool = False, rows=None):
        super().__init__(A.LM_SCAN_STEP, {_X: x, _DT: dt, _A: A_, _B: _grouped(B, 3), _C: _grouped(C, 3), _S1: state, _D: D,
                                          _Z: z, _DTB: dt_bias, _ROWS: rows}, tuple(x.shape), x,
                         A.LM_SOFTPLUS if dt_softplus else 0)

    def run(self, x, dt, A_, B, C, state, *, D=None, z=None, dt_bias=None, rows=None, y=None,
            stream: Optional[int] = None) -> torch.Tensor:
        q = _Ptrs()
        q[_X], q[_DT], q[_A], q[_B], q[_C] = x.data_ptr(), dt.data_ptr(), A_.data_ptr(), B.data_ptr(), C.data_ptr()
        q[_S1] = state.data_ptr()
        if D is not None:
            q[_D] = D.data_ptr()
        if z is not None:
            q[_Z] = z.data_ptr()
        if dt_bias is not None:
            q[_DTB] = dt_bias.data_ptr()
        if rows is not None:
            q[_ROWS] = rows.data_ptr()
        return self._launch(q, y, stream)


def selective_scan_step(x, dt, A_, B, C, state, *, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                        rows=None) -> torch.Tensor:
    """One token: x, dt, z [N, C], B and C [N, G, S] (or [N, S]), state f32
    [N, C, S] updated in place; ``rows`` as in ``causal_conv_step``."""
    y = _new(x)
    _call(A.LM_SCAN_STEP, [(_X, x), (_DT, dt), (_A, A_), (_B, _grouped(B, 3)), (_C, _grouped(C, 3)), (_S1, state), (_D, D),
                           (_Z, z), (_DTB, dt_bias), (_ROWS, rows)], [(_Y, y)], A.LM_SOFTPLUS if dt_softplus else 0)
    return y


# ---------------------------------------------------------- 4-bit products --

class PreparedMatvec4(_Step):
    """``matvec4`` for fixed descriptors (x [M, K])."""

    def __init__(self, x, packed, scales, zeros=None, bias=None):
        super().__init__(A.LM_MV4, {_X: x, _W: packed, _SCALES: scales, _ZEROS: zeros, _BIAS: bias},
                         (x.shape[0], packed.shape[0]), x)

    def run(self, x, packed, scales, zeros=None, bias=None, y=None, stream: Optional[int] = None) -> torch.Tensor:
        q = _Ptrs()
        q[_X], q[_W], q[_SCALES] = x.data_ptr(), packed.data_ptr(), scales.data_ptr()
        if zeros is not None:
            q[_ZEROS] = zeros.data_ptr()
        if bias is not None:
            q[_BIAS] = bias.data_ptr()
        return self._launch(q, y, stream)


def matvec4(x, packed, scales, zeros=None, bias=None) -> torch.Tensor:
    """x [..., K] times 4-bit weights: sum_k x[k] scales[n, k // group]
    (q[n, k] - zeros[n, k // group]) + bias[n], zeros 8 unless given.

    ``packed`` uint8 [N, K/2] holds the even k in the low four bits; scales and
    zeros [N, K/group] and x share a type; group is a multiple of 32.  Made for
    few rows: 16 cost about what one does, more repeat the weights' pass.  A
    row whose sums pass f32's range at 256 times x gives infinities or NaN."""
    x2 = x.reshape(-1, x.shape[-1])
    y = x2.new_empty((x2.shape[0], packed.shape[0]))
    _call(A.LM_MV4, [(_X, x2), (_W, packed), (_SCALES, scales), (_ZEROS, zeros), (_BIAS, bias)], [(_Y, y)])
    return y.view(x.shape[:-1] + (packed.shape[0],))


def quantize4(w: torch.Tensor, group: int = 128, symmetric: bool = True, dtype: torch.dtype = torch.bfloat16):
    """(packed, scales, zeros) of a weight [N, K]: round to nearest with one
    scale per group of columns, around 8 (zeros is None) or, not symmetric,
    around the group's own zero point."""
    n, k = w.shape
    if group < 1 or k % group or k % 2:
        raise ValueError(f"{k} columns do not make pairs and groups of {group}")
    g = w.float().reshape(n, k // group, group)
    if symmetric:
        scales = (g.abs().amax(2) / 7).to(dtype)
        scales[scales == 0] = 1  # a group of zeros
        zeros, z = None, 8.0
    else:
        lo, hi = g.amin(2).clamp(max=0), g.amax(2).clamp(min=0)
        scales = ((hi - lo) / 15).to(dtype)
        scales[scales == 0] = 1  # a group of zeros
        zeros = torch.round(-lo / scales.float()).clamp(0, 15).to(dtype)
        z = zeros.float()[..., None]
    q = torch.clamp(torch.round(g / scales.float()[..., None]) + z, 0, 15).to(torch.uint8).view(n, k)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scales, zeros
