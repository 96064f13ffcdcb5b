"""Host logic of the sequence operators, on the CPU: the exported calls and
struct layouts, what lm_plan accepts and refuses, and lm_run's own checks."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from depthwise_stencil_implicit_amd import _abi as A
from depthwise_stencil_implicit_amd import lm
from depthwise_stencil_implicit_amd.api import ConvError

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "miconv_lm.h")
BF, F = torch.bfloat16, torch.float32


def test_header_and_library_agree():
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"MICONV_API\s+[\w\s\*]*?\b(lm_\w+)\s*\(", text)))
    assert names == sorted(A.LM_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", A.LIB_PATH], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert {s for s in exported if s.startswith("lm_")} == set(names)


def test_struct_layout_matches_ctypes(tmp_path):
    src = tmp_path / "probe.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "miconv_lm.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu %zu %d %d %d %d\\n", sizeof(lm_args), sizeof(lm_plan_t), offsetof(lm_plan_t, t),'
                   ' offsetof(lm_plan_t, seqs), offsetof(lm_plan_t, saved_floats), offsetof(lm_plan_t, bytes), LM_NSLOT, LM_SAVED,'
                   ' LM_ZEROS, LM_MV4);\nreturn 0; }\n')
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-std=c99", f"-I{os.path.dirname(HEADER)}", str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    P = A.LmPlan
    assert got == [ctypes.sizeof(A.LmArgs), ctypes.sizeof(P), P.t.offset, P.seqs.offset, P.saved_floats.offset, P.bytes.offset,
                   A.LM_NSLOT, lm._SAVED, lm._ZEROS, A.LM_MV4]


def conv_tensors(n=2, c=8, l=10, k=4, dtype=BF):
    return {lm._X: torch.empty(n, c, l, dtype=dtype), lm._W: torch.empty(c, k, dtype=dtype), lm._BIAS: torch.empty(c, dtype=dtype),
            lm._Y: torch.empty(n, c, l, dtype=dtype), lm._S0: torch.empty(n, c, k - 1, dtype=dtype)}


def scan_tensors(n=2, c=8, l=10, s=16, g=2, dtype=BF):
    e = lambda *v, d=dtype: torch.empty(v, dtype=d)  # noqa: E731
    return {lm._X: e(n, c, l), lm._DT: e(n, c, l), lm._Z: e(n, c, l), lm._Y: e(n, c, l), lm._A: e(c, s, d=F), lm._D: e(c, d=F),
            lm._DTB: e(c, d=F), lm._B: e(n, g, s, l), lm._C: e(n, g, s, l), lm._S0: e(n, c, s, d=F)}


def mv_tensors(m=3, k=256, n=20, groups=2, dtype=BF):
    e = lambda *v, d=dtype: torch.empty(v, dtype=d)  # noqa: E731
    return {lm._X: e(m, k), lm._W: e(n, k // 2, d=torch.uint8), lm._SCALES: e(n, groups), lm._ZEROS: e(n, groups), lm._BIAS: e(n),
            lm._Y: e(m, n)}


def status(op, tensors, **kw):
    try:
        lm._make_plan(op, tensors, **kw)
        return A.OK
    except ConvError as e:
        return e.status


def test_plans_of_plain_calls():
    assert status(A.LM_CONV, conv_tensors()) == A.OK
    assert status(A.LM_SCAN, scan_tensors()) == A.OK
    assert status(A.LM_MV4, mv_tensors()) == A.OK
    p = lm._make_plan(A.LM_CONV, conv_tensors(n=1, c=4096, l=1), flags=A.LM_SILU)
    assert p.chunks == 1 and p.workspace_bytes == 0
    # A long row with few channels is split, a wide batch is not.
    assert lm._make_plan(A.LM_SCAN, scan_tensors(n=1, c=64, l=4096, g=1)).chunks > 8
    assert lm._make_plan(A.LM_SCAN, scan_tensors(n=32, c=2048, l=64, g=1)).chunks == 1
    # What selective_scan allocates for saved states is what the plan asks for.
    for n, l, s, lens in ((2, 33, 16, None), (1, 50, 20, [0, 17, 33]), (1, 64, 64, [64]), (3, 1, 1, None)):
        t = scan_tensors(n=n, c=6, l=l, s=s, g=1)
        off = torch.zeros(len(lens) + 1, dtype=torch.int32) if lens else None
        t.pop(lm._S0)
        t[lm._OFF] = off
        t[lm._SAVED] = lm._new_saved(t[lm._X], t[lm._A], off)
        assert status(A.LM_SCAN, t) == A.OK


CONV_BAD = [
    ({lm._X: torch.empty(2, 8, dtype=BF)}, A.EINVAL),                       # rank
    ({lm._W: torch.empty(8, 4, dtype=F)}, A.EINVAL),                        # mixed types
    ({lm._W: torch.empty(7, 4, dtype=BF)}, A.EINVAL),                       # channels
    ({lm._W: torch.empty(8, 9, dtype=BF), lm._S0: None}, A.EUNSUPPORTED),   # taps
    ({lm._W: torch.empty(8, 0, dtype=BF), lm._S0: None}, A.EINVAL),
    ({lm._S0: torch.empty(2, 8, 4, dtype=BF)}, A.EINVAL),                   # state's length
    ({lm._S0: torch.empty(3, 8, 3, dtype=BF)}, A.EINVAL),                   # state's rows
    ({lm._Y: None}, A.EINVAL),
    ({lm._Y: torch.empty(2, 8, 1, dtype=BF).expand(2, 8, 10)}, A.EINVAL),   # output in one place
    ({lm._Y: torch.empty(2, 8, 9, dtype=BF)}, A.EINVAL),
    ({lm._OFF: torch.empty(3, dtype=torch.int32)}, A.EINVAL),               # packed needs one row
    ({lm._A: torch.empty(8, 4)}, A.EINVAL),                                 # no tensor of this operator
]


@pytest.mark.parametrize("i", range(len(CONV_BAD)))
def test_conv_refusals(i):
    change, want = CONV_BAD[i]
    assert status(A.LM_CONV, {**conv_tensors(), **change}) == want


SCAN_BAD = [
    ({lm._DT: torch.empty(2, 8, 11, dtype=BF)}, A.EINVAL),
    ({lm._A: torch.empty(8, 16, dtype=BF)}, A.EINVAL),                      # A is f32
    ({lm._A: torch.empty(8, 65), lm._S0: None}, A.EUNSUPPORTED),
    ({lm._B: torch.empty(2, 3, 16, 10, dtype=BF), lm._C: torch.empty(2, 3, 16, 10, dtype=BF)}, A.EINVAL),  # groups
    ({lm._C: torch.empty(2, 2, 15, 10, dtype=BF)}, A.EINVAL),
    ({lm._B: torch.empty(2, 2, 16, 10, dtype=torch.float16)}, A.EINVAL),
    ({lm._D: torch.empty(7)}, A.EINVAL),
    ({lm._S0: torch.empty(2, 8, 16, dtype=BF)}, A.EINVAL),
    ({lm._SAVED: torch.empty(5)}, A.EINVAL),
    ({lm._OFF: torch.empty(0, dtype=torch.int32)}, A.EINVAL),
]


@pytest.mark.parametrize("i", range(len(SCAN_BAD)))
def test_scan_refusals(i):
    change, want = SCAN_BAD[i]
    assert status(A.LM_SCAN, {**scan_tensors(), **change}) == want


MV_BAD = [
    ({lm._SCALES: torch.empty(20, 3, dtype=BF), lm._ZEROS: None}, A.EINVAL),           # 256 / 3
    ({lm._SCALES: torch.empty(20, 16, dtype=BF), lm._ZEROS: None}, A.EUNSUPPORTED),    # groups of 16
    ({lm._SCALES: torch.empty(20, 2), lm._ZEROS: None}, A.EINVAL),
    ({lm._W: torch.empty(20, 100, dtype=torch.uint8)}, A.EINVAL),
    ({lm._W: torch.empty(20, 129, dtype=torch.uint8)[:, 1:]}, A.EUNSUPPORTED),         # rows off 16 bytes
    ({lm._W: torch.empty(20, 128)}, A.EINVAL),
    ({lm._BIAS: torch.empty(19, dtype=BF)}, A.EINVAL),
]


@pytest.mark.parametrize("i", range(len(MV_BAD)))
def test_mv4_refusals(i):
    change, want = MV_BAD[i]
    assert status(A.LM_MV4, {**mv_tensors(), **change}) == want


def test_step_state_rows():
    t = {lm._X: torch.empty(3, 8, dtype=BF), lm._W: torch.empty(8, 4, dtype=BF), lm._Y: torch.empty(3, 8, dtype=BF),
         lm._S1: torch.empty(5, 8, 3, dtype=BF)}
    assert status(A.LM_CONV_STEP, t) == A.EINVAL                            # five rows for three, unnamed
    assert status(A.LM_CONV_STEP, {**t, lm._ROWS: torch.empty(3, dtype=torch.int32)}) == A.OK
    assert status(A.LM_CONV_STEP, {**t, lm._ROWS: torch.empty(4, dtype=torch.int32)}) == A.EINVAL
    assert status(A.LM_CONV_STEP, {**t, lm._ROWS: torch.empty(3, dtype=torch.int64)}
                  if torch.int64 in lm._TYPES else {**t, lm._S1: None}) == A.EINVAL


def test_arguments_and_devices():
    with pytest.raises(ValueError, match="GPU only"):
        lm.causal_conv(torch.empty(1, 4, 4), torch.empty(4, 2))
    with pytest.raises(ValueError, match="activation"):
        lm._act("gelu")
    with pytest.raises(TypeError, match="unsupported dtype"):
        lm._make_plan(A.LM_CONV, {**conv_tensors(), lm._X: torch.empty(2, 8, 10, dtype=torch.float64)})
    assert status(A.LM_CONV, conv_tensors(), flags=A.LM_SOFTPLUS) == A.EINVAL
    assert status(A.LM_SCAN, scan_tensors(), max_len=-1) == A.EINVAL
    assert status(99, conv_tensors()) == A.EINVAL


def test_run_checks_pointers_before_any_device_call():
    t = {k: v for k, v in conv_tensors().items()}
    p = lm._make_plan(A.LM_CONV, t)
    run = lambda q, ws=None, n=0: A.lib().lm_run(ctypes.byref(p), q, ws, n, None)  # noqa: E731
    q = lm._Ptrs()
    assert run(q) == A.EINVAL
    for k, v in t.items():
        q[k] = v.data_ptr()
    q[lm._X] = t[lm._X].data_ptr() + 1
    assert run(q) == A.EALIGN
    q[lm._X] = t[lm._X].data_ptr()
    q[lm._GY] = t[lm._X].data_ptr()
    assert run(q) == A.EINVAL                                               # a pointer for an absent tensor
    s = scan_tensors(n=1, c=8, l=4096, g=1)
    s[lm._S0] = None
    p2 = lm._make_plan(A.LM_SCAN, s)
    assert p2.workspace_bytes > 0
    q = lm._Ptrs()
    for k, v in s.items():
        if v is not None:
            q[k] = v.data_ptr()
    assert A.lib().lm_run(ctypes.byref(p2), q, None, 0, None) == A.EINVAL
    assert A.lib().lm_run(None, q, None, 0, None) == A.EINVAL


def test_quantize4_layout():
    w = torch.randn(6, 64)
    packed, scales, zeros = lm.quantize4(w, 32, dtype=F)
    assert packed.shape == (6, 32) and scales.shape == (6, 2) and zeros is None
    q = torch.stack([packed & 15, packed >> 4], 2).reshape(6, 64).float() - 8
    assert bool(((q * scales.repeat_interleave(32, 1) - w).abs() <= scales.repeat_interleave(32, 1) * 0.5001).all())
    with pytest.raises(ValueError):
        lm.quantize4(w, 48)
