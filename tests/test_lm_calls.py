"""What the binding of the sequence operators hands to the library, on the CPU:
the outputs it allocates and the plans it keeps.  ``calls`` stands in for the
launch and records each call's plan and tensors."""
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
    monkeypatch.setattr(lm, "_on_gpu", lambda *t: None)
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
