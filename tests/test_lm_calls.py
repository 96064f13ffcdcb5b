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
