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
