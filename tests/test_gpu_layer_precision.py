"""What the recurrent layers' operators keep in 32 bits, against 64 bits and
bounds that a value rounded to 16 bits on the way would pass."""
import pytest
import torch

import layer_reference as Y
import lm_reference as R
from depthwise_stencil_implicit_amd import lm
from test_gpu_layer import BF, F, HF, NORM, norm_case
from test_gpu_lm import gen, rnd

pytestmark = pytest.mark.gpu


# ------------------------------------------- the norm's gradients at x + residual --

@pytest.mark.parametrize("i", [i for i, c in enumerate(NORM) if c[4]])
def test_norm_gradients_from_the_calls_own_tensors(i):
    x, res, gy, gr, w = norm_case(i)
    print(f"norm {NORM[i]}", flush=True)
    f = lm.rms_norm(x, w, residual=res, eps=1e-5, save=True)
    gr = gr if i % 2 else None
    back = lm.rms_norm_backward(gy, x, w, f.rstd, residual=res, gresidual=gr)
    v = x.cpu().double() + res.cpu().double()
    (dx, dw), (bx, bw) = Y.norm_backward(gy, v, w, f.rstd, gr)
    R.assert_close(back.dx, dx, bx, 160, "dx")
    R.assert_close(back.dw, dw, bw, NORM[i][1] * max(1, NORM[i][3]) + 160, "dw")
    only = lm.rms_norm_backward(gy, x, w, f.rstd, residual=res, need_dx=False)
    assert only.dx is None and torch.equal(only.dw, back.dw)
    only = lm.rms_norm_backward(gy, x, w, f.rstd, residual=res, gresidual=gr, need_dw=False)
    assert only.dw is None and torch.equal(only.dx, back.dx)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("c", [40, 1500])
def test_norm_gradients_tell_the_rounded_sum(dt, c):
    """dw of 300 rows from x and residual is within the bound of the unrounded
    sum; the formula at the sum as it was stored is not."""
    g = gen(c)
    x, res, gy, w = rnd(g, 300, c, dtype=dt).cuda(), rnd(g, 300, c, dtype=dt, scale=2.0).cuda(), rnd(g, 300, c, dtype=dt).cuda(), rnd(g, c, dtype=dt).cuda()
    f = lm.rms_norm(x, w, residual=res, save=True)
    v = x.cpu().double() + res.cpu().double()
    (_, dw), (_, bound) = Y.norm_backward(gy, v, w, f.rstd)
    R.assert_close(lm.rms_norm_backward(gy, x, w, f.rstd, residual=res).dw, dw, bound, 300 + 160, "dw")
    (_, stored), _ = Y.norm_backward(gy, f.residual, w, f.rstd)
    with pytest.raises(AssertionError, match="outside"):
        R.assert_close(stored.to(dt), dw, bound, 300 + 160, "stored")
