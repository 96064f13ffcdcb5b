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


# ----------------------------------------------- the adapters' inner sums in 24 bits --

STEP = 2.0 ** -19


def cancelling(dt, m, k, seed):
    """(x, a, b, t): inner sums t of 24 bits, exact in f32 and in any order, and
    weights against which pairs of them cancel to less than their last bit.

    x holds 16, 2^-4 and 2^-12 (times a power of two for each row); a t in 16 ..
    32, a multiple of 2^-19, is 16 hi + 2^-4 mid + 2^-12 lo of eight bits each."""
    g = gen(seed)
    E, R_, N = 2, 16, 70
    weights = (1 + torch.rand(2, 8, 2, generator=g)).to(dt).double()                  # beta, gamma of each pair
    weights[..., 1] = (weights[..., 0] * (0.85 + 0.3 * torch.rand(2, 8, generator=g))).to(dt).double()
    first = ((20 + 7 * torch.rand(2, 8, generator=g, dtype=torch.float64)) / STEP).round() * STEP
    second = (first * weights[..., 0] / weights[..., 1] / STEP).round() * STEP
    t = torch.stack([first, second], 2).view(E, R_)
    assert bool(((t >= 16) & (t < 32)).all())
    hi = torch.floor(t * 8) / 8
    mid = torch.floor((t - hi) * 2 ** 11) / 2 ** 11
    a = torch.zeros(E, R_, k, dtype=torch.float64)
    at = (0, 1, 2) if k < 64 else (5, k // 2, k - 1)
    for j, (col, v) in enumerate(zip(at, (hi / 16, mid * 16, (t - hi - mid) * 4096))):
        a[..., col] = v
    scale = 2.0 ** torch.randint(-1, 3, (m, 1), generator=g).double()
    x = torch.zeros(m, k, dtype=torch.float64)
    x[:, list(at)] = torch.tensor([16.0, 2.0 ** -4, 2.0 ** -12], dtype=torch.float64) * scale
    b = torch.zeros(E, N, R_, dtype=torch.float64)
    for n in range(N):
        p = n % 8
        b[:, n, 2 * p], b[:, n, 2 * p + 1] = weights[:, p, 0], -weights[:, p, 1]
    for v in (x, a, b):
        assert torch.equal(v.to(dt).double(), v)
    sums = scale * torch.einsum("mk,erk->mer", x / scale, a).flatten(1)
    assert torch.equal(sums.float().double(), sums)
    return x, a, b, sums.view(m, E, R_)


def leading(t, terms):
    """t cut to its first bf16 terms."""
    out = torch.zeros_like(t)
    for _ in range(terms):
        out += ((t - out).float().view(torch.int32) & -65536).view(torch.float32).double()
    return out


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("m,k", [(20, 3), (20, 96), (600, 70)])
def test_inner_sums_keep_24_bits(dt, m, k):
    """Second products that cancel all of their leading bits.  A result passes at
    most ten additions, a unit of 2^-24 of the absolute sum each where the
    matrix instruction cuts, and f16 weights leave out a product below one."""
    x, a, b, t = cancelling(dt, m, k, 7 * m + k)
    index = (torch.arange(m) * 5 // 3 % 2).to(torch.int32)
    mine = t[torch.arange(m), index.long()][:, None]                                 # [m, 1, ranks]
    w = b[index.long()]
    y, bound = (mine * w).sum(2), (mine * w).abs().sum(2)
    check = lambda v, what: R.assert_close(v.to(dt), y, bound, 12, what)  # noqa: E731
    got = lm.adapters(x.to(dt).cuda(), a.to(dt).cuda(), b.to(dt).cuda(), index.cuda())
    check(got, "y")
    for terms in (1, 2):
        with pytest.raises(AssertionError, match="outside"):
            check((leading(mine, terms) * w).sum(2), f"{terms} terms")
    if dt == HF:
        high = leading(w, 1)
        with pytest.raises(AssertionError, match="outside"):
            check((mine * high + leading(mine, 1) * (w - high)).sum(2), "the low weights' second term")
