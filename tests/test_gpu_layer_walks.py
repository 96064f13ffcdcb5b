"""Adapters whose workgroups walk over several blocks of outputs and share the
columns: rows gathered, found and sorted, ranks held in registers and not, last
blocks cut short, onto the base itself, rows without an adapter."""
import pytest
import torch

import lm_reference as R
from depthwise_stencil_implicit_amd import lm
from test_gpu_lm import gen, rnd

pytestmark = pytest.mark.gpu

BF, HF, F, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def planned(m, k, n, r, e):
    """(rows of a tile, parts of the columns, blocks of 256 outputs of a
    workgroup, those of the last one): adapter_shape of the library."""
    cdiv = lambda a, b: -(-a // b)  # noqa: E731
    few = m <= 512 and not (e <= 63 and m >= 16 * e and m * (k + n) > 1 << 20)
    groups = min(m, e + m // 16) if few else max(cdiv(m, 64), min(m, e // 8))
    parts = min(cdiv(256, groups), cdiv(k, 256), 16)
    work, blocks = groups if few else 2 * groups, cdiv(n, 256)
    spans = max(1, min(blocks, cdiv(4096, m) if few else blocks, ((768 if r <= 32 else 384) + work // 2) // work))
    reps = cdiv(blocks, spans)
    return (1 if few else 64), parts, reps, blocks - (cdiv(blocks, reps) - 1) * reps


CASES = [
    # dtype, rows, K, N', rank, E, base, 8-bit x, outputs apart
    (HF, 203, 600, 6913, 16, 40, True, False, False),      # gathered
    (BF, 203, 600, 6914, 20, 40, True, False, False),
    (F, 300, 520, 1795, 40, 60, True, False, False),
    (BF, 500, 600, 1536, 100, 300, True, True, False),
    (BF, 500, 300, 1539, 72, 300, False, False, False),
    (HF, 320, 300, 1282, 64, 200, True, False, True),
    (BF, 4100, 600, 2049, 16, 8, True, False, False),      # found
    (HF, 4100, 600, 2050, 40, 8, True, True, False),
    (BF, 4000, 515, 2304, 64, 5, True, False, False),
    (BF, 4100, 600, 2051, 72, 8, True, False, False),
    (BF, 4100, 600, 2049, 100, 8, True, False, False),
    (F, 4100, 300, 2049, 24, 8, False, False, False),
    (BF, 4100, 300, 2049, 12, 8, False, False, False),
    (BF, 3000, 600, 2312, 16, 8, True, False, True),
    (BF, 4100, 600, 2049, 16, 70, True, False, False),     # sorted
    (HF, 4100, 600, 2050, 40, 70, True, False, False),
    (BF, 4100, 900, 2304, 64, 90, True, True, False),
    (HF, 4100, 600, 2051, 72, 70, True, False, False),
    (BF, 4100, 600, 2049, 100, 70, False, False, False),
    (F, 4100, 600, 2049, 16, 70, True, False, False),
    (BF, 1100, 600, 2049, 20, 1000, True, False, False),
]


def exact(x, a, b, index, base, scaling, x_scales):
    """(y, bound) in 64 bits, adapter by adapter."""
    x = x.float().double() * (x_scales.double() if x_scales is not None else 1.0)
    y = base.double() if base is not None else torch.zeros((x.shape[0], b.shape[1]), dtype=torch.float64, device=x.device)
    bound = y.abs()
    for e in range(a.shape[0]):
        rows = (index == e).nonzero()[:, 0]
        if rows.numel():
            s, ae, be = scaling[e].double(), a[e].double().t().contiguous(), b[e].double().t().contiguous()
            y[rows] += s * (x[rows] @ ae) @ be
            bound[rows] += s.abs() * (x[rows].abs() @ ae.abs()) @ be.abs()
    return y.cpu(), bound.cpu()


@pytest.mark.parametrize("i", range(len(CASES)))
def test_walks_over_blocks_of_outputs(i):
    dt, m, k, n, r, e, has_base, f8, apart = CASES[i]
    rows, parts, reps, last = planned(m, k, n, r, e)
    assert reps > 1 and (parts > 1 or e >= 200)
    g = gen(2000 + i)
    x, a, b = rnd(g, m, k).cuda(), rnd(g, e, r, k, dtype=dt).cuda(), rnd(g, e, n, r, dtype=dt).cuda()
    xs = x.abs().amax(1, keepdim=True) / 448 if f8 else None
    x = (x / xs).to(F8) if f8 else x.to(dt)
    stored = lambda v: v.t().contiguous().t() if apart else v  # noqa: E731
    base = stored(rnd(g, m, n, dtype=dt).cuda()) if has_base else None
    scaling = (0.5 + torch.rand(e, generator=g)).cuda()
    index = torch.randint(-1, e + 1, (m,), generator=g)
    index[m // 3:m // 2] = index[m // 3]   # a run, and a hundred rows without an adapter at the least
    index[m // 2:m // 2 + m // 4] = torch.where(torch.rand(m // 4, generator=g) < 0.6, -1, index[m // 2:m // 2 + m // 4])
    index = index.to(torch.int32).cuda()
    kw = dict(scaling=scaling, x_scales=xs)
    print(f"adapters {CASES[i]}: {reps} blocks a workgroup, {last} at the end, {parts} parts", flush=True)
    out = stored(torch.full((m, n), 7.0, dtype=dt, device="cuda"))
    p = lm._make_plan(lm.A.LM_ADAPTERS, {lm._X: x, lm._A: a, lm._B: b, lm._ROWS: index, lm._Z: base, lm._D: scaling, lm._SCALES: xs, lm._Y: out})
    assert (p.chunk, p.chunks) == (rows, parts)
    got = lm.adapters(x, a, b, index, base=base, out=out, **kw)
    y, bound = exact(x, a, b, index, base, scaling, xs)
    # One rounding for each term of either sum, and those of the scales and parts.
    R.assert_close(got, y, bound, k + r + 64, "y")
    for _ in range(2):
        assert torch.equal(got, lm.adapters(x, a, b, index, base=base, out=stored(torch.empty_like(got)), **kw))
    if has_base:
        inplace = stored(base.clone())
        assert lm.adapters(x, a, b, index, base=inplace, out=inplace, **kw) is inplace and torch.equal(inplace, got)
