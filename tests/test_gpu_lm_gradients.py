"""The example's state space mixer in 64 bits (torch's autograd on the CPU, the
layer written out position by position) against its loss, its gradients and its
outputs on the GPU."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("state_space_mixer", os.path.join(ROOT, "examples", "state_space_mixer.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def silu(v):
    return v / (1 + torch.exp(-v))


def mixer64(p, x, inner, rank, states):
    """x [N, width, L] -> [N, width, L]."""
    uz = torch.matmul(p["w_in"], x)
    u, z = uz[:, :inner], uz[:, inner:]
    k = p["w_conv"].shape[1]
    front = torch.cat([torch.zeros(u.shape[0], inner, k - 1, dtype=u.dtype), u], 2)
    u = silu(p["b_conv"][:, None] + sum(p["w_conv"][:, j, None] * front[:, :, j:j + u.shape[2]] for j in range(k)))
    low = torch.matmul(p["w_x"], u)
    dt, B, C = low[:, :rank], low[:, rank:rank + states], low[:, rank + states:]
    d = torch.log1p(torch.exp(torch.matmul(p["w_dt"], dt) + p["dt_bias"][:, None]))
    h, ys = torch.zeros(x.shape[0], inner, states, dtype=x.dtype), []
    for t in range(x.shape[2]):
        h = torch.exp(d[:, :, t, None] * p["A"]) * h + (d[:, :, t] * u[:, :, t])[..., None] * B[:, None, :, t]
        ys.append((h * C[:, None, :, t]).sum(2) + p["D"] * u[:, :, t])
    return torch.matmul(p["w_out"], torch.stack(ys, 2) * silu(z))


@pytest.mark.parametrize("sizes,length", [(dict(width=24, inner=40, states=5, taps=3, rank=32), 21),
                                          (dict(width=64, inner=96, states=16, taps=4, rank=32), 70)])
def test_gradients_in_64_bits(sizes, length):
    m = example.StateSpaceMixer(dtype=torch.float32, **sizes)
    g = torch.Generator().manual_seed(8)
    x, target = (torch.randn((2, length, sizes["width"]), generator=g).cuda().transpose(1, 2) for _ in range(2))
    loss, grads, dx = m.loss_and_gradients(x, target)
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in m.p.items()}
    x64 = x.cpu().double().requires_grad_()
    out = mixer64(p, x64, m.inner, m.rank, m.states)
    want = ((out - target.cpu().double()) ** 2).mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * want.item()
    # A few hundred f32 roundings of 2^-24 on the way to any of them, each
    # passed on with a slope of a few: 1e-4 of a gradient's norm is far above
    # that and far below what a missing or misplaced term would leave.
    for k, v in {**grads, "x": dx}.items():
        r = x64.grad if k == "x" else p[k].grad
        assert v.shape == r.shape and r.norm() > 0
        assert ((v.cpu().double() - r).norm() / r.norm()).item() <= 1e-4, k
