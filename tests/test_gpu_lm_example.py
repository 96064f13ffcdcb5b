"""The state space mixer of the examples: gradients against differences of its
own loss, training that lowers it, and tokens that continue a prompt."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("state_space_mixer", os.path.join(ROOT, "examples", "state_space_mixer.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def data(m, n, l, width, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, l, width), generator=g).to(m.dtype).cuda().transpose(1, 2)


def test_gradients_against_differences():
    m = example.StateSpaceMixer(width=24, inner=40, states=5, taps=3, rank=32, dtype=torch.float32)
    x, target = data(m, 2, 21, 24, 1), data(m, 2, 21, 24, 2)
    _, grads, dx = m.loss_and_gradients(x, target)
    g = torch.Generator().manual_seed(3)
    for k, v in grads.items():
        d = torch.randn(v.shape, generator=g).cuda()
        d /= d.norm()
        p, e, loss = m.p[k], 1e-2, []
        for sign in (1, -1):
            m.p[k] = p + sign * e * d
            loss.append(m.loss_and_gradients(x, target)[0].double().item())
        m.p[k] = p
        diff = (loss[0] - loss[1]) / (2 * e)
        mine = (v.double() * d.double()).sum().item()
        # f32 losses near 1 over 2e-2, and the second difference of a step of 1e-2.
        assert abs(diff - mine) <= 2e-4 + 2e-2 * v.double().norm().item(), (k, diff, mine)
    assert torch.isfinite(dx).all()


def test_training_lowers_the_loss():
    m = example.StateSpaceMixer(width=64, inner=96, dtype=torch.float32)
    x, target = data(m, 2, 40, 64, 4), data(m, 2, 40, 64, 5)
    losses = []
    for _ in range(6):
        loss, grads, _ = m.loss_and_gradients(x, target)
        losses.append(loss.item())
        for k, g in grads.items():
            m.p[k] -= 2.0 * g.to(m.p[k].dtype)
    assert losses[-1] < losses[0], losses


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_continue_a_prompt(dtype):
    m = example.StateSpaceMixer(width=64, inner=96, dtype=dtype)
    m.quantize()
    x = data(m, 3, 24, 64, 6)
    whole, last = m.prompt(x)
    _, state = m.prompt(x[:, :, :10])
    tokens = torch.stack([m.step(x[:, :, t], state) for t in range(10, 24)], 2)
    # bf16: the activations between the operators and the prompt's dense
    # weights are rounded, a few times 2^-9 of their size each.
    tol = 1e-5 if dtype == torch.float32 else 3e-2
    for got, want in ((tokens, whole[:, :, 10:]), (state[0], last[0]), (state[1], last[1])):
        assert ((got - want).float().norm() / want.float().norm()).item() < tol
