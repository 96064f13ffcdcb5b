"""The recurrent block of the examples, its operators one after the other:
prompts, gradients and tokens against the same block in 64 bits."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
spec = importlib.util.spec_from_file_location("recurrent_block", os.path.join(ROOT, "examples", "recurrent_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)
F = torch.float32


def data(m, n, l, width, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, l, width), generator=g).to(m.dtype).cuda().transpose(1, 2)


def exact(m, p, x, residual, index=None):
    """(output, residual) of the block in 64 bits on the CPU, for autograd."""
    s = x + residual
    n = s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6) * p["w_norm"][:, None]
    ug = p["w_in"] @ n
    if index is not None:
        a = {k: v.detach().cpu().double() for k, v in m.adapters.items()}
        for e in range(a["a"].shape[0]):
            ug = ug + (index.cpu() == e)[:, None] * a["scaling"][e] * (a["b"][e] @ (a["a"][e] @ n))
    u, gate = ug[:, :m.inner], ug[:, m.inner:]
    taps = p["w_conv"].shape[1]
    wide = torch.nn.functional.pad(u, (taps - 1, 0))
    u = torch.nn.functional.silu(sum(p["w_conv"][:, j, None] * wide[:, :, j:j + u.shape[2]] for j in range(taps)) + p["b_conv"][:, None])
    a = torch.exp(-8 * torch.nn.functional.softplus(p["decay"])[:, None] * torch.sigmoid(p["w_r"] @ u))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(p["w_i"] @ u) * u
    h, hs = torch.zeros_like(b[:, :, 0]), []
    for t in range(b.shape[2]):
        h = a[:, :, t] * h + b[:, :, t]
        hs.append(h)
    return p["w_out"] @ (torch.stack(hs, 2) * torch.nn.functional.silu(gate)), s


def doubles(m, grad=False):
    return {k: v.detach().cpu().double().requires_grad_(grad) for k, v in m.p.items()}


def far(a, b):
    return ((a.cpu().double() - b.detach()).norm() / b.detach().norm()).item()


def test_gradients_against_64_bits():
    m = example.RecurrentBlock(width=24, inner=40, taps=3, dtype=F)
    x, residual, target = (data(m, 2, 151, 24, s) for s in (1, 2, 3))
    loss, grads, dx = m.loss_and_gradients(x, residual, target)
    p, v = doubles(m, True), x.cpu().double().requires_grad_(True)
    out, s = exact(m, p, v, residual.cpu().double())
    want = ((out + s - target.cpu().double()) ** 2).mean()
    want.backward()
    # f32 through eight operators, sums of at most 302 terms of either sign.
    assert abs(loss.item() - want.item()) <= 1e-5 * want.item() and far(dx, v.grad) < 1e-4
    for k, g in grads.items():
        assert far(g, p[k].grad) < 1e-4, k


@pytest.mark.parametrize("dtype", [F, torch.bfloat16])
def test_tokens_continue_a_prompt(dtype):
    m = example.RecurrentBlock(width=64, inner=96, dtype=dtype)
    m.quantize()
    x, residual = data(m, 3, 24, 64, 6), data(m, 3, 24, 64, 7)
    index = torch.tensor([1, -1, 3], dtype=torch.int32, device="cuda")
    of = lambda n: index[:, None].expand(3, n).contiguous()  # noqa: E731
    whole, total, last = m.prompt(x, residual, index=of(24))
    want, s = exact(m, doubles(m), x.cpu().double(), residual.cpu().double(), of(24))
    # bf16: what lies between the operators is rounded, a few times 2^-9 of its size each.
    tol = 1e-5 if dtype == F else 3e-2
    assert far(whole, want) < tol and far(total, s) < tol
    _, _, state = m.prompt(x[:, :, :10], residual[:, :, :10], index=of(10))
    tokens = [m.step(x[:, :, t], residual[:, :, t], state, index) for t in range(10, 24)]
    assert far(torch.stack([t[0] for t in tokens], 2), whole[:, :, 10:].cpu().double()) < tol
    assert all(torch.equal(t[1], total[:, :, 10 + i]) for i, t in enumerate(tokens))
    for got, end in zip(state, last):
        assert far(got, end.cpu().double()) < tol


def test_prompt_with_the_norm_in_8_bits():
    m = example.RecurrentBlock(width=64, inner=96, dtype=F)
    x, residual = data(m, 2, 40, 64, 8), data(m, 2, 40, 64, 9)
    index = torch.tensor([0, 2], dtype=torch.int32, device="cuda")[:, None].expand(2, 40).contiguous()
    whole, total, _ = m.prompt(x, residual, index=index)
    eight, same, _ = m.prompt(x, residual, index=index, eight=True)
    # Rows rounded by 2^-4 of a value at most, 2^-6 of the row on the average, here and there.
    assert torch.equal(total, same) and 1e-4 < far(eight, whole.cpu().double()) < 0.1


def test_the_example_runs():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "recurrent_block.py")], capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("training step") == 5 and "64 tokens after" in out.stdout and "8 bits" in out.stdout
