"""A state space mixer layer on the library's operators, as a language model
uses it: prompts, training steps and single tokens.

    python examples/state_space_mixer.py

    u, z   = in_projection(x)
    u      = silu(causal_conv(u))
    dt,B,C = x_projection(u);  dt = dt_projection(dt)
    y      = selective_scan(u, dt, A, B, C, D, z)
    out    = out_projection(y)

Activations are [N, channels, L], stored as L rows of channels.  Prompts and
training run the projections as 1x1 convolutions (plain GEMMs of the
convolution library), single tokens as products with 4-bit weights.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from depthwise_stencil_implicit_amd import api, lm  # noqa: E402


def project(x, w):
    """w [out, in] on every position of x [N, in, L]."""
    return api.conv(x.unsqueeze(2), w[:, :, None, None]).squeeze(2)


def project_backward(x, w, gy):
    dx, dw, _ = api.conv_backward(x.unsqueeze(2), w[:, :, None, None], gy.unsqueeze(2), need_db=False)
    return dx.squeeze(2), dw[:, :, 0, 0]


def rows(*parts):
    """Channels of the parts one after the other, stored as rows."""
    n, _, l = parts[0].shape
    out = torch.empty(n, l, sum(p.shape[1] for p in parts), dtype=parts[0].dtype, device=parts[0].device).transpose(1, 2)
    at = 0
    for p in parts:
        out[:, at:at + p.shape[1]] = p
        at += p.shape[1]
    return out


class StateSpaceMixer:
    def __init__(self, width=512, inner=1024, states=16, taps=4, rank=32, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        f32 = lambda t: t.float().cuda()  # noqa: E731
        self.inner, self.states, self.rank, self.dtype = inner, states, rank, dtype
        step = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(inner, generator=g))
        self.p = {"w_in": r(2 * inner, width) / math.sqrt(width), "w_x": r(rank + 2 * states, inner) / math.sqrt(inner),
                  "w_dt": r(inner, rank) / math.sqrt(rank), "w_out": r(width, inner) / math.sqrt(inner),
                  "w_conv": r(inner, taps) / math.sqrt(taps), "b_conv": torch.zeros(inner)}
        self.p = {k: v.to(dtype).cuda() for k, v in self.p.items()}
        self.p |= {"A": f32(-torch.arange(1.0, states + 1).repeat(inner, 1)), "D": f32(torch.ones(inner)),
                   "dt_bias": f32(step + torch.log(-torch.expm1(-step)))}
        self.q = None

    # ------------------------------------------------------------- prompts --

    def _forward(self, x, state, save=False):
        p, di, s = self.p, self.inner, self.states
        uz = project(x, p["w_in"])
        conv = lm.causal_conv(uz[:, :di], p["w_conv"], p["b_conv"], activation="silu", state=state and state[0],
                              return_state=True)
        low = project(conv.y, p["w_x"])
        dt, B, C = low[:, :self.rank], low[:, self.rank:self.rank + s], low[:, self.rank + s:]
        delta = project(dt, p["w_dt"])
        scan = lm.selective_scan(conv.y, delta, p["A"], B, C, D=p["D"], z=uz[:, di:], dt_bias=p["dt_bias"], dt_softplus=True,
                                 state=state and state[1], return_state=True, save=save)
        out = project(scan.y, p["w_out"])
        return out, (conv.state, scan.state), (uz, conv.y, dt, B, C, delta, scan)

    def prompt(self, x, state=None):
        """x [N, width, L] -> output and the state that decoding starts from."""
        return self._forward(x, state)[:2]

    # ------------------------------------------------------------ training --

    def loss_and_gradients(self, x, target):
        """Mean squared error and the gradients of every parameter and of x."""
        p, di = self.p, self.inner
        out, _, (uz, u, dt, B, C, delta, scan) = self._forward(x, None, save=True)
        diff = out.float() - target.float()
        go = rows((2 / diff.numel() * diff).to(self.dtype))
        gy, dw_out = project_backward(scan.y, p["w_out"], go)
        s = lm.selective_scan_backward(gy, u, delta, p["A"], B, C, D=p["D"], z=uz[:, di:], dt_bias=p["dt_bias"],
                                       dt_softplus=True, saved=scan.saved)
        d_dt, dw_dt = project_backward(dt, p["w_dt"], s.ddt)
        du, dw_x = project_backward(u, p["w_x"], rows(d_dt, s.dB, s.dC))
        c = lm.causal_conv_backward(s.dx + du, uz[:, :di], p["w_conv"], p["b_conv"], activation="silu")
        dx, dw_in = project_backward(x, p["w_in"], rows(c.dx, s.dz))
        grads = {"w_in": dw_in, "w_x": dw_x, "w_dt": dw_dt, "w_out": dw_out, "w_conv": c.dw, "b_conv": c.db, "A": s.dA,
                 "D": s.dD, "dt_bias": s.ddt_bias}
        return (diff ** 2).mean(), grads, dx

    # ------------------------------------------------------- single tokens --

    def quantize(self, group=32):
        """4-bit projections for decoding; the dense ones take the same values."""
        self.q = {}
        for k in ("w_in", "w_x", "w_dt", "w_out"):
            w = self.p[k]
            packed, scales, _ = lm.quantize4(w.float(), group, dtype=self.dtype)
            q = torch.stack([packed & 15, packed >> 4], 2).reshape(w.shape).float() - 8
            self.p[k] = (q * scales.float().repeat_interleave(group, 1)).to(self.dtype)
            self.q[k] = (packed, scales)

    def step(self, x, state):
        """One token x [N, width]; the state moves on in place."""
        p, q, di, s = self.p, self.q, self.inner, self.states
        uz = lm.matvec4(x, *q["w_in"])
        u = lm.causal_conv_step(uz[:, :di], p["w_conv"], p["b_conv"], state[0], activation="silu")
        low = lm.matvec4(u, *q["w_x"])
        delta = lm.matvec4(low[:, :self.rank], *q["w_dt"])
        y = lm.selective_scan_step(u, delta, p["A"], low[:, self.rank:self.rank + s], low[:, self.rank + s:], state[1], D=p["D"],
                                   z=uz[:, di:], dt_bias=p["dt_bias"], dt_softplus=True)
        return lm.matvec4(y, *q["w_out"])


def main():
    torch.manual_seed(0)
    m = StateSpaceMixer()
    x = torch.randn(4, 192, 512, device="cuda").to(m.dtype).transpose(1, 2)
    target = torch.randn(4, 192, 512, device="cuda").to(m.dtype).transpose(1, 2)
    for step in range(5):
        loss, grads, _ = m.loss_and_gradients(x, target)
        print(f"training step {step}: loss {loss.item():.4f}", flush=True)
        for k, g in grads.items():
            m.p[k] -= (2.0 * g.float()).to(m.p[k].dtype)
    m.quantize()
    whole, _ = m.prompt(x)
    _, state = m.prompt(x[:, :, :128])
    tokens = torch.stack([m.step(x[:, :, t], state) for t in range(128, 192)], 2)
    rel = ((tokens - whole[:, :, 128:]).float().norm() / whole[:, :, 128:].float().norm()).item()
    print(f"64 tokens after a prompt of 128: {rel:.1e} from the prompt of 192", flush=True)


if __name__ == "__main__":
    main()
