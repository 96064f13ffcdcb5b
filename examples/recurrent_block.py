"""A residual block with a gated linear recurrence on the library's operators,
as a language model uses it: prompts of several requests with adapters of their
own, training steps and single tokens.

    python examples/recurrent_block.py

    s      = x + residual;  n = rms_norm(s)
    u, g   = in_projection(n) + adapter of the request
    u      = silu(causal_conv(u))
    h      = gated_recurrence(u, r_projection(u), i_projection(u))
    out    = out_projection(h silu(g)),  the next block's x beside the residual s

Activations are [N, channels, L], stored as L rows of channels.  Prompts and
training run the projections as 1x1 convolutions, single tokens as products with
4-bit weights; prompts may also take the norm's rows in 8 bits, which both the
shared projection and the adapters read.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from depthwise_stencil_implicit_amd import lm  # noqa: E402
from examples.state_space_mixer import project, project_backward, rows  # noqa: E402

F8 = torch.float8_e4m3fn


def silu(v):
    return v.float() * torch.sigmoid(v.float())


class RecurrentBlock:
    def __init__(self, width=512, inner=768, taps=4, adapters=4, rank=16, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.inner, self.dtype = inner, dtype
        k = -torch.log(0.9 + 0.099 * torch.rand(inner, generator=g))   # what is forgotten in a step at an open gate
        self.p = {"w_norm": 1 + 0.1 * r(width), "w_in": r(2 * inner, width) / math.sqrt(width), "w_conv": r(inner, taps) / math.sqrt(taps),
                  "b_conv": torch.zeros(inner), "w_r": r(inner, inner) / math.sqrt(inner), "w_i": r(inner, inner) / math.sqrt(inner),
                  "w_out": r(width, inner) / math.sqrt(inner)}
        self.p = {n: v.to(dtype).cuda() for n, v in self.p.items()}
        self.p["decay"] = torch.log(torch.expm1(k / 8)).float().cuda()
        self.adapters = {"a": (r(adapters, rank, width) / math.sqrt(width)).to(dtype).cuda(),
                         "b": (0.1 * r(adapters, 2 * inner, rank)).to(dtype).cuda(), "scaling": (1 + r(adapters) / 8).cuda()}
        self.q = None

    # ------------------------------------------------------------- prompts --

    def _forward(self, x, residual, state=None, index=None, save=False, eight=False):
        p, di, a = self.p, self.inner, self.adapters
        n = lm.rms_norm(x, p["w_norm"], residual=residual, save=save, out_dtype=F8 if eight else None)
        # Values of 8 bits times the row's scale; a plain product otherwise.
        ug = project(n.y.to(self.dtype) if eight else n.y, p["w_in"])
        if eight:
            ug = (ug.float() * n.scales).to(self.dtype)
        if index is not None:
            lm.adapters(n.y, a["a"], a["b"], index, base=ug, scaling=a["scaling"], x_scales=n.scales, out=ug)
        conv = lm.causal_conv(ug[:, :di], p["w_conv"], p["b_conv"], activation="silu", state=state and state[0], return_state=True)
        r, i = project(conv.y, p["w_r"]), project(conv.y, p["w_i"])
        rec = lm.gated_recurrence(conv.y, r, i, p["decay"], state=state and state[1], return_state=True, save=save)
        gated = rows((rec.y.float() * silu(ug[:, di:])).to(self.dtype))
        return project(gated, p["w_out"]), n, (conv.state, rec.state), (ug, conv.y, r, i, rec, gated)

    def prompt(self, x, residual, state=None, index=None, eight=False):
        """x and residual [N, width, L], index int32 [N, L] or None -> (output,
        new residual, the state that decoding starts from)."""
        out, n, state, _ = self._forward(x, residual, state, index, eight=eight)
        return out, n.residual, state

    # ------------------------------------------------------------ training --

    def loss_and_gradients(self, x, residual, target):
        """Mean squared error of output plus residual, and the gradients of every
        parameter and of x (the residual's is the same)."""
        p, di = self.p, self.inner
        out, n, _, (ug, u, r, i, rec, gated) = self._forward(x, residual, save=True)
        diff = out.float() + n.residual.float() - target.float()
        go = rows((2 / diff.numel() * diff).to(self.dtype))
        dz, dw_out = project_backward(gated, p["w_out"], go)
        gate, q = ug[:, di:].float(), torch.sigmoid(ug[:, di:].float())
        dgate = (dz.float() * rec.y.float() * q * (1 + gate * (1 - q))).to(self.dtype)
        s = lm.gated_recurrence_backward(rows((dz.float() * gate * q).to(self.dtype)), u, r, i, p["decay"], saved=rec.saved)
        d_r, dw_r = project_backward(u, p["w_r"], s.dr)
        d_i, dw_i = project_backward(u, p["w_i"], s.di)
        c = lm.causal_conv_backward(rows(s.dx + d_r + d_i), ug[:, :di], p["w_conv"], p["b_conv"], activation="silu")
        dn, dw_in = project_backward(n.y, p["w_in"], rows(c.dx, dgate))
        norm = lm.rms_norm_backward(dn, n.residual, p["w_norm"], n.rstd, gresidual=go)
        grads = {"w_norm": norm.dw, "w_in": dw_in, "w_conv": c.dw, "b_conv": c.db, "w_r": dw_r, "w_i": dw_i, "decay": s.ddecay, "w_out": dw_out}
        return (diff ** 2).mean(), grads, norm.dx

    # ------------------------------------------------------- single tokens --

    def quantize(self, group=32):
        """4-bit projections for decoding; the dense ones take the same values."""
        self.q = {}
        for k in ("w_in", "w_r", "w_i", "w_out"):
            w = self.p[k]
            packed, scales, _ = lm.quantize4(w.float(), group, dtype=self.dtype)
            q = torch.stack([packed & 15, packed >> 4], 2).reshape(w.shape).float() - 8
            self.p[k] = (q * scales.float().repeat_interleave(group, 1)).to(self.dtype)
            self.q[k] = (packed, scales)

    def step(self, x, residual, state, index=None):
        """One token, x and residual [N, width], index int32 [N] or None: output
        and new residual; the state moves on in place."""
        p, q, di, a = self.p, self.q, self.inner, self.adapters
        n = lm.rms_norm(x, p["w_norm"], residual=residual)
        ug = lm.matvec4(n.y, *q["w_in"])
        if index is not None:
            lm.adapters(n.y, a["a"], a["b"], index, base=ug, scaling=a["scaling"], out=ug)
        u = lm.causal_conv_step(ug[:, :di], p["w_conv"], p["b_conv"], state[0], activation="silu")
        h = lm.gated_recurrence_step(u, lm.matvec4(u, *q["w_r"]), lm.matvec4(u, *q["w_i"]), p["decay"], state[1])
        return lm.matvec4((h.float() * silu(ug[:, di:])).to(self.dtype), *q["w_out"]), n.residual


def main():
    m = RecurrentBlock()
    make = lambda: torch.randn(4, 192, 512, device="cuda").to(m.dtype).transpose(1, 2)  # noqa: E731
    torch.manual_seed(0)
    x, residual, target = make(), make(), make()
    for step in range(5):
        loss, grads, _ = m.loss_and_gradients(x, residual, target)
        print(f"training step {step}: loss {loss.item():.4f}", flush=True)
        for k, g in grads.items():
            m.p[k] -= (2.0 * g.float()).to(m.p[k].dtype)
    m.quantize()
    index = torch.tensor([2, -1, 0, 2], dtype=torch.int32, device="cuda")   # a request each, one without an adapter
    of = lambda n: index[:, None].expand(4, n).contiguous()  # noqa: E731
    whole, _, _ = m.prompt(x, residual, index=of(192))
    _, _, state = m.prompt(x[:, :, :128], residual[:, :, :128], index=of(128))
    tokens = torch.stack([m.step(x[:, :, t], residual[:, :, t], state, index)[0] for t in range(128, 192)], 2)
    far = lambda a, b: ((a - b).float().norm() / b.float().norm()).item()  # noqa: E731
    print(f"64 tokens after a prompt of 128: {far(tokens, whole[:, :, 128:]):.1e} from the prompt of 192", flush=True)
    eight, _, _ = m.prompt(x, residual, index=of(192), eight=True)
    print(f"the prompt with the norm in 8 bits: {far(eight, whole):.1e} from it", flush=True)


if __name__ == "__main__":
    main()
