"""A pre-norm block whose mixer is the gated delta rule: a training step, the
prefill of a prompt, and decoding from the state it leaves.

    r = x + residual (f32)            m3scan_norm_fwd
    h = norm(r)
    q, k, v, a, b = h @ w_in          one projection; q, k, v stay column views
    g = -exp(a_log) softplus(a + dt_bias),  beta = sigmoid(b)
    o = delta rule(q, k, v, g, beta)  m3scan_delta_fwd / m3scan_delta_decode
    y = o @ w_out                     the next block's x, beside r

Run with ``python examples/gated_delta_block.py`` on a GPU."""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
import torch.nn.functional as F

from mamba_selective_scan_gb300 import binding as m3


class GatedDeltaBlock:
    """Weights and calls of one block; ``dtype`` is the activations'."""

    def __init__(self, d_model, k_heads, v_heads, head_k=128, head_v=128, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)
        self.hk, self.hv, self.dk, self.dv = k_heads, v_heads, head_k, head_v
        self.widths = [k_heads * head_k, k_heads * head_k, v_heads * head_v, v_heads, v_heads]
        self.norm_w, self.norm_b = torch.ones(d_model, device=device), torch.zeros(d_model, device=device)
        self.w_in = (rand(d_model, sum(self.widths)) * d_model ** -0.5).to(dtype)
        self.w_out = (rand(v_heads * head_v, d_model) * (v_heads * head_v) ** -0.5).to(dtype)
        self.a_log = torch.log(1 + 15 * torch.rand(v_heads, generator=g, device=device))
        self.dt_bias = rand(v_heads) - 4.0

    def _split(self, p):
        """Views of q, k, v in the projection's output, and what the gates are made of."""
        q, k, v, a, b = p.split(self.widths, -1)
        return q.unflatten(-1, (self.hk, self.dk)), k.unflatten(-1, (self.hk, self.dk)), v.unflatten(-1, (self.hv, self.dv)), a, b

    def _gates(self, a, b):
        g = -torch.exp(self.a_log) * F.softplus(a.float() + self.dt_bias)
        return g.to(a.dtype), torch.sigmoid(b.float()).to(b.dtype)

    def _pad(self, p):
        """The projection with its rows padded to 16 bytes, as the views' token stride must be."""
        extra = -p.shape[-1] % (16 // p.element_size())
        return F.pad(p, (0, extra)) if extra else p

    def forward(self, x, residual=None, state=None, train=False):
        """x [B, T, d_model], residual f32.  Returns (y, r, state, saved)."""
        h, r, mean, rstd = m3.m3scan_norm_fwd(x, self.norm_w, self.norm_b, residual=residual,
                                              residual_out=None if residual is not None else torch.empty_like(x, dtype=torch.float32))
        p = self._pad(h @ self.w_in)
        q, k, v, a, b = self._split(p[..., :sum(self.widths)])
        g, beta = self._gates(a, b)
        o, state, ckpt = m3.m3scan_delta_fwd(q, k, v, g, beta, state=state, qk_l2norm=True, want_ckpt=train)
        y = o.flatten(2) @ self.w_out
        return y, r, state, (h, r, mean, rstd, p, g, beta, o, ckpt) if train else None

    def backward(self, saved, dy, dr):
        """Gradients of a training step: (dx, d_residual, dict of the weights'); dr is what reaches r past this block (f32)."""
        h, r, mean, rstd, p, g, beta, o, ckpt = saved
        n = sum(self.widths)
        q, k, v, a, b = self._split(p[..., :n])
        w = {"w_out": o.flatten(0, 1).flatten(1).t() @ dy.flatten(0, 1)}
        d_o = (dy @ self.w_out.t()).unflatten(2, (self.hv, self.dv))
        dp = torch.zeros_like(p)  # dq, dk and dv land in their columns
        dq, dk, dv, da, db = self._split(dp[..., :n])
        gr = m3.m3scan_delta_bwd(q, k, v, g, beta, ckpt, d_o, qk_l2norm=True, out={"dq": dq, "dk": dk, "dv": dv})
        dg = gr["dg"].float() * -torch.exp(self.a_log)
        w["a_log"] = (gr["dg"].float() * g.float()).sum((0, 1))
        da.copy_(dg * torch.sigmoid(a.float() + self.dt_bias))
        w["dt_bias"] = (dg * torch.sigmoid(a.float() + self.dt_bias)).sum((0, 1))
        db.copy_(gr["dbeta"].float() * beta.float() * (1 - beta.float()))
        d_in = dp[..., :n]
        w["w_in"] = h.flatten(0, 1).t() @ d_in.flatten(0, 1)
        dh = d_in @ self.w_in.t()
        nb = m3.m3scan_norm_bwd(dh, r, self.norm_w, mean, rstd, d_residual_out=dr)
        w["norm_w"], w["norm_b"] = nb["d_weight"], nb["d_bias"]
        return nb["dx"], nb["d_residual"], w

    def decode(self, x, residual, state):
        """One token per sequence, x [B, 1, d_model]; ``state`` is updated in place.  Returns (y, r)."""
        h, r, _, _ = m3.m3scan_norm_fwd(x, self.norm_w, self.norm_b, residual=residual, want_stats=False,
                                        residual_out=None if residual is not None else torch.empty_like(x, dtype=torch.float32))
        p = self._pad(h @ self.w_in)
        q, k, v, a, b = self._split(p[..., :sum(self.widths)])
        g, beta = self._gates(a, b)
        o = m3.m3scan_delta_decode(q, k, v, g, beta, state, qk_l2norm=True)
        return o.flatten(2) @ self.w_out, r


def main():
    torch.manual_seed(0)
    block = GatedDeltaBlock(1024, 8, 16)
    x = torch.randn(2, 300, 1024, device="cuda", dtype=torch.bfloat16)
    y, r, state, saved = block.forward(x, train=True)
    dx, _, grads = block.backward(saved, torch.randn_like(y), torch.zeros_like(r))
    print("training step:", {n: tuple(g.shape) for n, g in grads.items()}, "dx", tuple(dx.shape))
    _, _, state, _ = block.forward(x[:, :299].contiguous())
    last, _ = block.decode(x[:, 299:].contiguous(), None, state)
    err = ((last - y[:, 299:]).float().norm() / y[:, 299:].float().norm()).item()
    print(f"last token decoded from the prompt's state: off by {err:.1e} of the full pass")


if __name__ == "__main__":
    main()
