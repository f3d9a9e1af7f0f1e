"""A pre-norm block whose mixer is linear attention with a decay for each head
and rotated queries and keys: a training step, the prefill of a prompt, and
decoding from the state it leaves.

    r = x + residual (f32)            m3scan_norm_fwd
    h = norm(r)
    q, k, v = h @ w_in                one projection; q, k, v stay column views
    q, k = rotate(norm(q)), ...       m3scan_qkrot_fwd
    o = linear attention(q, k, v)     m3scan_linattn_fwd / m3scan_linattn_decode
    y = o @ w_out                     the next block's x, beside r

Run with ``python examples/linear_attention_block.py`` on a GPU."""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mamba_selective_scan_gb300 import binding as m3


class LinearAttentionBlock:
    """Weights and calls of one block; ``dtype`` is the activations'."""

    def __init__(self, d_model, k_heads, v_heads, head_k=128, head_v=128, rot=None, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)
        self.hk, self.hv, self.dk, self.dv = k_heads, v_heads, head_k, head_v
        self.widths = [k_heads * head_k, k_heads * head_k, v_heads * head_v]
        self.norm_w, self.norm_b = torch.ones(d_model, device=device), torch.zeros(d_model, device=device)
        self.w_in = (rand(d_model, sum(self.widths)) * d_model ** -0.5).to(dtype)
        self.w_out = (rand(v_heads * head_v, d_model) * (v_heads * head_v) ** -0.5).to(dtype)
        self.q_weight, self.k_weight = 1 + 0.1 * rand(head_k), 1 + 0.1 * rand(head_k)
        r = (head_k if rot is None else rot) // 2
        self.inv_freq = (10000.0 ** (-torch.arange(r, device=device, dtype=torch.float64) / r)).float()
        # heads that look back over some thousand tokens, down to a few
        self.log_decay = -torch.exp2(torch.linspace(-10.0, -1.0, v_heads, device=device))

    def _split(self, p):
        q, k, v = p.split(self.widths, -1)
        return q.unflatten(-1, (self.hk, self.dk)), k.unflatten(-1, (self.hk, self.dk)), v.unflatten(-1, (self.hv, self.dv))

    def _mixer_inputs(self, h, positions):
        p = h @ self.w_in
        q, k, v = self._split(p)
        qr, kr = m3.m3scan_qkrot_fwd(q, k, self.q_weight, self.k_weight, positions, self.inv_freq)
        return p, qr, kr, v

    def forward(self, x, residual=None, state=None, start=0, train=False):
        """x [B, T, d_model], residual f32; the first token is at position
        ``start``.  Returns (y, r, state, saved)."""
        h, r, mean, rstd = m3.m3scan_norm_fwd(x, self.norm_w, self.norm_b, residual=residual,
                                              residual_out=None if residual is not None else torch.empty_like(x, dtype=torch.float32))
        positions = torch.arange(start, start + x.shape[1], device=x.device)
        p, q, k, v = self._mixer_inputs(h, positions)
        o, state_out = m3.m3scan_linattn_fwd(q, k, v, self.log_decay, state=state)
        y = o.flatten(2) @ self.w_out
        return y, r, state_out, (h, r, mean, rstd, p, positions, q, k, o, state) if train else None

    def backward(self, saved, dy, dr):
        """Gradients of a training step: (dx, d_residual, dict of the weights'); dr is what reaches r past this block (f32)."""
        h, r, mean, rstd, p, positions, qr, kr, o, state = saved
        q, k, v = self._split(p)
        w = {"w_out": o.flatten(0, 1).flatten(1).t() @ dy.flatten(0, 1)}
        d_o = (dy @ self.w_out.t()).unflatten(2, (self.hv, self.dv))
        dp = torch.empty_like(p)  # dq, dk and dv land in their columns
        dq, dk, dv = self._split(dp)
        m3.m3scan_linattn_bwd(qr, kr, v, self.log_decay, d_o, state=state, out={"dq": dq, "dk": dk, "dv": dv})
        # (in place: of the rotated q and k, then of the projection's)
        gr = m3.m3scan_qkrot_bwd(dq, dk, q, k, self.q_weight, self.k_weight, positions, self.inv_freq, out={"dq": dq, "dk": dk})
        w["q_weight"], w["k_weight"] = gr["d_q_weight"], gr["d_k_weight"]
        w["w_in"] = h.flatten(0, 1).t() @ dp.flatten(0, 1)
        nb = m3.m3scan_norm_bwd(dp @ self.w_in.t(), r, self.norm_w, mean, rstd, d_residual_out=dr)
        w["norm_w"], w["norm_b"] = nb["d_weight"], nb["d_bias"]
        return nb["dx"], nb["d_residual"], w

    def decode(self, x, residual, state, positions):
        """One token per sequence, x [B, 1, d_model], at ``positions`` (int64
        [B, 1]); ``state`` is updated in place.  Returns (y, r)."""
        h, r, _, _ = m3.m3scan_norm_fwd(x, self.norm_w, self.norm_b, residual=residual, want_stats=False,
                                        residual_out=None if residual is not None else torch.empty_like(x, dtype=torch.float32))
        _, q, k, v = self._mixer_inputs(h, positions)
        o = m3.m3scan_linattn_decode(q, k, v, self.log_decay, state)
        return o.flatten(2) @ self.w_out, r


def main():
    torch.manual_seed(0)
    block = LinearAttentionBlock(1024, 8, 8)
    x = torch.randn(2, 300, 1024, device="cuda", dtype=torch.bfloat16)
    y, r, state, saved = block.forward(x, train=True)
    dx, _, grads = block.backward(saved, torch.randn_like(y), torch.zeros_like(r))
    print("training step:", {n: tuple(g.shape) for n, g in grads.items()}, "dx", tuple(dx.shape))
    _, _, state, _ = block.forward(x[:, :299].contiguous())
    last, _ = block.decode(x[:, 299:].contiguous(), None, state, torch.full((2, 1), 299, device="cuda"))
    err = ((last - y[:, 299:]).float().norm() / y[:, 299:].float().norm()).item()
    print(f"last token decoded from the prompt's state: off by {err:.1e} of the full pass")


if __name__ == "__main__":
    main()
