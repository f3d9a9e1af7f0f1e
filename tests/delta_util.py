"""Gated delta rule and layer norm in float64, from their definitions: the
recurrence token by token, gradients by autograd through it."""

import torch

L2_EPS = 1e-6


def delta_inputs(B, T, Hk, Hv, dk, dv, dtype, seed=0, device="cpu", state=True, packed=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    act = torch.nn.functional.silu
    if packed:
        row = act(r(B, T, 2 * Hk * dk + Hv * dv)).to(dtype).to(device)
        q, k, v = row.split([Hk * dk, Hk * dk, Hv * dv], -1)
        q, k, v = q.unflatten(2, (Hk, dk)), k.unflatten(2, (Hk, dk)), v.unflatten(2, (Hv, dv))
    else:
        q, k, v = (act(r(B, T, h, d)).to(dtype).to(device) for h, d in ((Hk, dk), (Hk, dk), (Hv, dv)))
    gl = (-torch.nn.functional.softplus(r(B, T, Hv) - 2.0) * (0.5 + 8 * torch.rand(Hv, generator=g))).to(dtype)
    beta = torch.sigmoid(r(B, T, Hv)).to(dtype)
    x = {"q": q, "k": k, "v": v, "g": gl.to(device), "beta": beta.to(device),
         "d_o": r(B, T, Hv, dv).to(dtype).to(device),
         "state": (0.3 * r(B, Hv, dk, dv)).to(device) if state else None,
         "d_state_out": (0.3 * r(B, Hv, dk, dv)).to(device) if state else None}
    return x


def delta_ref(q, k, v, g, beta, state, scale, l2norm):
    """(o, state) of float64 tensors; differentiable."""
    B, T, Hv, dv = v.shape
    Hk, dk = k.shape[2:]
    if l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + L2_EPS).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + L2_EPS).sqrt()
    q, k = (x.repeat_interleave(Hv // Hk, 2) for x in (q, k))
    S = torch.zeros(B, Hv, dk, dv, dtype=v.dtype, device=v.device) if state is None else state
    outs = []
    for t in range(T):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + torch.einsum("bhk,bhv->bhkv", k[:, t], u)
        outs.append(scale * torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    return (torch.stack(outs, 1) if outs else v.new_zeros(B, 0, Hv, dv)), S


def delta_ref_grads(x, scale, l2norm):
    """float64 results and gradients on x's values: dict with o, state_out and
    d<input>."""
    names = ["q", "k", "v", "g", "beta"] + (["state"] if x["state"] is not None else [])
    f = {n: x[n].detach().double().cpu().clone().requires_grad_() for n in names}
    o, S = delta_ref(f["q"], f["k"], f["v"], f["g"], f["beta"], f.get("state"), scale, l2norm)
    loss = (o * x["d_o"].double().cpu()).sum()
    if x["d_state_out"] is not None:
        loss = loss + (S * x["d_state_out"].double().cpu()).sum()
    grads = torch.autograd.grad(loss, [f[n] for n in names], allow_unused=True)
    r = {"o": o.detach(), "state_out": S.detach()}
    for n, gr in zip(names, grads):
        r["d_state" if n == "state" else "d" + n] = torch.zeros_like(f[n]) if gr is None else gr
    return r


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference (absolute
    where the reference is zero)."""
    got = got.double().cpu()
    if not torch.isfinite(got).all():
        return float("inf")
    n = ref.norm().item()
    return (got - ref).norm().item() / (n if n > 0 else 1.0)
