"""Linear attention with a decay per head, and the norm and rotation of queries
and keys, in float64 from their definitions; gradients by autograd."""

import torch


def lin_inputs(B, T, Hk, Hv, dk, dv, dtype, seed=0, device="cpu", state=True, packed=False, log_decay=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    if packed:
        row = r(B, T, 2 * Hk * dk + Hv * dv).to(dtype).to(device)
        q, k, v = row.split([Hk * dk, Hk * dk, Hv * dv], -1)
        q, k, v = q.unflatten(2, (Hk, dk)), k.unflatten(2, (Hk, dk)), v.unflatten(2, (Hv, dv))
    else:
        q, k, v = (r(B, T, h, d).to(dtype).to(device) for h, d in ((Hk, dk), (Hk, dk), (Hv, dv)))
    if log_decay is None:  # slow, middling and fast heads
        log_decay = -torch.exp(-7.5 + 8.5 * torch.rand(Hv, generator=g))
    else:
        log_decay = torch.tensor([log_decay[h % len(log_decay)] for h in range(Hv)], dtype=torch.float32)
    return {"q": q, "k": k, "v": v, "log_decay": log_decay.to(device), "d_o": r(B, T, Hv, dv).to(dtype).to(device),
            "state": (0.3 * r(B, Hv, dk, dv)).to(device) if state else None,
            "d_state_out": (0.3 * r(B, Hv, dk, dv)).to(device) if state else None}


def lin_ref(q, k, v, log_decay, state, scale):
    """(o, state) of float64 tensors; differentiable."""
    B, T, Hv, dv = v.shape
    Hk, dk = k.shape[2:]
    q, k = (x.repeat_interleave(Hv // Hk, 2) for x in (q, k))
    lam = log_decay.exp()[:, None, None]
    S = torch.zeros(B, Hv, dk, dv, dtype=v.dtype, device=v.device) if state is None else state
    outs = []
    for t in range(T):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(scale * (S * q[:, t, :, :, None]).sum(-2))
    return (torch.stack(outs, 1) if outs else v.new_zeros(B, 0, Hv, dv)), S


def lin_ref_grads(x, scale, ref=lin_ref):
    """float64 results and gradients on x's values: dict with o, state_out, dq,
    dk, dv and d_state."""
    names = ["q", "k", "v"] + (["state"] if x["state"] is not None else [])
    f = {n: x[n].detach().double().clone().requires_grad_() for n in names}
    o, S = ref(f["q"], f["k"], f["v"], x["log_decay"].double(), f.get("state"), scale)
    loss = (o * x["d_o"].double()).sum()
    if x["d_state_out"] is not None:
        loss = loss + (S * x["d_state_out"].double()).sum()
    grads = torch.autograd.grad(loss, [f[n] for n in names], allow_unused=True)
    r = {"o": o.detach().cpu(), "state_out": S.detach().cpu()}
    for n, gr in zip(names, grads):
        r["d_state" if n == "state" else "d" + n] = (torch.zeros_like(f[n]) if gr is None else gr).cpu()
    return r


def rot_inputs(B, T, Hq, Hk, D, rot, dtype, seed=0, device="cpu", start=1000, packed=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    if packed:
        row = r(B, T, (Hq + Hk) * D).to(dtype).to(device)
        q, k = row[..., :Hq * D].unflatten(2, (Hq, D)), row[..., Hq * D:].unflatten(2, (Hk, D))
    else:
        q, k = r(B, T, Hq, D).to(dtype).to(device), r(B, T, Hk, D).to(dtype).to(device)
    R = rot // 2
    return {"q": q, "k": k, "q_weight": (1 + 0.2 * r(D)).to(device), "k_weight": (1 + 0.2 * r(D)).to(device),
            "positions": (torch.randint(0, start + 1, (B, 1), generator=g) + torch.arange(T)).to(device),
            "inv_freq": (10000.0 ** (-torch.arange(R, dtype=torch.float64) / max(R, 1))).float().to(device),
            "dq_out": r(B, T, Hq, D).to(dtype).to(device), "dk_out": r(B, T, Hk, D).to(dtype).to(device)}


def rot_ref(x, w, positions, inv_freq, eps, interleaved):
    """One tensor [B, T, H, D] normalised and turned, float64; differentiable
    in x and w."""
    D, R = x.shape[-1], inv_freq.numel()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        n = n * w
    f = (positions.double()[..., None] * inv_freq.double()).expand(*x.shape[:2], R)[:, :, None]
    if interleaved:
        a, b = n[..., 0:2 * R:2], n[..., 1:2 * R:2]
    else:
        a, b = n[..., :R], n[..., R:2 * R]
    a, b = a * f.cos() - b * f.sin(), a * f.sin() + b * f.cos()
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, n[..., 2 * R:]], -1)


def rot_ref_grads(x, eps, interleaved):
    r = {}
    for n in "qk":
        t = x[n].detach().double().clone().requires_grad_()
        w = x[n + "_weight"]
        w = None if w is None else w.double().clone().requires_grad_()
        y = rot_ref(t, w, x["positions"], x["inv_freq"], eps, interleaved)
        g = torch.autograd.grad((y * x[f"d{n}_out"].double()).sum(), [t] + ([] if w is None else [w]))
        r[n + "_out"], r["d" + n] = y.detach().cpu(), g[0].cpu()
        r[f"d_{n}_weight"] = None if w is None else g[1].cpu()
    return r


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference (absolute
    where the reference is zero)."""
    got = got.double().cpu()
    if not torch.isfinite(got).all():
        return float("inf")
    n = ref.norm().item()
    return (got - ref).norm().item() / (n if n > 0 else 1.0)


def lin_ref_chunked(q, k, v, log_decay, state, scale, chunk=64):
    """``lin_ref`` by chunks, for long sequences of finite values;
    differentiable."""
    B, T, Hv, dv = v.shape
    Hk, dk = k.shape[2:]
    q, k, v = (x.repeat_interleave(Hv // x.shape[2], 2).transpose(1, 2) for x in (q, k, v))  # [B, H, T, d]
    S = torch.zeros(B, Hv, dk, dv, dtype=v.dtype, device=v.device) if state is None else state
    i = torch.arange(chunk, device=v.device)
    ld = log_decay[:, None, None]
    pairs = torch.where(i[:, None] < i, 0.0, torch.exp(ld * (i[:, None] - i).clamp(min=0)))
    outs = []
    for t in range(0, T, chunk):
        qc, kc, vc = (x[:, :, t:t + chunk] for x in (q, k, v))
        n = vc.shape[2]
        o = ((qc @ kc.transpose(-1, -2)) * pairs[:, :n, :n]) @ vc + torch.exp(ld * (i[:n, None] + 1)) * (qc @ S)
        S = torch.exp(ld * n) * S + (kc * torch.exp(ld * (n - 1 - i[:n, None]))).transpose(-1, -2) @ vc
        outs.append(scale * o)
    return torch.cat(outs, 2).transpose(1, 2), S
