"""Workloads of the block operators around the scan: layer norm (with the f32
residual stream) and the gated delta rule, in training, prefill and decoding.

``own`` False: the operators in plain form, elementary torch operations in 32
bits, rounded once at the end.  ``own`` True: the library's calls.  ``exact``
gives the same outputs from the definitions in 64 bits.

Gated delta rule, per batch row and value head (S is [head_k, head_v]; k and q
of key head h serve value heads h * v_heads / k_heads and the ones after it):

    S' = exp(g_t) S_{t-1}
    u  = beta_t (v_t - S'^T k_t)
    S_t = S' + k_t u^T
    o_t = scale S_t^T q_t

with q and k divided by their 2-norms first where ``l2norm`` is set.
"""

import math

import torch

own = False

EPS = 1e-5  # layer norm
L2_EPS = 1e-6  # added to the sum of squares under the square root

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# At most this many (token, value head) pairs in a training pass, and in a forward one.
MOST_TRAIN = 4 * 4096 * 40
MOST_FWD = 65536 * 16


def _norm(name, op, rows, dim, dtype, residual):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual}


def _delta(name, op, batch, t, hk, hv, dk, dv, dtype, state, packed=False):
    return {"name": name, "op": op, "batch": batch, "t": t, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "dtype": dtype,
            "state": state, "packed": packed, "l2norm": True}


def listed():
    return [
        # one token of 64 sequences through a block's norm (d_inner 5120, d_model 2560): latency
        _norm("norm_fwd_step_64x2560", "norm_fwd", 64, 2560, "bf16", True),
        # training or prefill of the 4 x 4096 x 5120 layer
        _norm("norm_fwd_16384x2560", "norm_fwd", 4 * 4096, 2560, "bf16", True),
        # the same block's backward at the 8 x 2048 x 1536 layer (d_model 768)
        _norm("norm_bwd_16384x768", "norm_bwd", 8 * 2048, 768, "bf16", True),
        # odd sizes, no residual stream, 32-bit activations
        _norm("norm_bwd_odd_4099x1003", "norm_bwd", 4099, 1003, "f32", False),
        # decoding: one sequence (latency), and 64 sequences of a 40-head layer with shared key heads
        _delta("delta_decode_b1_h16", "delta_decode", 1, 1, 16, 16, 128, 128, "bf16", True),
        _delta("delta_decode_b64_h40", "delta_decode", 64, 1, 20, 40, 128, 128, "bf16", True),
        # a short ragged prompt continued from a state, small heads
        _delta("delta_fwd_t77", "delta_fwd", 2, 77, 4, 8, 64, 96, "bf16", True),
        # prefill of the 8 x 2048 x 1536 layer, q, k and v as columns of one projection
        _delta("delta_fwd_b8_t2048_h12", "delta_fwd", 8, 2048, 12, 12, 128, 128, "bf16", False, True),
        # one long sequence, d_inner 2048
        _delta("delta_fwd_b1_t65536_h16", "delta_fwd", 1, 65536, 16, 16, 128, 128, "bf16", False),
        # training: the 8 x 128 x 512 trainer layer in 32 bits
        _delta("delta_train_f32_b8_t128_h4", "delta_train", 8, 128, 4, 4, 128, 128, "f32", False),
        # a window of a longer text, from and to a carried state, ragged, with shared key heads
        _delta("delta_train_b3_t1501_h12", "delta_train", 3, 1501, 6, 12, 128, 64, "bf16", True, True),
        # the 4 x 4096 x 5120 layer
        _delta("delta_train_b4_t4096_h40", "delta_train", 4, 4096, 20, 40, 128, 128, "bf16", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "delta_decode", "delta_fwd", "delta_fwd", "delta_train", "delta_train"])
    if op.startswith("norm"):
        dim = _log(rng, 64, 5120)
        dim -= 0 if rng.random() < 0.3 else dim % 8
        rows = _log(rng, 1, max(1, min(65536, 16384 * 2560 // dim)))
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        c = _norm("", op, rows, dim, dtype, rng.random() < 0.7)
    elif op == "delta_decode":
        share, hk = rng.choice([1, 1, 2, 4]), rng.randint(1, 20)
        hv = hk * share
        batch = _log(rng, 1, max(1, min(256, 64 * 40 // hv)))
        c = _delta("", op, batch, 1, hk, hv, rng.choice([64, 96, 128]), rng.choice([64, 128]),
                   "f32" if rng.random() < 0.2 else "bf16", True)
    else:
        share, hk = rng.choice([1, 1, 2, 3]), rng.randint(1, 16)
        hv = hk * share
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        most = (MOST_TRAIN if op == "delta_train" else MOST_FWD) // (16 if dtype == "f32" else 1)
        batch = rng.randint(1, 8)
        t = _log(rng, 1, max(1, min(65536 if op == "delta_fwd" else 16384, most // (batch * hv))))
        c = _delta("", op, batch, t, hk, hv, rng.choice([64, 80, 128, 128]), rng.choice([64, 72, 128, 128]), dtype,
                   rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def n(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def u(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        s["x"] = n(rows, dim, dtype=dt)
        s["weight"], s["bias"] = 1.0 + n(dim, std=0.1), n(dim, std=0.1)
        # a residual stream whose columns have offsets and scales of their own
        s["residual"] = n(rows, dim) * u(0.5, 3.0, dim) + n(dim, std=0.5) if case["residual"] else None
        if case["op"] == "norm_bwd":
            s["dy"] = n(rows, dim, dtype=dt)
            s["d_residual_out"] = n(rows, dim) if case["residual"] else None
            x = s["x"].float() if s["residual"] is None else s["residual"]  # what the forward normalised and left
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["normed"] = s["x"] if s["residual"] is None else s["residual"]
        return s
    b, t, hk, hv, dk, dv = (case[k] for k in ("batch", "t", "hk", "hv", "dk", "dv"))
    act = torch.nn.functional.silu
    qw, kw, vw = hk * dk, hk * dk, hv * dv
    if case["packed"]:  # columns of one projection's output
        row = act(n(b, t, qw + kw + vw)).to(dt)
        q, k, v = row[..., :qw], row[..., qw:qw + kw], row[..., qw + kw:]
    else:
        q, k, v = act(n(b, t, qw)).to(dt), act(n(b, t, kw)).to(dt), act(n(b, t, vw)).to(dt)
    s["q"], s["k"], s["v"] = q.unflatten(2, (hk, dk)), k.unflatten(2, (hk, dk)), v.unflatten(2, (hv, dv))
    # log decay as a Mamba layer makes it: -exp(a_log) softplus(delta_raw + dt_bias)
    a = u(1.0, 16.0, hv)
    step = torch.exp(u(math.log(1e-3), math.log(1e-1), hv))
    dt_bias = step + torch.log(-torch.expm1(-step))
    s["g"] = (-a * torch.nn.functional.softplus(n(b, t, hv) + dt_bias)).to(dt)
    s["beta"] = torch.sigmoid(n(b, t, hv)).to(dt)
    s["state"] = n(b, hv, dk, dv, std=0.3) if case["state"] else None
    if case["op"] == "delta_train":
        s["d_o"] = n(b, t, hv, dv, dtype=dt)
        s["d_state_out"] = n(b, hv, dk, dv, std=0.3) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from mamba_selective_scan_gb300 import binding as m3

    op, l2 = s["case"]["op"], s["case"].get("l2norm", False)
    if op == "norm_fwd":
        y, res, mean, rstd = m3.m3scan_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        return {"y": y, "residual": res, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return m3.m3scan_norm_bwd(s["dy"], s["normed"], s["weight"], s["mean"], s["rstd"], d_residual_out=s["d_residual_out"])
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "delta_decode":
        o = m3.m3scan_delta_decode(*args, s["state"], qk_l2norm=l2)
        return {"o": o, "state": s["state"]}
    if op == "delta_fwd":
        o, st, _ = m3.m3scan_delta_fwd(*args, state=s["state"], qk_l2norm=l2)
        return {"o": o, "state": st}
    with_state = s["state"] is not None
    o, st, ckpt = m3.m3scan_delta_fwd(*args, state=s["state"], qk_l2norm=l2, want_ckpt=True, want_state=with_state)
    g = m3.m3scan_delta_bwd(*args, ckpt, s["d_o"], d_state_out=s["d_state_out"], want_d_state=with_state, qk_l2norm=l2)
    return {"o": o, "state": st, **g}


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "norm_fwd":
        x = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"]
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(1) + EPS)
        y = c * rstd[:, None] * s["weight"] + s["bias"]
        return {"y": y.to(dt), "residual": x if s["residual"] is not None else None, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (s["normed"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        wdy = dy * s["weight"]
        dx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
        if s["d_residual_out"] is not None:
            dx = dx + s["d_residual_out"]
        return {"dx": dx.to(dt), "d_residual": dx if s["d_residual_out"] is not None else None,
                "d_weight": (dy * xh).sum(0), "d_bias": dy.sum(0)}
    ins = [s[k].float() for k in ("q", "k", "v", "g", "beta")]
    if op == "delta_decode":
        q, k, v, g, beta = (x[:, 0] for x in ins)
        q, k = _plain_heads(q, k, v.shape[1], case["l2norm"])
        st = s["state"] * torch.exp(g)[..., None, None]
        w = beta[..., None] * (v - (st * k[..., None]).sum(-2))
        st = st + k[..., None] * w[..., None, :]
        o = (st * q[..., None]).sum(-2) * case["dk"] ** -0.5
        s["state"].copy_(st)
        return {"o": o.to(dt)[:, None], "state": s["state"]}
    if op == "delta_fwd":
        with torch.no_grad():
            o, st = _plain_delta(*ins, s["state"], case["dk"] ** -0.5, case["l2norm"])
        return {"o": o.to(dt), "state": st}
    with_state = s["state"] is not None
    leaves = [x.detach().requires_grad_() for x in ins + ([s["state"]] if with_state else [])]
    o, st = _plain_delta(*leaves[:5], leaves[5] if with_state else None, case["dk"] ** -0.5, case["l2norm"])
    outs, ups = ([o, st], [s["d_o"].float(), s["d_state_out"]]) if with_state else ([o], [s["d_o"].float()])
    gr = torch.autograd.grad(outs, leaves, ups)
    r = {"o": o.detach().to(dt), "state": st.detach() if with_state else None}
    r.update({n: x.to(dt) for n, x in zip(("dq", "dk", "dv", "dg", "dbeta"), gr)})
    r["d_state"] = gr[5] if with_state else None
    return r


def _plain_heads(q, k, hv, l2norm):
    if l2norm:
        q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + L2_EPS)
        k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + L2_EPS)
    share = hv // k.shape[-2]
    return q.repeat_interleave(share, -2), k.repeat_interleave(share, -2)


def _plain_delta(q, k, v, g, beta, state, scale, l2norm, chunk=64):
    """Chunked form: within a chunk the updates u solve (I + A) u = beta (v - exp(gamma) S k), A strictly
    lower triangular; only the state goes from chunk to chunk."""
    b, t, hv, dv = v.shape
    q, k = _plain_heads(q, k, hv, l2norm)
    dk = k.shape[-1]
    pad = -t % chunk
    n = (t + pad) // chunk

    def chunks(x):  # [b, t, h, d] -> [b, h, n, chunk, d]
        return torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).transpose(1, 2).unflatten(2, (n, chunk))

    q, k, v = chunks(q * scale), chunks(k), chunks(v)
    g, beta = chunks(g[..., None])[..., 0], chunks(beta[..., None])
    gam = g.cumsum(-1)
    low = torch.ones(chunk, chunk, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(~low, float("-inf")))
    a = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1)
    # (I + A)^-1 by blocks of 1, 2, 4, ...: [[P, 0], [-R C P, R]]
    inv = torch.ones(b, hv, n, chunk, 1, 1, device=q.device)
    size = 1
    while size < chunk:
        blocks = a.unflatten(-1, (chunk // (2 * size), 2 * size)).unflatten(-3, (chunk // (2 * size), 2 * size))
        c = torch.diagonal(blocks, dim1=-4, dim2=-2).movedim(-1, -3)[..., size:, :size]
        p, r = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        inv = torch.cat([torch.cat([p, torch.zeros_like(p)], -1), torch.cat([-(r @ c @ p), r], -1)], -2)
        size *= 2
    inv = inv[..., 0, :, :]
    eg = torch.exp(gam)[..., None]
    uu, ww = inv @ (beta * v), inv @ (beta * eg * k)
    att = (q @ k.transpose(-1, -2)) * decay
    qg = q * eg
    kt = (k * torch.exp(gam[..., -1:] - gam)[..., None]).transpose(-1, -2)
    last = torch.exp(gam[..., -1])[..., None, None]
    st = torch.zeros(b, hv, dk, dv, device=q.device) if state is None else state
    outs = []
    for i in range(n):  # the state's way through the chunks
        u = uu[:, :, i] - ww[:, :, i] @ st
        outs.append(qg[:, :, i] @ st + att[:, :, i] @ u)
        st = last[:, :, i] * st + kt[:, :, i] @ u
    o = torch.cat(outs, 2) if outs else v.new_zeros(b, hv, 0, dv)
    return o[:, :, :t].transpose(1, 2), st


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, rows, dim = case["rows"] * case["dim"], case["rows"], case["dim"]
        if case["op"] == "norm_fwd":  # x, y, the residual stream in and out, the parameters, mean and rstd
            return {"bytes": n * (2 * e + (8 if case["residual"] else 0)) + 8 * dim + 8 * rows, "flops": 9 * n}
        # dy, the normalised input, dx, the residual stream's gradient in and out, the weight and its gradients
        per = 2 * e + (12 if case["residual"] else e)
        return {"bytes": n * per + 12 * dim + 8 * rows, "flops": 15 * n}
    b, t, hk, hv, dk, dv = (case[k] for k in ("batch", "t", "hk", "hv", "dk", "dv"))
    qk, vo, gate, st = b * t * hk * dk * e, b * t * hv * dv * e, b * t * hv * e, b * hv * dk * dv * 4
    fwd = 2 * qk + 2 * vo + 2 * gate
    flops = 6 * b * t * hv * dk * dv  # S'^T k, k u^T, S^T q
    if case["op"] == "delta_decode":
        return {"bytes": fwd + 2 * st, "flops": flops}
    if case["op"] == "delta_fwd":
        return {"bytes": fwd + (2 if case["state"] else 1) * st, "flops": flops}
    # training: q, k, v, g, beta, d_o read once; o and five gradients written once (and the states' ways in and out)
    back = 2 * qk + 2 * vo + 2 * gate
    return {"bytes": fwd + back + (4 * st if case["state"] else 0), "flops": 4 * flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "norm_fwd":
        h = f["x"] + f["residual"] if case["residual"] else f["x"]
        var, mean = torch.var_mean(h, dim=1, correction=0)
        sd = (var + EPS).sqrt()
        y = (h - mean.unsqueeze(1)) / sd.unsqueeze(1) * f["weight"] + f["bias"]
        return {"y": y, "residual": h if case["residual"] else None, "mean": mean, "rstd": 1 / sd}
    if case["op"] == "norm_bwd":
        # the derivative of sum(dy * y) for the mean and rstd that the pass is given
        dim = case["dim"]
        z = (f["normed"] - f["mean"].unsqueeze(1)) * f["rstd"].unsqueeze(1)
        e = f["dy"] * f["weight"]
        dots = torch.stack([e.sum(1), (e * z).sum(1)], 1) / dim
        d = (e - dots[:, :1] - z * dots[:, 1:]) * f["rstd"].unsqueeze(1)
        if case["residual"]:
            d += f["d_residual_out"]
        return {"dx": d, "d_residual": d if case["residual"] else None, "d_weight": torch.einsum("rd,rd->d", f["dy"], z),
                "d_bias": f["dy"].sum(0)}
    return _exact_delta(case, f)


def _exact_delta(case, f):
    """Token by token; the reverse pass recomputes the states of 64 tokens at a time."""
    b, t, hv, dk, dv = (case[k] for k in ("batch", "t", "hv", "dk", "dv"))
    if t > 20000 and case["op"] == "delta_train":
        return None
    share, scale = hv // case["hk"], dk ** -0.5
    nq = nk = 1.0
    if case["l2norm"]:
        nq = (f["q"] ** 2).sum(-1, keepdim=True).add(L2_EPS).sqrt()
        nk = (f["k"] ** 2).sum(-1, keepdim=True).add(L2_EPS).sqrt()
    heads = torch.arange(hv, device="cuda") // share
    q, k = (f["q"] / nq)[:, :, heads] * scale, (f["k"] / nk)[:, :, heads]
    # time first, so that a step's values are one slice
    q, k, v = (x.transpose(0, 1).contiguous() for x in (q, k, f["v"]))
    a, beta = f["g"].exp().transpose(0, 1).contiguous(), f["beta"].transpose(0, 1).contiguous()
    m = torch.zeros(b, hv, dk, dv, dtype=torch.float64, device="cuda")
    if case["state"]:
        m = m + f["state"]

    def step(m, i):
        m1 = m * a[i][..., None, None]
        gap = v[i] - torch.einsum("bhkv,bhk->bhv", m1, k[i])
        return m1, gap, m1 + torch.einsum("bhk,bhv->bhkv", k[i], beta[i][..., None] * gap)

    o = torch.empty(t, b, hv, dv, dtype=torch.float64, device="cuda")
    starts = []
    for i in range(t):
        if i % 64 == 0 and case["op"] == "delta_train":
            starts.append(m)
        m = step(m, i)[2]
        o[i] = torch.einsum("bhkv,bhk->bhv", m, q[i])
    out = {"o": o.transpose(0, 1)}
    if case["op"] != "delta_train":
        return {**out, "state": m}
    out["state"] = m if case["state"] else None
    d = f["d_state_out"].clone() if case["state"] else torch.zeros_like(m)
    do = f["d_o"].transpose(0, 1).contiguous()
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    da, dbeta = torch.zeros_like(a), torch.zeros_like(beta)
    for c in range(len(starts) - 1, -1, -1):
        lo, hi = 64 * c, min(t, 64 * c + 64)
        kept, m = [], starts[c]
        for i in range(lo, hi):
            m1, gap, nxt = step(m, i)
            kept.append((m, m1, gap, nxt))
            m = nxt
        for i in range(hi - 1, lo - 1, -1):
            m0, m1, gap, nxt = kept.pop()
            dq[i] = torch.einsum("bhkv,bhv->bhk", nxt, do[i])
            d = d + torch.einsum("bhk,bhv->bhkv", q[i], do[i])
            du = torch.einsum("bhkv,bhk->bhv", d, k[i])
            dbeta[i] = (du * gap).sum(-1)
            dgap = beta[i][..., None] * du
            dv_[i] = dgap
            dk_[i] = torch.einsum("bhkv,bhv->bhk", d, beta[i][..., None] * gap) - torch.einsum("bhkv,bhv->bhk", m1, dgap)
            d = d - torch.einsum("bhk,bhv->bhkv", k[i], dgap)
            da[i] = torch.einsum("bhkv,bhkv->bh", d, m0)
            d = d * a[i][..., None, None]

    def shared(x, raw, norm):  # sums over the value heads of a key head, then back through the division by the norm
        x = x.transpose(0, 1).unflatten(2, (case["hk"], share)).sum(3)
        if not case["l2norm"]:
            return x
        unit = raw / norm
        return (x - unit * (unit * x).sum(-1, keepdim=True)) / norm

    out.update(dq=shared(dq * scale, f["q"], nq), dk=shared(dk_, f["k"], nk), dv=dv_.transpose(0, 1),
               dg=(da * a).transpose(0, 1), dbeta=dbeta.transpose(0, 1), d_state=d if case["state"] else None)
    return out
