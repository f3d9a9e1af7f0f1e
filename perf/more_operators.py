"""Workloads of a linear-attention mixer: the norm and rotation of its queries
and keys, and linear attention with a decay per head, in training, prefill and
decoding.

``own`` False: the operators in plain form, elementary torch operations in 32
bits (angles and powers of the decays in 64), rounded once at the end.  ``own``
True: the library's calls.  ``exact`` gives the same outputs from the
definitions in 64 bits.

Queries and keys, per token and head x of ``dim`` values, ``rot`` = 2 R of them
rotated (pair i is (i, i + R), or (2 i, 2 i + 1) where ``interleaved``):

    n = x / sqrt(mean(x^2) + eps) * weight
    (a, b) of pair i  ->  (a cos f - b sin f, a sin f + b cos f),  f = position * inv_freq[i]

Linear attention, per batch row and value head (S is [head_k, head_v]; k and q
of key head h serve value heads h * v_heads / k_heads and the ones after it):

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T
    o_t = scale S_t^T q_t
"""

import math

import torch

own = False

EPS = 1e-6

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# At most this many (token, value head) pairs in a training pass, and in a forward one.
MOST_TRAIN = 4 * 4096 * 40
MOST_FWD = 65536 * 16
# At most this many (token, head) pairs of queries and keys together.
MOST_ROT = 4 * 4096 * 80


def _rot(name, op, batch, t, hq, hk, dim, rot, dtype, packed=False, interleaved=False, start=0):
    return {"name": name, "op": op, "batch": batch, "t": t, "hq": hq, "hk": hk, "dim": dim, "rot": rot, "dtype": dtype,
            "packed": packed, "interleaved": interleaved, "start": start}


def _lin(name, op, batch, t, hk, hv, dk, dv, dtype, state, packed=False):
    return {"name": name, "op": op, "batch": batch, "t": t, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "dtype": dtype,
            "state": state, "packed": packed}


def listed():
    return [
        # one token of 64 sequences, each at a place of its own in a long text: latency
        _rot("qkrot_fwd_step_64_h16", "qkrot_fwd", 64, 1, 16, 16, 128, 128, "bf16", start=500000),
        # training or prefill of the 4 x 4096 x 5120 layer, q and k as columns of one projection
        _rot("qkrot_fwd_b4_t4096_h40", "qkrot_fwd", 4, 4096, 40, 40, 128, 128, "bf16", packed=True),
        # the backward at the 8 x 2048 x 1536 layer
        _rot("qkrot_bwd_b8_t2048_h12", "qkrot_bwd", 8, 2048, 12, 12, 128, 128, "bf16"),
        # odd sizes in 32 bits: more query than key heads, part of a head rotated, neighbouring pairs
        _rot("qkrot_bwd_odd_b3_t1501", "qkrot_bwd", 3, 1501, 10, 5, 80, 48, "f32", interleaved=True, start=70001),
        # decoding: one sequence (latency), and 64 sequences of a 40-head layer
        _lin("linattn_decode_b1_h16", "linattn_decode", 1, 1, 16, 16, 128, 128, "bf16", True),
        _lin("linattn_decode_b64_h40", "linattn_decode", 64, 1, 40, 40, 128, 128, "bf16", True),
        # a short ragged prompt continued from a state, small heads, shared keys
        _lin("linattn_fwd_t77", "linattn_fwd", 2, 77, 4, 8, 64, 96, "bf16", True),
        # prefill of the 8 x 2048 x 1536 layer, q, k and v as columns of one projection
        _lin("linattn_fwd_b8_t2048_h12", "linattn_fwd", 8, 2048, 12, 12, 128, 128, "bf16", False, True),
        # one long sequence, d_inner 2048
        _lin("linattn_fwd_b1_t65536_h16", "linattn_fwd", 1, 65536, 16, 16, 128, 128, "bf16", False),
        # training: the 8 x 128 x 512 trainer layer in 32 bits
        _lin("linattn_train_f32_b8_t128_h4", "linattn_train", 8, 128, 4, 4, 128, 128, "f32", False),
        # a window of a longer text, from and to a carried state, ragged, with shared key heads
        _lin("linattn_train_b3_t1501_h12", "linattn_train", 3, 1501, 6, 12, 128, 64, "bf16", True, True),
        # the 4 x 4096 x 5120 layer
        _lin("linattn_train_b4_t4096_h40", "linattn_train", 4, 4096, 40, 40, 128, 128, "bf16", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qkrot_fwd", "qkrot_bwd", "linattn_decode", "linattn_fwd", "linattn_fwd", "linattn_train", "linattn_train"])
    if op.startswith("qkrot"):
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        hk = rng.randint(1, 20)
        hq = hk * rng.choice([1, 1, 2, 4])
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        most = MOST_ROT * 128 // (dim * (hq + hk)) // (2 if dtype == "f32" else 1) // (2 if op == "qkrot_bwd" else 1)
        batch = _log(rng, 1, 64)
        t = 1 if rng.random() < 0.15 else _log(rng, 1, max(1, min(65536, most // batch)))
        c = _rot("", op, batch, t, hq, hk, dim, rot, dtype, rng.random() < 0.5, rng.random() < 0.4, _log(rng, 1, 10 ** 6))
    elif op == "linattn_decode":
        share, hk = rng.choice([1, 1, 2, 4]), rng.randint(1, 20)
        hv = hk * share
        batch = _log(rng, 1, max(1, min(256, 64 * 40 // hv)))
        c = _lin("", op, batch, 1, hk, hv, rng.choice([64, 96, 128]), rng.choice([64, 128]),
                 "f32" if rng.random() < 0.2 else "bf16", True)
    else:
        share, hk = rng.choice([1, 1, 2, 3]), rng.randint(1, 16)
        hv = hk * share
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        most = (MOST_TRAIN if op == "linattn_train" else MOST_FWD) // (16 if dtype == "f32" else 1) // share
        batch = rng.randint(1, 8)
        t = _log(rng, 1, max(1, min(65536 if op == "linattn_fwd" else 16384, most // (batch * hv))))
        c = _lin("", op, batch, t, hk, hv, rng.choice([64, 80, 128, 128]), rng.choice([64, 72, 128, 128]), dtype,
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

    def columns(packed, *heads):  # (heads, size) of each tensor: columns of one projection's output, or each on its own
        widths = [h * d for h, d in heads]
        if packed:
            parts = n(b, t, sum(widths), dtype=dt).split(widths, 2)
        else:
            parts = [n(b, t, w, dtype=dt) for w in widths]
        return [p.unflatten(2, hd) for p, hd in zip(parts, heads)]

    b, t = case["batch"], case["t"]
    s = {"case": case}
    if case["op"].startswith("qkrot"):
        d, r = case["dim"], case["rot"] // 2
        s["q"], s["k"] = columns(case["packed"], (case["hq"], d), (case["hk"], d))
        s["q_weight"], s["k_weight"] = 1.0 + n(d, std=0.1), 1.0 + n(d, std=0.1)
        # every sequence goes on from a place of its own
        first = (u(0.0, 1.0, b, 1).double() * (case["start"] + 1)).long()
        s["positions"] = first + torch.arange(t, device="cuda")
        s["inv_freq"] = (10000.0 ** (-torch.arange(r, device="cuda", dtype=torch.float64) / r)).float()
        if case["op"] == "qkrot_bwd":
            s["dq_out"], s["dk_out"] = n(b, t, case["hq"], d, dtype=dt), n(b, t, case["hk"], d, dtype=dt)
        return s
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    s["q"], s["k"], s["v"] = columns(case["packed"], (hk, dk), (hk, dk), (hv, dv))
    # from heads that look back over thousands of tokens to heads that see a few
    s["log_decay"] = -torch.exp(u(math.log(2.0 ** -11), math.log(0.7), hv))
    s["state"] = n(b, hv, dk, dv, std=0.3) if case["state"] else None
    if case["op"] == "linattn_train":
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

    case = s["case"]
    op = case["op"]
    if op.startswith("qkrot"):
        rest = (s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"])
        if op == "qkrot_fwd":
            q, k = m3.m3scan_qkrot_fwd(*rest, eps=EPS, interleaved=case["interleaved"])
            return {"q": q, "k": k}
        return m3.m3scan_qkrot_bwd(s["dq_out"], s["dk_out"], *rest, eps=EPS, interleaved=case["interleaved"])
    args = (s["q"], s["k"], s["v"], s["log_decay"])
    if op == "linattn_decode":
        o = m3.m3scan_linattn_decode(*args, s["state"])
        return {"o": o, "state": s["state"]}
    if op == "linattn_fwd":
        o, st = m3.m3scan_linattn_fwd(*args, state=s["state"])
        return {"o": o, "state": st}
    with_state = s["state"] is not None
    o, st = m3.m3scan_linattn_fwd(*args, state=s["state"], want_state=with_state)
    g = m3.m3scan_linattn_bwd(*args, s["d_o"], state=s["state"], d_state_out=s["d_state_out"], want_d_state=with_state)
    return {"o": o, "state": st, **g}


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op.startswith("qkrot"):
        f = s["positions"].double()[:, :, None, None] * s["inv_freq"].double()
        turn = (f.cos().float(), f.sin().float(), case["interleaved"])
        if op == "qkrot_fwd":
            return {"q": _plain_turn(_plain_norm(s["q"], s["q_weight"])[0], *turn).to(dt),
                    "k": _plain_turn(_plain_norm(s["k"], s["k_weight"])[0], *turn).to(dt)}
        dq, dwq = _plain_rot_bwd(s["dq_out"], s["q"], s["q_weight"], turn)
        dk, dwk = _plain_rot_bwd(s["dk_out"], s["k"], s["k_weight"], turn)
        return {"dq": dq.to(dt), "dk": dk.to(dt), "d_q_weight": dwq, "d_k_weight": dwk}
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    scale = case["dk"] ** -0.5
    if op == "linattn_decode":
        share = case["hv"] // case["hk"]
        q, k, v = (x[:, 0] for x in (q.repeat_interleave(share, 2), k.repeat_interleave(share, 2), v))
        st = s["state"] * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
        o = (st * q[..., None]).sum(-2) * scale
        s["state"].copy_(st)
        return {"o": o.to(dt)[:, None], "state": s["state"]}
    if op == "linattn_fwd":
        with torch.no_grad():
            o, st = _plain_lin(q, k, v, s["log_decay"], s["state"], scale)
        return {"o": o.to(dt), "state": st}
    with_state = s["state"] is not None
    leaves = [x.detach().requires_grad_() for x in [q, k, v] + ([s["state"]] if with_state else [])]
    o, st = _plain_lin(*leaves[:3], s["log_decay"], leaves[3] if with_state else None, scale)
    outs, ups = ([o, st], [s["d_o"].float(), s["d_state_out"]]) if with_state else ([o], [s["d_o"].float()])
    gr = torch.autograd.grad(outs, leaves, ups)
    r = {"o": o.detach().to(dt), "state": st.detach() if with_state else None}
    r.update({name: x.to(dt) for name, x in zip(("dq", "dk", "dv"), gr)})
    r["d_state"] = gr[3] if with_state else None
    return r


def _plain_norm(x, w):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r * w, x, r


def _plain_turn(n, cos, sin, interleaved):
    r = cos.shape[-1]
    if interleaved:
        a, b = n[..., 0:2 * r:2], n[..., 1:2 * r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = n[..., :r], n[..., r:2 * r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, n[..., 2 * r:]], -1)


def _plain_rot_bwd(dy, x, w, turn):
    cos, sin, interleaved = turn
    dn = _plain_turn(dy.float(), cos, -sin, interleaved)
    _, x, r = _plain_norm(x, w)
    xh = x * r
    e = dn * w
    return r * (e - xh * (e * xh).mean(-1, keepdim=True)), (dn * xh).sum((0, 1, 2))


def _plain_lin(q, k, v, log_decay, state, scale, chunk=64):
    """Chunked form: products within a chunk, and the chunks' states as sums over the chunks before them."""
    b, t, hv, dv = v.shape
    share = hv // k.shape[2]
    dk = k.shape[-1]
    pad = -t % chunk
    n = (t + pad) // chunk

    def chunks(x):  # [b, t, h, d] -> [b, h, n, chunk, d]
        return torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).transpose(1, 2).unflatten(2, (n, chunk))

    q, k, v = chunks(q.repeat_interleave(share, 2) * scale), chunks(k.repeat_interleave(share, 2)), chunks(v)
    ld = log_decay.double()[:, None]

    def power(e):  # the decay to the powers e, 0 where e < 0: [h, 1, ...]
        e = e.double()
        return torch.where(e < 0, 0.0, torch.exp(ld.view(-1, *[1] * e.dim()) * e.clamp(min=0))).float().unsqueeze(1)

    i = torch.arange(chunk, device=v.device)
    c = torch.arange(n, device=v.device)
    o = ((q @ k.transpose(-1, -2)) * power(i[:, None] - i)) @ v
    ends = ((k * power(chunk - 1 - i)[..., None]).transpose(-1, -2) @ v).flatten(-2)  # [b, h, n, dk dv]
    before = power((c[:, None] - 1 - c) * chunk)[:, 0] @ ends
    if state is not None:
        before = before + power(c * chunk)[:, 0, :, None] * state.flatten(-2)[:, :, None]
    before = before.unflatten(-1, (dk, dv))
    o = o + power(i + 1)[..., None] * (q @ before)
    # the last chunk's end, after the tokens that are there
    rest = chunk - pad
    e = rest - 1 - i
    last = (k[:, :, -1] * power(e)[:, 0, :, None]).transpose(-1, -2) @ v[:, :, -1]
    st = power(torch.tensor(rest, device=v.device))[..., None] * before[:, :, -1] + last
    return o.flatten(2, 3)[:, :, :t].transpose(1, 2), st


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    b, t = case["batch"], case["t"]
    if case["op"].startswith("qkrot"):
        n = b * t * (case["hq"] + case["hk"]) * case["dim"]
        small = 8 * b * t + 2 * case["rot"] + 8 * case["dim"]  # positions, frequencies, weights
        if case["op"] == "qkrot_fwd":  # q and k in and out
            return {"bytes": 2 * n * e + small, "flops": 8 * n}
        return {"bytes": 3 * n * e + small + 8 * case["dim"], "flops": 16 * n}  # q, k, their outputs' gradients in; dq, dk out
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    qk, vo, st = 2 * b * t * hk * dk * e, 2 * b * t * hv * dv * e, b * hv * dk * dv * 4
    flops = 4 * b * t * hv * dk * dv  # k v^T and S^T q
    if case["op"] != "linattn_train":
        return {"bytes": qk + vo + (2 if case["state"] else 1) * st + 4 * hv, "flops": flops}
    # q, k, v, d_o read once; o, dq, dk, dv written once (and the states' ways in and out)
    return {"bytes": 2 * qk + 2 * vo + (4 * st if case["state"] else 0) + 4 * hv, "flops": 3 * flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"].startswith("qkrot"):
        return _exact_rot(case, f)
    return _exact_lin(case, f)


def _exact_rot(case, f):
    d, r = case["dim"], case["rot"] // 2
    # pairs as complex numbers
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), f["positions"].unsqueeze(-1) * f["inv_freq"]).unsqueeze(2)
    at = torch.arange(r, device="cuda")
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + r)

    def rotated(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "qkrot_fwd":
        return {n: rotated(f[n] * f[n + "_weight"] / ((f[n] ** 2).sum(-1, keepdim=True) / d + EPS).sqrt(), turn) for n in "qk"}
    out = {}
    for n in "qk":
        x, w = f[n], f[n + "_weight"]
        up = rotated(f["d%s_out" % n], turn.conj())
        m = (x ** 2).sum(-1, keepdim=True) / d + EPS
        out["d%s" % n] = up * w / m.sqrt() - x * (up * w * x).sum(-1, keepdim=True) / (d * m ** 1.5)
        out["d_%s_weight" % n] = torch.einsum("bthd,bthd->d", up, x / m.sqrt())
    return out


def _exact_lin(case, f):
    """Token by token: outputs and dq on the way forward, dk and dv on the way back."""
    b, t, hv, dk, dv = (case[k] for k in ("batch", "t", "hv", "dk", "dv"))
    share, scale, train = hv // case["hk"], dk ** -0.5, case["op"] == "linattn_train"
    heads = torch.arange(hv, device="cuda") // share
    # time first, so that a step's values are one slice
    q, k, v = (x.transpose(0, 1).contiguous() for x in (f["q"][:, :, heads] * scale, f["k"][:, :, heads], f["v"]))
    lam = f["log_decay"].exp()[:, None, None]
    m = torch.zeros(b, hv, dk, dv, dtype=torch.float64, device="cuda")
    if case["state"]:
        m = m + f["state"]
    o = torch.empty(t, b, hv, dv, dtype=torch.float64, device="cuda")
    do = f["d_o"].transpose(0, 1).contiguous() if train else None
    dq = torch.empty_like(q)
    for i in range(t):
        m = torch.addcmul(m * lam, k[i].unsqueeze(-1), v[i].unsqueeze(-2))
        o[i] = torch.einsum("bhkv,bhk->bhv", m, q[i])
        if train:
            dq[i] = torch.einsum("bhkv,bhv->bhk", m, do[i])
    out = {"o": o.transpose(0, 1), "state": m if case["state"] or not train else None}
    if not train:
        return out
    dk_, dv_ = torch.empty_like(k), torch.empty_like(v)
    d = torch.zeros_like(m)
    if case["state"]:
        d = d + f["d_state_out"]
    for i in range(t - 1, -1, -1):
        d = torch.addcmul(d, q[i].unsqueeze(-1), do[i].unsqueeze(-2))
        dk_[i] = torch.einsum("bhkv,bhv->bhk", d, v[i])
        dv_[i] = torch.einsum("bhkv,bhk->bhv", d, k[i])
        d = d * lam

    def shared(x):  # sums over the value heads of a key head
        return x.transpose(0, 1).unflatten(2, (case["hk"], share)).sum(3)

    out.update(dq=shared(dq) * scale, dk=shared(dk_), dv=dv_.transpose(0, 1), d_state=d if case["state"] else None)
    return out
