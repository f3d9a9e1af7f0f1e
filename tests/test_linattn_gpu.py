"""Linear attention with a decay per head on the GPU against the float64
recurrence and its autograd gradients.

Tolerances (2-norm of the difference over the 2-norm of the result), from the
arithmetic: an output rounded to bf16 is off by at most 2^-8 of its value
(3.9e-3, about 1.7e-3 in the 2-norm over many), and two of its operands may be
rounded to bf16 on the way, each about 1.7e-3 in the 2-norm: 6e-3 covers the
first at its worst and the others as they add up.  f32 results are f32 sums of
products of at least 17 bits (2^-18 each, 4e-6): 2e-5."""

import pytest
import torch

from lin_util import lin_inputs, lin_ref, lin_ref_grads, rel
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 6e-3, torch.float32: 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ["o", "state_out", "dq", "dk", "dv"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _check_all(got, ref, names):
    bad = {}
    for n in names:
        e = rel(got[n], ref[n])
        if not e <= TOL[got[n].dtype]:
            bad[n] = e
    assert not bad, bad


def _run(x, scale=0.0, **kw):
    args = [x[n] for n in ("q", "k", "v", "log_decay")]
    o, st = binding.m3scan_linattn_fwd(*args, state=x["state"], scale=scale, **kw)
    r = binding.m3scan_linattn_bwd(*args, x["d_o"], state=x["state"], d_state_out=x["d_state_out"],
                                   want_d_state=x["state"] is not None, scale=scale, **kw)
    r.update(o=o, state_out=st)
    return r


CASES = [
    # B, T, Hk, Hv, dk, dv, dtype, state, packed
    (1, 1, 1, 1, 8, 8, "bf16", True, False),
    (2, 1, 2, 4, 128, 128, "bf16", True, True),
    (2, 2, 1, 2, 16, 24, "bf16", False, False),
    (2, 31, 2, 2, 64, 64, "bf16", True, False),
    (1, 33, 1, 3, 128, 128, "bf16", True, True),
    (2, 63, 2, 4, 80, 72, "bf16", True, True),
    (1, 64, 2, 2, 128, 128, "bf16", False, False),
    (2, 65, 2, 2, 128, 128, "bf16", True, False),
    (1, 127, 1, 1, 128, 64, "bf16", True, False),
    (1, 128, 2, 2, 64, 128, "bf16", True, True),
    (3, 129, 1, 2, 96, 128, "bf16", True, False),
    (1, 300, 2, 2, 128, 128, "bf16", True, False),
    (1, 1, 2, 2, 128, 128, "f32", True, False),
    (2, 15, 1, 2, 8, 16, "f32", True, False),
    (2, 33, 1, 2, 40, 128, "f32", True, True),
    (1, 130, 2, 2, 128, 128, "f32", True, False),
    (2, 200, 2, 2, 128, 56, "f32", False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(case):
    B, T, Hk, Hv, dk, dv, dt, state, packed = case
    x = lin_inputs(B, T, Hk, Hv, dk, dv, DT[dt], seed=T + dk, device="cuda", state=state, packed=packed)
    _check_all(_run(x), lin_ref_grads(x, dk ** -0.5), NAMES + (["d_state"] if state else []))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 64, 200])
def test_decays_of_every_kind(dt, T):
    """No decay at all, decays that keep nothing, that pass f32's smallest
    value within a few tokens, and a head that grows."""
    ld = [0.0, float("-inf"), -1e-6, -0.7, -40.0, -103.0, -1e4, 0.01]
    x = lin_inputs(1, T, 4, 8, 64, 128, DT[dt], seed=T, device="cuda", log_decay=ld)
    _check_all(_run(x), lin_ref_grads(x, 64 ** -0.5), NAMES + ["d_state"])


@pytest.mark.parametrize("scale", [0.25, -1.5])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scale(dt, scale):
    x = lin_inputs(2, 70, 1, 2, 32, 64, DT[dt], seed=3, device="cuda")
    _check_all(_run(x, scale=scale), lin_ref_grads(x, scale), NAMES + ["d_state"])


@pytest.mark.parametrize("B,T,Hk,Hv,state", [(8, 200, 10, 20, True), (40, 64, 4, 4, False), (31, 129, 5, 10, True), (51, 2, 3, 3, True)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_heads_than_sms(dt, B, T, Hk, Hv, state):
    x = lin_inputs(B, T, Hk, Hv, 64, 72, DT[dt], seed=B, device="cuda", state=state)
    _check_all(_run(x), lin_ref_grads(x, 64 ** -0.5), NAMES + (["d_state"] if state else []))


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv,dt,state", [
    (1, 1100, 1, 1, 128, 128, "bf16", True), (2, 2000, 2, 2, 128, 128, "bf16", True), (1, 1301, 1, 3, 64, 96, "bf16", True),
    (2, 1537, 2, 4, 72, 40, "bf16", False), (5, 1030, 2, 4, 128, 64, "bf16", True), (1, 1999, 1, 2, 128, 128, "f32", True), (2, 1301, 1, 3, 40, 72, "f32", False)])
def test_few_heads_over_long_sequences(B, T, Hk, Hv, dk, dv, dt, state):
    x = lin_inputs(B, T, Hk, Hv, dk, dv, DT[dt], seed=T, device="cuda", state=state)
    _check_all(_run(x), lin_ref_grads(x, dk ** -0.5), NAMES + (["d_state"] if state else []))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slow_decays_over_many_chunks(dt):
    """A state that hardly fades over hundreds of chunks: the decay of a chunk
    must not be rounded in a way that adds up."""
    x = lin_inputs(1, 16384, 2, 2, 64, 64, DT[dt], seed=5, device="cuda", state=True, log_decay=[-3e-7, -2e-5])
    o, st = binding.m3scan_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"])
    i = torch.arange(16384, device="cuda", dtype=torch.float64)
    w = torch.exp(x["log_decay"].double() * (16383 - i)[:, None])[None, :, :, None]
    ref = torch.einsum("bthk,bthv->bhkv", x["k"].double() * w, x["v"].double())
    ref += torch.exp(16384 * x["log_decay"].double())[:, None, None] * x["state"].double()
    assert rel(st, ref.cpu()) <= TOL[torch.float32]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", [(1, 2, 2, 128, 128), (3, 2, 4, 64, 96), (20, 10, 20, 128, 72), (2, 1, 1, 8, 8)])
def test_decode(B, Hk, Hv, dk, dv, T, dt):
    x = lin_inputs(B, T, Hk, Hv, dk, dv, DT[dt], seed=B + T, device="cuda", packed=True)
    state = x["state"].clone()
    o = binding.m3scan_linattn_decode(x["q"], x["k"], x["v"], x["log_decay"], state)
    ref = lin_ref_grads(x, dk ** -0.5)
    _check_all({"o": o, "state_out": state}, ref, ["o", "state_out"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_windows_chain(dt):
    """A sequence in windows of odd lengths, the state carried in place, and
    its last tokens one by one: as the sequence at once."""
    x = lin_inputs(2, 200, 2, 4, 64, 128, DT[dt], seed=9, device="cuda")
    ref = lin_ref_grads(x, 64 ** -0.5)
    state, outs = x["state"].clone(), []
    for lo, hi in ((0, 77), (77, 78), (78, 197)):
        o, st = binding.m3scan_linattn_fwd(*(x[n][:, lo:hi].contiguous() for n in "qkv"), x["log_decay"], state=state, state_out=state)
        assert st is state
        outs.append(o)
    for i in range(197, 200):
        outs.append(binding.m3scan_linattn_decode(*(x[n][:, i:i + 1].contiguous() for n in "qkv"), x["log_decay"], state))
    _check_all({"o": torch.cat(outs, 1), "state_out": state}, ref, ["o", "state_out"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [150, 1200])
def test_backward_windows_chain(dt, T):
    """Gradients of two windows, the second's d_state being the first's
    d_state_out and overwritten in place."""
    x = lin_inputs(1, T, 1, 2, 64, 64, DT[dt], seed=11, device="cuda")
    ref = lin_ref_grads(x, 64 ** -0.5)
    half = 97
    a, b = ({n: x[n][:, s].contiguous() for n in ("q", "k", "v", "d_o")} for s in (slice(0, half), slice(half, None)))
    _, mid = binding.m3scan_linattn_fwd(a["q"], a["k"], a["v"], x["log_decay"], state=x["state"])
    ds = x["d_state_out"].clone()
    gb = binding.m3scan_linattn_bwd(b["q"], b["k"], b["v"], x["log_decay"], b["d_o"], state=mid, d_state_out=ds, out={"d_state": ds})
    assert gb["d_state"] is ds
    ga = binding.m3scan_linattn_bwd(a["q"], a["k"], a["v"], x["log_decay"], a["d_o"], state=x["state"], d_state_out=ds, out={"d_state": ds})
    got = {n: torch.cat([ga[n], gb[n]], 1) for n in ("dq", "dk", "dv")}
    _check_all({**got, "d_state": ds}, ref, ["dq", "dk", "dv", "d_state"])


BAD = [("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("k", float("-inf")), ("q", float("nan")), ("d_o", float("inf"))]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,t", [(150, 70), (150, 63), (150, 64), (40, 0), (40, 39), (1300, 700)])
@pytest.mark.parametrize("name,value", BAD)
def test_not_finite_stays_where_it_belongs(dt, T, t, name, value):
    """A value that is not finite reaches what the recurrence says, and nothing
    else: not the tokens it comes after, other heads or other columns."""
    x = lin_inputs(1, T, 2, 2, 64, 72, DT[dt], seed=T + t, device="cuda")
    x[name][0, t, 1, 5] = value
    got, ref = _run(x), lin_ref_grads(x, 64 ** -0.5)
    for n in NAMES + ["d_state"]:
        assert torch.equal(torch.isfinite(got[n]).cpu(), torch.isfinite(ref[n])), n
        fine = torch.isfinite(ref[n])
        e = (got[n].double().cpu() - ref[n])[fine].norm() / ref[n][fine].norm().clamp(min=1e-30)
        assert e <= TOL[got[n].dtype], (n, e)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_not_finite_state_and_decay(dt):
    x = lin_inputs(1, 90, 2, 2, 64, 64, DT[dt], seed=2, device="cuda")
    x["state"][0, 1, 3, 7] = float("inf")
    got, ref = _run(x), lin_ref_grads(x, 64 ** -0.5)
    for n in ("o", "state_out", "dq"):
        assert torch.equal(torch.isfinite(got[n]).cpu(), torch.isfinite(ref[n])), n
    x = lin_inputs(1, 90, 2, 2, 64, 64, DT[dt], seed=2, device="cuda", log_decay=[-0.1, float("nan")])
    got, ref = _run(x), lin_ref_grads(x, 64 ** -0.5)
    for n in ("o", "state_out"):  # (head 0 is untouched)
        assert torch.isfinite(got[n][:, :, 0] if n == "o" else got[n][:, 0]).all()
        assert torch.isnan(got[n][:, :, 1] if n == "o" else got[n][:, 1]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,Hv", [(2, 150, 2, 4), (1, 1500, 1, 1), (20, 130, 8, 8)])
def test_same_bits_on_every_call(dt, B, T, Hk, Hv):
    x = lin_inputs(B, T, Hk, Hv, 64, 64, DT[dt], seed=1, device="cuda")
    a, b = _run(x), _run(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_outputs_in_columns_of_one_gradient(dt):
    """dq, dk and dv as columns of the projection's gradient; what lies between
    them stays."""
    x = lin_inputs(2, 100, 2, 4, 64, 32, DT[dt], seed=4, device="cuda", packed=True)
    ref = lin_ref_grads(x, 64 ** -0.5)
    w = [128, 128, 128, 16]
    row = torch.full((2, 100, sum(w)), 7.0, dtype=DT[dt], device="cuda")
    p = row.split(w, -1)
    out = {"dq": p[0].unflatten(2, (2, 64)), "dk": p[1].unflatten(2, (2, 64)), "dv": p[2].unflatten(2, (4, 32))}
    r = binding.m3scan_linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["d_o"], state=x["state"], d_state_out=x["d_state_out"], out=out)
    _check_all(r, ref, ["dq", "dk", "dv"])
    assert (p[3] == 7.0).all()


@pytest.mark.parametrize("B,T", [(0, 5), (2, 0)])
def test_no_tokens(B, T):
    """Without tokens a state and its gradient pass through."""
    x = lin_inputs(B, T, 1, 2, 64, 64, torch.bfloat16, device="cuda")
    o, st = binding.m3scan_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"])
    assert o.shape == x["v"].shape and torch.equal(st, x["state"])
    _, st = binding.m3scan_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"])
    assert (st == 0).all()
    r = binding.m3scan_linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["d_o"], state=x["state"], d_state_out=x["d_state_out"], want_d_state=True)
    assert torch.equal(r["d_state"], x["d_state_out"])
    before = x["state"].clone()
    binding.m3scan_linattn_decode(x["q"], x["k"], x["v"], x["log_decay"], x["state"])
    assert torch.equal(before, x["state"])


@pytest.mark.parametrize("B,T,H", [(2, 100, 4), (1, 1500, 2), (40, 130, 4)])
def test_captured_and_replayed(B, T, H):
    """A forward and a backward in one graph, replayed on other inputs, beside
    a second graph that shares their workspace."""
    x, y = (lin_inputs(B, T, H, H, 64, 64, torch.bfloat16, seed=s, device="cuda") for s in (1, 2))
    dims = binding.M3LinattnDims(B, T, H, H, 64, 64, 0, 0, 0, 0, 0, 0, 0.0, 0)
    ws = binding.Workspace(binding.m3scan_linattn_plan(dims, binding.M3_BF16).workspace_bytes, "cuda")
    want = [_run(v) for v in (x, y)]
    _run(x, workspace=ws)
    held = {n: t.clone() for n, t in x.items()}
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = _run(held, workspace=ws)
        graphs.append((g, r))
    for v, w in ((x, want[0]), (y, want[1]), (x, want[0])):
        for n in held:
            held[n].copy_(v[n])
        for g, r in graphs:
            g.replay()
            torch.cuda.synchronize()
            for n in w:
                assert torch.equal(r[n], w[n]), n
    assert binding.m3scan_get_status(ws) == 0


def test_on_another_stream():
    x = lin_inputs(2, 300, 2, 2, 128, 128, torch.bfloat16, seed=8, device="cuda")
    want = _run(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(x, stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", [(40, 200, 4), (1, 1500, 2)])
def test_two_calls_at_once(dt, B, T, H):
    xs = [lin_inputs(B, T, H, H, 64, 64, DT[dt], seed=s, device="cuda") for s in (3, 4)]
    want = [_run(x) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[_run(x, stream=s) for x, s in zip(xs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            for n in w:
                assert torch.equal(g[n], w[n]), n
    assert binding.m3scan_device_status() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,Hv", [(40, 200, 2, 4), (1, 1500, 1, 2), (2, 100, 2, 2)])
def test_workspace_holds_anything(dt, B, T, Hk, Hv):
    """What a workspace held past its status block changes nothing."""
    x = lin_inputs(B, T, Hk, Hv, 64, 72, DT[dt], seed=5, device="cuda")
    want = _run(x)
    dims = binding.M3LinattnDims(B, T, Hk, Hv, 64, 72, 0, 0, 0, 0, 0, 0, 0.0, 0)
    ws = binding.Workspace(binding.m3scan_linattn_plan(dims, binding.M3_BF16 if dt == "bf16" else binding.M3_F32).workspace_bytes, "cuda")
    ws.buf[binding.STATUS_BYTES:] = 255
    got = _run(x, workspace=ws)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert binding.m3scan_get_status(ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_captured(dt):
    """A captured token, replayed: the state moves on with every replay."""
    x = lin_inputs(3, 1, 2, 4, 64, 64, DT[dt], seed=9, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "log_decay")]
    state, want = x["state"].clone(), x["state"].clone()
    binding.m3scan_linattn_decode(*args, x["state"].clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = binding.m3scan_linattn_decode(*args, state)
    for _ in range(3):
        g.replay()
        ref = binding.m3scan_linattn_decode(*args, want)
        torch.cuda.synchronize()
        assert torch.equal(o, ref) and torch.equal(state, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_past_32_bits(dt):
    """Tokens a megabyte or more apart: the last ones lie past 2^31 elements."""
    T, stride = 2100, 1 << 20
    row = torch.empty(1, T, stride, dtype=DT[dt], device="cuda")
    x = lin_inputs(1, T, 1, 1, 64, 64, DT[dt], seed=6, device="cuda")
    far = {}
    for i, n in enumerate("qkv"):
        far[n] = row[..., 64 * i:64 * i + 64].unflatten(2, (1, 64))
        far[n].copy_(x[n])
    args, fargs = ([d[n] for n in "qkv"] + [x["log_decay"]] for d in (x, far))
    o, st = binding.m3scan_linattn_fwd(*args)
    fo, fst = binding.m3scan_linattn_fwd(*fargs)
    assert torch.equal(o, fo) and torch.equal(st, fst)
    g = binding.m3scan_linattn_bwd(*args, x["d_o"])
    out = {"d" + n: row[..., 256 + 64 * i:320 + 64 * i].unflatten(2, (1, 64)) for i, n in enumerate("qkv")}
    fg = binding.m3scan_linattn_bwd(*fargs, x["d_o"], out=out)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(g[n], fg[n]), n


def test_gradients_against_differences():
    """The loss along a direction, by the calls alone (f32)."""
    x = lin_inputs(1, 60, 1, 2, 16, 24, torch.float32, seed=7, device="cuda")

    def loss(q, k, v, s):
        o, st = binding.m3scan_linattn_fwd(q, k, v, x["log_decay"], state=s)
        return ((o.double() * x["d_o"]).sum() + (st.double() * x["d_state_out"]).sum()).item()

    r = _run(x)
    gen = torch.Generator().manual_seed(3)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("state", "d_state")):
        u = torch.randn(x[n].shape, generator=gen).cuda()
        vals = {m: x[m] for m in ("q", "k", "v", "state")}
        h = 0.5  # the loss is linear in each of them alone: a step of any size gives the derivative
        up = loss(*({**vals, n: x[n] + h * u}.values()))
        down = loss(*({**vals, n: x[n] - h * u}.values()))
        want = (r[d].double() * u).sum().item()
        size = (r[d].double().norm() * u.double().norm()).item()
        assert abs((up - down) / (2 * h) - want) <= 1e-5 * size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,ld", [(2, 2, 40.0), (2, 7, 2.0), (2, 7, 11.0), (1, 33, 2.4), (2, 45, 1.7), (60, 7, 9.0)])
def test_growing_heads_of_short_sequences(dt, B, T, ld):
    """A head that grows, beside one that fades: everything is finite where the
    growth over the sequence is, whatever it would be over a whole chunk.
    (exp of up to 80 rounds its argument: 2^-18 of the value, within the
    tolerances.)"""
    x = lin_inputs(B, T, 2, 4, 64, 72, DT[dt], seed=T, device="cuda", log_decay=[ld, -0.1])
    _check_all(_run(x), lin_ref_grads(x, 64 ** -0.5), NAMES + ["d_state"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_growing_heads_behind_the_last_whole_chunk(dt):
    """100 tokens that grow past f32's range: the first 36 in time and the last
    36 backwards in time do not know of it."""
    x = lin_inputs(1, 100, 1, 2, 64, 64, DT[dt], seed=1, device="cuda", log_decay=[1.5, -0.1])
    got, ref = _run(x), lin_ref_grads(x, 64 ** -0.5)
    part = {"o": slice(0, 36), "dq": slice(0, 36), "dk": slice(64, 100), "dv": slice(64, 100)}
    _check_all({n: got[n][:, s, :1] for n, s in part.items()}, {n: ref[n][:, s, :1] for n, s in part.items()}, list(part))
