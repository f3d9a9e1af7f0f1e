"""Gated delta rule on the GPU against the float64 recurrence and its
autograd gradients.

Tolerances (2-norm of the difference over the 2-norm of the result), from the
arithmetic: an output rounded to bf16 is off by at most 2^-9 per element
(1.95e-3; about 1.7e-3 in the 2-norm), and what happens before the rounding
may add as much again: 4e-3.  f32 outputs come from sums of f32-grade products
over up to a few hundred terms: 2e-5."""

import pytest
import torch

from delta_util import delta_inputs, delta_ref, delta_ref_grads, rel
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 4e-3, torch.float32: 2e-5}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def _run(x, l2norm, scale=0.0):
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, st, ck = binding.m3scan_delta_fwd(*args, state=x["state"], qk_l2norm=l2norm, scale=scale, want_ckpt=True)
    r = binding.m3scan_delta_bwd(*args, ck, x["d_o"], d_state_out=x["d_state_out"],
                                 want_d_state=x["state"] is not None, qk_l2norm=l2norm, scale=scale)
    r.update(o=o, state_out=st)
    return r


CASES = [
    # B, T, Hk, Hv, dk, dv, dtype, state, packed
    (1, 1, 1, 1, 8, 8, "bf16", True, False),
    (2, 3, 1, 2, 16, 24, "bf16", False, False),
    (2, 31, 2, 2, 64, 64, "bf16", True, False),
    (1, 32, 2, 2, 128, 128, "bf16", True, False),
    (1, 33, 1, 3, 128, 128, "bf16", True, True),
    (2, 63, 2, 4, 80, 72, "bf16", True, True),
    (1, 64, 2, 2, 128, 128, "bf16", False, False),
    (2, 65, 2, 2, 128, 128, "bf16", True, False),
    (1, 127, 1, 1, 128, 64, "bf16", True, False),
    (1, 128, 2, 2, 64, 128, "bf16", True, True),
    (3, 129, 1, 2, 96, 128, "bf16", True, False),
    (1, 300, 2, 2, 128, 128, "bf16", True, False),
    (1, 1, 2, 2, 128, 128, "f32", True, False),
    (2, 33, 1, 2, 40, 128, "f32", True, True),
    (1, 130, 2, 2, 128, 128, "f32", True, False),
    (2, 200, 2, 2, 128, 56, "f32", False, False),
]


@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(case, l2norm):
    B, T, Hk, Hv, dk, dv, dt, state, packed = case
    x = delta_inputs(B, T, Hk, Hv, dk, dv, DT[dt], seed=T + dk, device="cuda", state=state, packed=packed)
    if not l2norm:  # unnormalised keys: short enough that beta |k|^2 stays below 2
        for n in ("q", "k"):
            x[n] = (x[n].float() * (0.8 / dk ** 0.5)).to(DT[dt])
    got = _run(x, l2norm)
    ref = delta_ref_grads(x, dk ** -0.5, l2norm)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta"] + (["d_state"] if state else []))


@pytest.mark.parametrize("B,T,Hk,Hv,state", [(8, 200, 10, 20, True), (40, 64, 4, 4, False), (31, 129, 5, 10, True), (51, 1, 3, 3, True)])
def test_more_heads_than_sms(B, T, Hk, Hv, state):
    """Heads in equal shares: some are begun by one block and ended by the
    next, which takes the state (or its adjoint) over."""
    x = delta_inputs(B, T, Hk, Hv, 64, 72, torch.bfloat16, seed=B, device="cuda", state=state)
    got = _run(x, True)
    ref = delta_ref_grads(x, 64 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta"] + (["d_state"] if state else []))


@pytest.mark.parametrize("B,T,H", [(1, 1100, 1), (2, 2000, 2)])
def test_few_heads_in_segments(B, T, H):
    """Few heads over a long sequence: time segments, whose start states come
    from the segments' transitions."""
    x = delta_inputs(B, T, H, H, 128, 128, torch.bfloat16, seed=T, device="cuda")
    got = _run(x, True)
    ref = delta_ref_grads(x, 128 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state"])


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv,state", [(1, 1301, 1, 3, 64, 96, True), (2, 1537, 2, 4, 72, 40, False), (5, 1030, 2, 4, 128, 64, True)])
def test_segments_of_shared_and_narrow_heads(B, T, Hk, Hv, dk, dv, state):
    """Time segments with heads narrower than their tiles, key heads shared by
    value heads, and a last segment that is shorter than the others."""
    x = delta_inputs(B, T, Hk, Hv, dk, dv, torch.bfloat16, seed=T, device="cuda", state=state)
    got = _run(x, True)
    ref = delta_ref_grads(x, dk ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta"] + (["d_state"] if state else []))


@pytest.mark.parametrize("B,T,Hk,Hv", [(9, 470, 8, 16), (3, 700, 50, 50)])
def test_more_chunks_than_blocks(B, T, Hk, Hv):
    """More (chunk, head) pairs than the preparing kernel has blocks: each goes
    through several."""
    x = delta_inputs(B, T, Hk, Hv, 32, 24, torch.bfloat16, seed=B, device="cuda")
    got = _run(x, True)
    ref = delta_ref_grads(x, 32 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state"])


@pytest.mark.parametrize("B,T,H", [(1, 1100, 2), (8, 130, 20), (2, 90, 3)])
def test_in_a_graph(B, T, H):
    """Forward and backward captured and replayed on new values: the bits of
    calls outside it (time segments, shares of heads, plain heads)."""
    names = ("q", "k", "v", "g", "beta")
    x = delta_inputs(B, T, H, H, 64, 64, torch.bfloat16, seed=3, device="cuda")
    y = delta_inputs(B, T, H, H, 64, 64, torch.bfloat16, seed=4, device="cuda")

    def both(x):
        o, st, ck = binding.m3scan_delta_fwd(*[x[n] for n in names], state=x["state"], qk_l2norm=True, want_ckpt=True)
        return o, st, binding.m3scan_delta_bwd(*[x[n] for n in names], ck, x["d_o"], d_state_out=x["d_state_out"], qk_l2norm=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x)
    want = both(y)
    for n in x:
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n, w in want[2].items():
        assert (w is None and got[2][n] is None) or torch.equal(got[2][n], w), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_extreme_gates(dt):
    """-inf and very negative log decays forget the state; beta 0 writes
    nothing; a zero key row is normalised to zero."""
    x = delta_inputs(1, 150, 1, 2, 128, 128, DT[dt], seed=5, device="cuda")
    x["g"][:, 3::17] = float("-inf")
    x["g"][:, 7::31] = -500.0
    x["g"][:, 11::13] = 0.0
    x["beta"][:, 5::7] = 0.0
    x["beta"][:, 6::7] = 1.0
    x["k"][:, 9::19] = 0.0
    got = _run(x, True)
    y = dict(x)
    y["g"] = x["g"].clamp(min=-800.0)  # exp(-800) is 0 in float64
    ref = delta_ref_grads(y, 128 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeated_keys(dt):
    """The same key every token, beta 1, no decay: the inverse's entries do
    not shrink away from the diagonal."""
    x = delta_inputs(1, 100, 1, 1, 64, 64, DT[dt], seed=8, device="cuda")
    x["k"] = x["k"][:, :1].expand(-1, 100, -1, -1).contiguous()
    x["beta"][:] = 1.0
    x["g"][:] = 0.0
    got = _run(x, True)
    ref = delta_ref_grads(x, 64 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dv"])


def test_scale_argument():
    x = delta_inputs(1, 70, 1, 1, 64, 64, torch.bfloat16, seed=2, device="cuda")
    got = _run(x, True, scale=0.37)
    ref = delta_ref_grads(x, 0.37, True)
    _check_all(got, ref, ["o", "dq", "dk", "dv", "d_state"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0, 1, 64, 130])
def test_windows_chain(dt, T):
    """A sequence cut in two windows, the state carried: the same as one."""
    x = delta_inputs(2, T + 67, 1, 2, 64, 128, DT[dt], seed=T, device="cuda")
    names = ("q", "k", "v", "g", "beta")
    whole, st, _ = binding.m3scan_delta_fwd(*[x[n] for n in names], state=x["state"], qk_l2norm=True)
    a, mid, _ = binding.m3scan_delta_fwd(*[x[n][:, :T].contiguous() for n in names], state=x["state"], qk_l2norm=True)
    b, end, _ = binding.m3scan_delta_fwd(*[x[n][:, T:].contiguous() for n in names], state=mid, qk_l2norm=True)
    assert rel(torch.cat([a, b], 1), whole.double().cpu()) <= TOL[DT[dt]]
    assert rel(end, st.double().cpu()) <= 2e-5


@pytest.mark.parametrize("B,Hk,Hv,dk,dv,dt", [(1, 1, 1, 8, 8, "bf16"), (1, 2, 4, 128, 128, "bf16"), (40, 4, 16, 64, 96, "bf16"),
                                             (3, 2, 2, 128, 128, "f32"), (16, 5, 40, 128, 128, "bf16")])
def test_decode_continues_prefill(B, Hk, Hv, dk, dv, dt):
    """Single tokens from a carried state, updated in place."""
    x = delta_inputs(B, 5, Hk, Hv, dk, dv, DT[dt], seed=B, device="cuda")
    ref = delta_ref_grads(x, dk ** -0.5, True)
    S = x["state"].clone()
    outs = []
    for t in range(5):
        outs.append(binding.m3scan_delta_decode(*[x[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "g", "beta")], S,
                                                qk_l2norm=True))
    assert rel(torch.cat(outs, 1), ref["o"]) <= TOL[DT[dt]]
    assert rel(S, ref["state_out"]) <= 2e-5


def test_same_bits_every_call():
    x = delta_inputs(2, 333, 2, 4, 128, 128, torch.bfloat16, seed=1, device="cuda")
    a, b = _run(x, True), _run(x, True)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_on_another_stream():
    x = delta_inputs(1, 200, 1, 2, 128, 128, torch.bfloat16, seed=4, device="cuda")
    want = _run(x, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _run(x, True)
    s.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_gradient_views_of_one_buffer():
    """dq, dk and dv written into columns of one projection's gradient leave
    its other columns alone."""
    B, T, Hk, Hv, dk, dv = 2, 70, 2, 4, 64, 64
    x = delta_inputs(B, T, Hk, Hv, dk, dv, torch.bfloat16, seed=6, device="cuda", packed=True)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    _, _, ck = binding.m3scan_delta_fwd(*args, state=x["state"], qk_l2norm=True, want_ckpt=True)
    plain = binding.m3scan_delta_bwd(*args, ck, x["d_o"], qk_l2norm=True)
    row = torch.full((B, T, 2 * Hk * dk + Hv * dv + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k, v, rest = row.split([Hk * dk, Hk * dk, Hv * dv, 16], -1)
    out = {"dq": q.unflatten(2, (Hk, dk)), "dk": k.unflatten(2, (Hk, dk)), "dv": v.unflatten(2, (Hv, dv))}
    binding.m3scan_delta_bwd(*args, ck, x["d_o"], qk_l2norm=True, out=out)
    for n in out:
        assert torch.equal(out[n], plain[n]), n
    assert (rest == 7.0).all()


def test_gradients_against_differences():
    """Central differences of the f32 forward along random directions."""
    x = delta_inputs(1, 70, 1, 2, 32, 32, torch.float32, seed=9, device="cuda")
    got = _run(x, True)

    def loss(y):
        o, st, _ = binding.m3scan_delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], state=y["state"], qk_l2norm=True)
        return ((o.double() * x["d_o"].double()).sum() + (st.double() * x["d_state_out"].double()).sum()).item()

    gen = torch.Generator(device="cuda").manual_seed(0)
    for n in ("q", "k", "v", "g", "beta", "state"):
        d = torch.randn(x[n].shape, generator=gen, device="cuda")
        d *= x[n].norm() / d.norm()
        eps = 1e-3
        num = (loss({**x, n: x[n] + eps * d}) - loss({**x, n: x[n] - eps * d})) / (2 * eps)
        ana = (got["d_" + n if n == "state" else "d" + n].double() * d.double()).sum().item()
        size = (got["d_" + n if n == "state" else "d" + n].double().norm() * d.double().norm()).item() / d.numel() ** 0.5
        # truncation ~ eps^2, and the f32 forward's rounding (1e-6 of the loss's terms) over eps
        assert abs(num - ana) <= 2e-2 * max(abs(ana), size), n


def test_nan_stays_in_its_row():
    """A NaN in one head's values reaches that head's outputs only."""
    x = delta_inputs(1, 80, 2, 2, 64, 64, torch.bfloat16, seed=3, device="cuda")
    clean = _run(x, True)
    x["v"][0, 40, 1, 3] = float("nan")
    got = _run(x, True)
    assert torch.equal(got["o"][:, :, 0], clean["o"][:, :, 0])
    assert torch.equal(got["o"][:, :40], clean["o"][:, :40])
    assert torch.isnan(got["o"][0, 40, 1, 3])
    assert torch.equal(got["dv"][:, :, 0], clean["dv"][:, :, 0])


def test_segments_of_changing_decays():
    """Long time segments whose chunks decay differently from the ones two
    before and two behind them (the stage their factors share): the chunks'
    own decays count in every call."""
    x = delta_inputs(1, 6000, 2, 2, 128, 64, torch.bfloat16, seed=12, device="cuda")
    chunk = torch.arange(6000, device="cuda") // 64
    x["g"] *= 0.02
    x["g"][:, chunk % 4 >= 2] = -0.25
    names = ("q", "k", "v", "g", "beta")
    got = _run(x, True)
    _check_all(got, delta_ref_grads(x, 128 ** -0.5, True), ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state"])
    for _ in range(30):
        o, st, _ = binding.m3scan_delta_fwd(*[x[n] for n in names], state=x["state"], qk_l2norm=True)
        assert torch.equal(o, got["o"]) and torch.equal(st, got["state_out"])


NOT_FINITE = [(n, v) for n in ("g", "beta", "k", "q", "v") for v in ("nan", "inf")]


def _spoil(x, name, value, at):
    """x with one value of key head 0 or value head 1 of the last sequence not finite from token `at`."""
    y = dict(x)
    y[name] = x[name].clone()
    i = {"g": (-1, at, 1), "beta": (-1, at, 1), "v": (-1, at, 1, 5)}.get(name, (-1, at, 0, 3))
    y[name][i] = float(value)
    return y


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hk,Hv,at", [(1, 100, 1, 2, 40), (1, 1100, 1, 2, 601), (8, 130, 10, 20, 70)])
def test_nan_gate_is_not_a_reset(B, T, Hk, Hv, at, dt):
    """exp(NaN) is NaN: the outputs from that token on and the state (in f32
    also the gradients that depend on it), none of which may come out finite."""
    if dt == "f32" and T > 1000:
        pytest.skip("no segments in f32")
    x = delta_inputs(B, T, Hk, Hv, 64, 64, DT[dt], seed=at, device="cuda")
    y = _spoil(x, "g", "nan", at)
    got = _run(y, True)
    ref = delta_ref_grads(y, 64 ** -0.5, True)
    for n in ("o", "state_out") + (("dq", "dk", "dv", "dg", "dbeta", "d_state") if dt == "f32" else ()):
        assert not (torch.isfinite(got[n]).cpu() & ~torch.isfinite(ref[n])).any(), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name,value", NOT_FINITE)
def test_not_finite_in_decode(name, value, dt):
    x = delta_inputs(3, 4, 2, 4, 64, 72, DT[dt], seed=2, device="cuda")
    y = _spoil(x, name, value, 1)
    names = ("q", "k", "v", "g", "beta")
    ref, rst = delta_ref(*[y[n].double().cpu() for n in names], y["state"].double().cpu(), 64 ** -0.5, True)
    for step in (1, 4):
        S = y["state"].clone()
        o = torch.cat([binding.m3scan_delta_decode(*[y[n][:, t:t + step].contiguous() for n in names], S, qk_l2norm=True)
                       for t in range(0, 4, step)], 1)
        assert torch.equal(torch.isfinite(o), torch.isfinite(ref).cuda())
        assert torch.equal(torch.isfinite(S), torch.isfinite(rst).cuda())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["g", "q", "v"])
@pytest.mark.parametrize("B,T,Hk,Hv,at", [(1, 150, 2, 4, 40), (1, 1100, 2, 4, 601), (8, 130, 10, 20, 70)])
def test_not_finite_in_gradients(B, T, Hk, Hv, at, name, dt):
    """No gradient is finite that the definition's is not, those that are
    finite are right, and other key heads' are the same bits."""
    if dt == "f32" and B * T > 500:
        pytest.skip("no segments or shares in f32")
    x = delta_inputs(B, T, Hk, Hv, 64, 64, DT[dt], seed=at, device="cuda")
    y = _spoil(x, name, "nan", at)
    clean, got, ref = _run(x, True), _run(y, True), delta_ref_grads(y, 64 ** -0.5, True)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_state"):
        g, r = got[n].double().cpu(), ref[n]
        ok = torch.isfinite(g)
        assert not (ok & ~torch.isfinite(r)).any(), n
        d = (g[ok] - r[ok]).norm()
        assert d <= TOL[got[n].dtype] * r[ok].norm(), n
        h = g.shape[1 if n == "d_state" else 2] // Hk  # (key head 0's own)
        rest = (slice(None), slice(h, None)) if n == "d_state" else (slice(None), slice(None), slice(h, None))
        assert torch.equal(got[n][rest], clean[n][rest]), n


@pytest.mark.parametrize("B,T,Hk,Hv,at", [(1, 150, 2, 4, 40), (2, 130, 1, 3, 64), (1, 70, 1, 2, 0), (1, 90, 1, 2, 89)])
@pytest.mark.parametrize("name,value", NOT_FINITE)
@pytest.mark.parametrize("dt,l2norm", [("bf16", True), ("bf16", False), ("f32", True)])
def test_not_finite_from_its_token_on(dt, l2norm, name, value, B, T, Hk, Hv, at):
    """A value that is not finite reaches what the recurrence lets it reach:
    nothing of earlier tokens or other heads, and all that depends on it."""
    x = delta_inputs(B, T, Hk, Hv, 64, 72, DT[dt], seed=at, device="cuda")
    if not l2norm:
        for n in ("q", "k"):
            x[n] = (x[n].float() * 0.1).to(DT[dt])
    y = _spoil(x, name, value, at)
    names = ("q", "k", "v", "g", "beta")
    clean = binding.m3scan_delta_fwd(*[x[n] for n in names], state=x["state"], qk_l2norm=l2norm)
    got = binding.m3scan_delta_fwd(*[y[n] for n in names], state=y["state"], qk_l2norm=l2norm)
    ref = delta_ref(*[y[n].double().cpu() for n in names], y["state"].double().cpu(), 64 ** -0.5, l2norm)
    for g, c, r in zip(got, clean, ref):
        ok = torch.isfinite(r).cuda()
        assert torch.equal(torch.isfinite(g), ok)
        if name == "q" or g is got[0]:
            assert torch.equal(g[ok], c[ok])


@pytest.mark.parametrize("B,T,Hk,Hv,at", [(1, 1100, 1, 2, 601), (8, 130, 10, 20, 70)])
@pytest.mark.parametrize("name", ["g", "beta", "k", "v"])
def test_not_finite_in_segments_and_shares(name, B, T, Hk, Hv, at):
    x = delta_inputs(B, T, Hk, Hv, 64, 64, torch.bfloat16, seed=at, device="cuda")
    y = _spoil(x, name, "nan", at)
    names = ("q", "k", "v", "g", "beta")
    clean, _, _ = binding.m3scan_delta_fwd(*[x[n] for n in names], state=x["state"], qk_l2norm=True)
    got, st, _ = binding.m3scan_delta_fwd(*[y[n] for n in names], state=y["state"], qk_l2norm=True)
    ref, rst = delta_ref(*[y[n].double().cpu() for n in names], y["state"].double().cpu(), 64 ** -0.5, True)
    ok = torch.isfinite(ref).cuda()
    assert torch.equal(torch.isfinite(got), ok) and torch.equal(got[ok], clean[ok])
    assert torch.equal(torch.isfinite(st), torch.isfinite(rst).cuda())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["beta", "k"])
@pytest.mark.parametrize("B,T,Hk,Hv,at", [(1, 150, 2, 4, 40), (1, 1100, 2, 4, 601), (8, 130, 10, 20, 70)])
def test_gradients_of_keys_and_beta_not_finite(B, T, Hk, Hv, at, name, dt):
    test_not_finite_in_gradients(B, T, Hk, Hv, at, name, dt)

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("low", [float("-inf"), -60.0])
@pytest.mark.parametrize("every", [2, 3, 5, 8])
def test_decays_between_resets(every, low, dt):
    """Many forgetting tokens in a chunk (short sequences packed into one): the
    small decays between them keep their precision, which shows in the f32
    results (the state; every gradient of f32 activations)."""
    x = delta_inputs(1, 192, 1, 2, 64, 64, DT[dt], seed=every, device="cuda")
    x["g"] = -0.5 * torch.rand(1, 192, 2, generator=torch.Generator().manual_seed(every)).to(DT[dt]).cuda()
    x["g"][:, ::every] = low
    got = _run(x, True)
    y = dict(x)
    y["g"] = x["g"].clamp(min=-800.0)  # exp(-800) is 0 in float64
    ref = delta_ref_grads(y, 64 ** -0.5, True)
    _check_all(got, ref, ["o", "state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state"])


@pytest.mark.parametrize("B,T,Hk,Hv,dt", [(1, 1100, 1, 2, "bf16"), (2, 2000, 2, 2, "bf16"), (8, 130, 10, 20, "bf16"),
                                          (2, 100, 1, 2, "bf16"), (2, 70, 1, 2, "f32"), (2, 0, 1, 2, "bf16")])
def test_state_in_place(B, T, Hk, Hv, dt):
    """The state carried in place, and its gradient: the bits of calls with
    separate ones (with time segments, whose last may end before the first
    one's block starts, too)."""
    x = delta_inputs(B, T, Hk, Hv, 128, 64, DT[dt], seed=T, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want = _run(x, True)
    for _ in range(5):
        S, dS = x["state"].clone(), x["d_state_out"].clone()
        o, st, ck = binding.m3scan_delta_fwd(*args, state=S, state_out=S, qk_l2norm=True, want_ckpt=True)
        r = binding.m3scan_delta_bwd(*args, ck, x["d_o"], d_state_out=dS, out={"d_state": dS}, qk_l2norm=True)
        assert st is S and r["d_state"] is dS
        assert torch.equal(o, want["o"]) and torch.equal(S, want["state_out"]) and torch.equal(dS, want["d_state"])
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(r[n], want[n]), n
