"""Calls with ``stream=``: the results, and whose memory a call takes."""

import pytest
import torch

from delta_util import delta_inputs
from mamba_selective_scan_gb300 import binding
from mamba_selective_scan_gb300.inputs import make_inputs
from parity_util import to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _norm(dt, rows=300, dim=512, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = {"x": r(rows, dim).to(dt), "w": r(dim), "b": r(dim), "dy": r(rows, dim).to(dt), "res": r(rows, dim), "dres": r(rows, dim)}

    def run(**kw):
        y, r, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"], residual=x["res"], **kw)
        return {"y": y, "r": r, **binding.m3scan_norm_bwd(x["dy"], r, x["w"], mean, rstd, d_residual_out=x["dres"], **kw)}
    return run


def _delta(dt, B, T, H, seed=0):
    x = delta_inputs(B, T, H, H, 64, 64, dt, seed=seed, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]

    def run(**kw):
        o, st, ck = binding.m3scan_delta_fwd(*args, state=x["state"], want_ckpt=True, qk_l2norm=True, **kw)
        r = binding.m3scan_delta_bwd(*args, ck, x["d_o"], d_state_out=x["d_state_out"], want_d_state=True, qk_l2norm=True, **kw)
        return {"o": o, "state": st, **r}
    return run


def _decode(dt):
    x = delta_inputs(8, 1, 4, 4, 128, 128, dt, seed=5, device="cuda")

    def run(**kw):
        S = x["state"].clone()
        torch.cuda.synchronize()
        return {"o": binding.m3scan_delta_decode(*[x[n] for n in ("q", "k", "v", "g", "beta")], S, qk_l2norm=True, **kw), "S": S}
    return run


CALLS = {"norm-bf16": lambda: _norm(torch.bfloat16), "norm-f32": lambda: _norm(torch.float32),
         "delta-bf16": lambda: _delta(torch.bfloat16, 2, 200, 2), "delta-segments": lambda: _delta(torch.bfloat16, 1, 1100, 2),
         "delta-shares": lambda: _delta(torch.bfloat16, 8, 130, 20), "delta-f32": lambda: _delta(torch.float32, 2, 90, 2),
         "decode": lambda: _decode(torch.bfloat16)}


@pytest.mark.parametrize("name", list(CALLS))
def test_takes_memory_of_its_stream(name, monkeypatch):
    """Every allocation of a call with stream=s is made with s current, and
    the results are those of a call without it."""
    run = CALLS[name]()
    want = run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    homes = []
    for alloc in ("empty", "empty_like", "zeros", "zeros_like"):
        def spy(*a, _f=getattr(torch, alloc), **kw):
            homes.append(torch.cuda.current_stream().cuda_stream)
            return _f(*a, **kw)
        monkeypatch.setattr(torch, alloc, spy)
    got = run(stream=s)
    monkeypatch.undo()
    s.synchronize()
    assert homes and set(homes) == {s.cuda_stream}
    assert torch.cuda.current_stream().cuda_stream != s.cuda_stream
    for n, w in want.items():
        assert torch.equal(got[n], w), n


def test_two_streams_in_turn():
    """Calls on two streams with nothing between them: each takes scratch that
    the other is not using."""
    runs = [_delta(torch.bfloat16, 4, 512, 8, seed=i) for i in range(2)] + [_delta(torch.bfloat16, 8, 130, 20, seed=i) for i in (2, 3)]
    want = [r() for r in runs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[r(stream=streams[(i + j) % 2]) for i, r in enumerate(runs)] for j in range(2)]
        torch.cuda.synchronize()
        for rows in got:
            for g, w in zip(rows, want):
                for n in w:
                    assert torch.equal(g[n], w[n]), n


def _scan(act, call):
    inp = make_inputs(2, 40, 64, act=act, seed=3)
    d = to_device(inp)
    a = [d[n] for n in ("x", "delta_raw", "z", "B", "C", "conv_w", "conv_b", "dt_bias", "a_log", "D")]
    h = torch.zeros(2, 16, 64, device="cuda")
    c = torch.zeros(2, 3, 64, dtype=d["x"].dtype, device="cuda")

    def run(**kw):
        if call == "decode":
            S, C = h.clone(), c.clone()
            torch.cuda.synchronize()
            gated, _ = binding.m3scan_decode(*a, S, C, **kw)
            return {"gated": gated, "S": S, "C": C}
        if call == "state":
            gated, ck, _, h1, c1 = binding.m3scan_fwd_state(*a, ssm_state=h, conv_state=c, **kw)
            return {"gated": gated, "h": h1, "c": c1,
                    **binding.m3scan_bwd_state(*a, ck, d["d_gated"], conv_state=c, deterministic=True, **kw)}
        gated, ck, _ = binding.m3scan_fwd(*a, **kw)
        bwd = binding.m3scan_bwd_two_phase if call == "two_phase" else binding.m3scan_bwd
        return {"gated": gated, **bwd(*a, ck, d["d_gated"], deterministic=True, **kw)}
    return run


SCANS = {f"scan-{act}-{call}": (act, call) for act in ("f32", "bf16") for call in ("plain", "state", "two_phase", "decode")}


@pytest.mark.parametrize("name", list(SCANS))
def test_scan_takes_memory_of_its_stream(name, monkeypatch):
    monkeypatch.setitem(CALLS, name, lambda: _scan(*SCANS[name]))
    test_takes_memory_of_its_stream(name, monkeypatch)
