"""Linear attention with a decay per head where heads are long runs of chunks:
more heads than SMs, which take equal shares of all chunks and hand states on,
and heads in one segment; and the errors that the kernels are documented to have.

Tolerances (2-norm of the difference over the 2-norm of the result).  A bf16
result is rounded once, 1.66e-3 for values spread over their binades.  The
state that a chunk starts from and the weights between its tokens enter as one
bf16 term each: each puts an error of that size on its part of the result, both
together one of 1.66e-3, so that the result is 1.66e-3 sqrt(2) = 2.35e-3 off; a
tenth more covers the spread over inputs: 2.6e-3.  Up to 512 tokens the weights
are two terms, and what is left is the state's part, a third of the squares at
most in sequences of 64 and 77 tokens: 1.66e-3 sqrt(4 / 3) = 1.92e-3, bound
2.05e-3.

States are f32 sums of products with f32's own error: a rounding of up to 2^-24
per chunk (as independent errors 3.4e-8 sqrt(chunks): 5.5e-7 for 256), and
2^-24 to 2^-23 for the products and their sums: 1.5e-6, over 16384 tokens 2e-6.
f32 sequences round their state once in 16 tokens, 1.1e-6 over 16384 tokens, and
the sums of their products are off by about as much again: 4e-6."""

import pytest
import torch

from lin_util import lin_inputs, lin_ref_chunked, lin_ref_grads, rel
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ["o", "state_out", "dq", "dk", "dv", "d_state"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _run(x):
    args = [x[n] for n in ("q", "k", "v", "log_decay")]
    o, st = binding.m3scan_linattn_fwd(*args, state=x["state"])
    r = binding.m3scan_linattn_bwd(*args, x["d_o"], state=x["state"], d_state_out=x["d_state_out"], want_d_state=True)
    return {"o": o, "state_out": st, **r}


def _rows(x, rows):
    """Those batch rows of a call's inputs or results."""
    return {n: t if n == "log_decay" else t[rows] for n, t in x.items()}


def _check(got, ref, tol):
    bad = {n: e for n in NAMES if not (e := rel(got[n], ref[n])) <= tol[got[n].dtype]}
    assert not bad, bad


def _plan(B, T, Hk, Hv, dk, dv, dt):
    d = binding.M3LinattnDims(B, T, Hk, Hv, dk, dv, *[0] * 6, 0.0, 0)
    return binding.m3scan_linattn_plan(d, binding.M3_F32 if dt == "f32" else binding.M3_BF16)


SHARES = [
    # B, T, Hk, Hv, dk, dv: equal shares in both directions, but 80 heads in the backward alone
    (20, 709, 4, 8, 64, 64),
    (11, 1301, 8, 16, 128, 64),
    (13, 577, 12, 12, 128, 128),
    (10, 1100, 4, 8, 64, 72),
    (153, 520, 1, 1, 40, 128),
]


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", SHARES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_heads_over_many_chunks(dt, B, T, Hk, Hv, dk, dv):
    assert _plan(B, T, Hk, Hv, dk, dv, dt).fwd_launches == 1
    x = lin_inputs(B, T, Hk, Hv, dk, dv, DT[dt], seed=T, device="cuda", packed=True)
    _check(_run(x), lin_ref_grads(x, dk ** -0.5, lin_ref_chunked), {torch.bfloat16: 2.6e-3, torch.float32: 1.5e-6 if dt == "bf16" else 4e-6})


@pytest.mark.parametrize("B", [40, 25])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slow_decays_in_one_run(dt, B):
    """States that hardly fade over whole heads of 256 chunks (4 B heads: in
    shares, or a block each), with a short chunk at the end.  The first two
    decays over 64 tokens lie in the middle between two f32 values: rounded to
    one of them, 256 times the same way, they put results 4e-6 off."""
    T, H = 16384 - 23, 4
    assert _plan(B, T, H, H, 64, 64, dt).fwd_launches == 1
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s, dtype=DT[dt]: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x = {n: r(B, T, H, 64) for n in ("q", "k", "v", "d_o")}
    x["state"], x["d_state_out"] = (30 * r(B, H, 64, 64, dtype=torch.float32) for _ in range(2))
    x["log_decay"] = torch.tensor([-1.5 * 2.0 ** -30, -2.5 * 2.0 ** -30, -3e-7, -2e-5], device="cuda")
    rows = [0, B // 2, B - 1]
    got = _rows(_run(x), rows)
    ref = lin_ref_grads(_rows(x, rows), 64 ** -0.5, lin_ref_chunked)
    _check(got, ref, {torch.bfloat16: 2.6e-3, torch.float32: 2e-6 if dt == "bf16" else 4e-6})


@pytest.mark.parametrize("name,value", [("v", float("nan")), ("k", float("-inf")), ("q", float("nan")), ("d_o", float("inf"))])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_not_finite_in_handed_on_heads(dt, name, value):
    x = lin_inputs(20, 709, 4, 8, 64, 64, DT[dt], seed=2, device="cuda")
    x[name][3, 600, 3, 5] = value
    got = _run(x)
    others = [b for b in range(20) if b != 3]
    assert all(torch.isfinite(t).all() for t in _rows(got, others).values())
    got, ref = _rows(got, [3]), lin_ref_grads(_rows(x, [3]), 64 ** -0.5)
    for n in NAMES:
        fine = torch.isfinite(ref[n])
        assert torch.equal(torch.isfinite(got[n]).cpu(), fine), n
        e = (got[n].double().cpu() - ref[n])[fine].norm() / ref[n][fine].norm().clamp(min=1e-30)
        assert e <= (2.6e-3 if got[n].dtype is torch.bfloat16 else 4e-6), (n, e)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_same_bits_of_handed_on_heads(dt):
    x = lin_inputs(11, 1301, 8, 16, 64, 64, DT[dt], seed=3, device="cuda")
    a = _run(x)
    for _ in range(3):
        b = _run(x)
        for n in NAMES:
            assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("T", [64, 77])
def test_short_sequences_have_two_terms_of_the_weights(T):
    x = lin_inputs(2, T, 4, 8, 64, 96, torch.bfloat16, seed=T, device="cuda", log_decay=[-0.5, -0.05, -0.005, -0.0005])
    _check(_run(x), lin_ref_grads(x, 64 ** -0.5), {torch.bfloat16: 2.05e-3, torch.float32: 1.5e-6})


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", [(2, 300, 2, 4, 128, 128), (1, 4000, 2, 2, 128, 64), (30, 200, 2, 8, 64, 128)])
def test_states_of_bf16_sequences_are_f32_sums(B, T, Hk, Hv, dk, dv):
    x = lin_inputs(B, T, Hk, Hv, dk, dv, torch.bfloat16, seed=B, device="cuda")
    _check(_run(x), lin_ref_grads(x, dk ** -0.5, lin_ref_chunked), {torch.bfloat16: 2.6e-3, torch.float32: 1.5e-6})
