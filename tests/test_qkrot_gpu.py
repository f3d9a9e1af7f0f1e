"""Norm and rotation of queries and keys on the GPU against the float64
definition and its autograd gradients.

Tolerances: outputs are f32 arithmetic rounded once.  To bf16 each value is off
by at most 2^-8 of itself, so the 2-norm of the differences is at most 2^-8
(3.91e-3) of the outputs': 4e-3 (a head of eight values came to 2.7e-3; many
values come to 1.7e-3).  To f32 it is 2^-24 on top of some 2^-22 of f32
arithmetic (a few roundings of 2^-24 each, the cosines' 2^-22): 1e-6.  The weights' gradients are f32 sums: 2e-6 of the 2-norm of
what is added, which for random signs is the sum's own size."""

from fractions import Fraction

import pytest
import torch

from lin_util import rel, rot_inputs, rot_ref_grads
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 4e-3, torch.float32: 1e-6}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _run(x, il=False, eps=EPS, **kw):
    rest = [x[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")]
    q, k = binding.m3scan_qkrot_fwd(*rest, eps=eps, interleaved=il, **kw)
    r = binding.m3scan_qkrot_bwd(x["dq_out"], x["dk_out"], *rest, eps=eps, interleaved=il, **kw)
    r.update(q_out=q, k_out=k)
    return r


def _check(got, ref, sums=2e-6):
    bad = {}
    for n, want in ref.items():
        if want is None:
            assert got[n] is None
            continue
        e = rel(got[n], want)
        if not e <= (sums if n.startswith("d_") else TOL[got[n].dtype]):
            bad[n] = e
    assert not bad, bad


CASES = [
    # B, T, Hq, Hk, D, rot, dtype, packed
    (1, 1, 1, 1, 8, 8, "bf16", False),
    (2, 3, 4, 2, 128, 128, "bf16", True),
    (64, 1, 16, 16, 128, 128, "bf16", False),
    (2, 50, 5, 3, 64, 64, "bf16", False),
    (1, 33, 3, 1, 128, 64, "bf16", True),
    (1, 70, 2, 2, 256, 256, "bf16", False),
    (3, 17, 7, 7, 80, 48, "bf16", True),
    (2, 19, 2, 1, 96, 86, "bf16", False),
    (1, 21, 2, 2, 128, 2, "bf16", False),
    (1, 9, 2, 2, 72, 0, "bf16", False),
    (1, 9, 3, 2, 37, 22, "bf16", False),
    (2, 40, 4, 2, 128, 128, "f32", True),
    (3, 31, 10, 5, 80, 48, "f32", False),
    (1, 12, 1, 1, 256, 250, "f32", False),
    (1, 30, 2, 3, 52, 52, "f32", True),
    (1, 7, 2, 2, 33, 32, "f32", False),
]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(case, il):
    B, T, Hq, Hk, D, rot, dt, packed = case
    x = rot_inputs(B, T, Hq, Hk, D, rot, DT[dt], seed=T + D, device="cuda", packed=packed)
    _check(_run(x, il), rot_ref_grads(x, EPS, il), sums=2e-6 if B * T > 1 else 1e-5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_tokens(dt):
    """More tokens than the blocks take at once."""
    x = rot_inputs(2, 9001, 3, 2, 64, 64, DT[dt], seed=1, device="cuda")
    _check(_run(x), rot_ref_grads(x, EPS, False))


@pytest.mark.parametrize("il", [False, True])
def test_far_positions(il):
    """Positions in the millions and past 32 bits, and before zero: the angle is exact."""
    x = rot_inputs(1, 8, 2, 2, 128, 128, torch.float32, seed=1, device="cuda")
    pos = [0, 1, -1, -1234567, 10 ** 7 + 1, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 36 + 3]
    x["positions"] = torch.tensor([pos], device="cuda")
    # the reference's own angle is a product in 64 bits: off by 2^36 x 2^-53
    # radians at most
    _check(_run(x, il), rot_ref_grads(x, EPS, il), sums=1e-5)


def test_angles_beyond_a_double():
    """Angles of a far position against exact arithmetic: the frequency in
    turns is off by 3 x 2^-65 at most, at 2^38 that is 1.4e-7 radians (and one
    double's product would be off by some 1e-5)."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    x = rot_inputs(1, 6, 1, 1, 16, 16, torch.float32, seed=3, device="cuda")
    x["inv_freq"] = torch.tensor([1.0, 0.9, -0.7, 0.11, 3.3, 1e-3, 42.5, 1e-9], device="cuda")
    pos = [2 ** 38 + 1, 2 ** 38 - 12345, -(2 ** 37) - 77, 2 ** 36 + 5, 987654321987, 3]
    x["positions"] = torch.tensor([pos], device="cuda")
    turns = [[float(p * Fraction(f) / (2 * pi) % 1) for f in x["inv_freq"].tolist()] for p in pos]
    ang = torch.tensor(turns, dtype=torch.float64) * float(2 * pi)
    q, k = binding.m3scan_qkrot_fwd(*(x[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")), eps=EPS)
    for t, w, out in ((x["q"], x["q_weight"], q), (x["k"], x["k_weight"], k)):
        t, w = t.double().cpu(), w.double().cpu()
        n = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w
        a, b = n[..., :8], n[..., 8:]
        c, s = ang.cos()[None, :, None], ang.sin()[None, :, None]
        assert rel(out, torch.cat((a * c - b * s, a * s + b * c), -1)) <= TOL[torch.float32]


def test_frequencies_of_every_size():
    x = rot_inputs(1, 50, 2, 2, 16, 16, torch.float32, seed=1, device="cuda", start=3000)
    x["inv_freq"] = torch.tensor([0.0, 1e-30, 1.0, -0.3, 3.0, 6.2831855, 700.25, 1e4], device="cuda")
    _check(_run(x), rot_ref_grads(x, EPS, False), sums=1e-5)
    x["inv_freq"][2] = float("inf")
    r = _run(x)
    bad = torch.isnan(r["q_out"]).any(1).any(1).any(0).cpu()
    assert bad.nonzero().flatten().tolist() == [2, 10]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_without_weights_and_shared_positions(dt):
    x = rot_inputs(2, 30, 2, 2, 64, 64, DT[dt], seed=1, device="cuda")
    x["q_weight"] = x["k_weight"] = None
    x["positions"] = torch.arange(5, 35, device="cuda")
    _check(_run(x), rot_ref_grads(x, EPS, False))
    # a view of positions whose batch rows are all the same
    y = dict(x, positions=x["positions"].expand(2, 30))
    a, b = _run(x), _run(y)
    for n in a:
        assert a[n] is None and b[n] is None or torch.equal(a[n], b[n])
    z = dict(x, positions=None, inv_freq=None)
    _check({n: t for n, t in _run(z).items()}, rot_ref_grads(dict(z, positions=x["positions"], inv_freq=torch.empty(0, device="cuda")), EPS, False))


def test_weights_added_to():
    x = rot_inputs(2, 30, 2, 2, 64, 64, torch.bfloat16, seed=1, device="cuda")
    once = _run(x)
    rest = [x[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")]
    r = binding.m3scan_qkrot_bwd(x["dq_out"], x["dk_out"], *rest, eps=EPS, accumulate_param_grads=True,
                                 out={"d_q_weight": torch.ones(64, device="cuda")})
    assert torch.equal(r["d_q_weight"], once["d_q_weight"] + 1) and torch.equal(r["d_k_weight"], once["d_k_weight"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_place_and_in_columns(dt):
    """Outputs over the inputs, inside one projection's output; what lies
    behind them stays."""
    x = rot_inputs(2, 30, 4, 2, 64, 64, DT[dt], seed=1, device="cuda")
    want = _run(x)
    row = torch.full((2, 30, 6 * 64 + 16), 5.0, dtype=DT[dt], device="cuda")
    q, k = row[..., :256].unflatten(2, (4, 64)), row[..., 256:384].unflatten(2, (2, 64))
    q.copy_(x["q"])
    k.copy_(x["k"])
    w = [x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")]
    binding.m3scan_qkrot_fwd(q, k, *w, eps=EPS, q_out=q, k_out=k)
    assert torch.equal(q, want["q_out"]) and torch.equal(k, want["k_out"]) and (row[..., 384:] == 5).all()
    q.copy_(x["dq_out"])
    k.copy_(x["dk_out"])
    binding.m3scan_qkrot_bwd(q, k, x["q"], x["k"], *w, eps=EPS, out={"dq": q, "dk": k})
    assert torch.equal(q, want["dq"]) and torch.equal(k, want["dk"]) and (row[..., 384:] == 5).all()


def test_not_finite_stays_in_its_head():
    x = rot_inputs(1, 20, 3, 2, 64, 64, torch.bfloat16, seed=1, device="cuda")
    x["q"][0, 7, 1, 3] = float("nan")
    x["k"][0, 9, 0, 0] = float("inf")
    r = _run(x)
    ref = rot_ref_grads(x, EPS, False)
    for n in ("q_out", "k_out", "dq", "dk"):
        fine = torch.isfinite(r[n]).all(-1).cpu()
        assert (~fine).nonzero().tolist() == [[0, 7, 1] if "q" in n else [0, 9, 0]]
        assert rel(r[n][fine.cuda()], ref[n][fine]) <= TOL[torch.bfloat16]


@pytest.mark.parametrize("eps", [0.0, 1e-3])
def test_zero_rows(eps):
    x = rot_inputs(1, 4, 2, 2, 64, 64, torch.float32, seed=1, device="cuda")
    x["q"] = x["q"] * 0 if eps else x["q"]
    r = _run(x, eps=eps)
    _check(r, rot_ref_grads(x, eps, False), sums=1e-5)


def test_no_tokens():
    x = rot_inputs(0, 4, 2, 2, 64, 64, torch.float32, device="cuda")
    r = _run(x)
    assert r["q_out"].shape == (0, 4, 2, 64) and (r["d_q_weight"] == 0).all() and (r["d_k_weight"] == 0).all()


def test_captured_streams_and_same_bits():
    x = rot_inputs(3, 100, 4, 2, 128, 128, torch.bfloat16, seed=2, device="cuda")
    want = _run(x)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        r = _run(x)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = _run(x, stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(r[n], want[n]) and torch.equal(got[n], want[n]), n


def test_offsets_past_32_bits():
    T, stride = 2100, 1 << 20
    row = torch.empty(1, T, stride, dtype=torch.bfloat16, device="cuda")
    x = rot_inputs(1, T, 1, 1, 64, 64, torch.bfloat16, seed=6, device="cuda")
    want = _run(x)
    q, k = row[..., :64].unflatten(2, (1, 64)), row[..., 64:128].unflatten(2, (1, 64))
    q.copy_(x["q"])
    k.copy_(x["k"])
    w = [x[n] for n in ("q_weight", "k_weight", "positions", "inv_freq")]
    out = {"dq": row[..., 128:192].unflatten(2, (1, 64)), "dk": row[..., 192:256].unflatten(2, (1, 64))}
    r = binding.m3scan_qkrot_bwd(x["dq_out"], x["dk_out"], q, k, *w, eps=EPS, out=out)
    assert torch.equal(r["dq"], want["dq"]) and torch.equal(r["dk"], want["dk"])
    binding.m3scan_qkrot_fwd(q, k, *w, eps=EPS, q_out=q, k_out=k)
    assert torch.equal(q, want["q_out"]) and torch.equal(k, want["k_out"])


def test_gradients_against_differences():
    """The loss along a direction, by the calls alone (f32); its curvature
    leaves h^2 / 6 of the third derivative, of the order of the first."""
    x = rot_inputs(1, 6, 2, 2, 32, 32, torch.float32, seed=3, device="cuda")

    def loss(**kw):
        y = {**x, **kw}
        q, k = binding.m3scan_qkrot_fwd(*[y[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")], eps=EPS)
        return ((q.double() * x["dq_out"]).sum() + (k.double() * x["dk_out"]).sum()).item()

    r = _run(x)
    gen = torch.Generator().manual_seed(3)
    for n, d in (("q", "dq"), ("k", "dk"), ("q_weight", "d_q_weight"), ("k_weight", "d_k_weight")):
        u = torch.randn(x[n].shape, generator=gen).cuda()
        h = 1e-2
        diff = (loss(**{n: x[n] + h * u}) - loss(**{n: x[n] - h * u})) / (2 * h)
        want = (r[d].double() * u).sum().item()
        size = (r[d].double().norm() * u.double().norm()).item()
        assert abs(diff - want) <= 1e-3 * size


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D,rot,dt", [(64, 32, "bf16"), (80, 48, "f32"), (80, 50, "bf16"), (37, 22, "f32"), (128, 4, "bf16"), (128, 126, "f32")])
@pytest.mark.parametrize("name,value", [("q", float("inf")), ("q", float("nan")), ("dq_out", float("inf")), ("dq_out", float("nan")),
                                        ("q_weight", float("-inf")), ("q_weight", float("nan"))])
def test_not_finite_among_values_that_do_not_turn(name, value, D, rot, dt, il):
    """A value or a weight behind the turned ones that is not finite reaches
    what the definition says: its own output and the head's sums, not the
    values that it lies beside."""
    x = rot_inputs(2, 5, 3, 1, D, rot, DT[dt], seed=D, device="cuda")
    for place in {rot, D - 1}:
        y = dict(x)
        y[name] = x[name].clone()
        y[name][(..., place) if name == "q_weight" else (1, 3, 2, place)] = value
        got, ref = _run(y, il), rot_ref_grads(y, EPS, il)
        for n, want in ref.items():
            fine = torch.isfinite(want)
            assert torch.equal(torch.isfinite(got[n]).cpu(), fine), n
            assert rel(got[n][fine.cuda()], want[fine]) <= (2e-6 if n.startswith("d_") else TOL[got[n].dtype]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_not_finite_weight_of_a_pair(dt):
    """The weight of a turned value reaches both values of its pair."""
    x = rot_inputs(2, 5, 3, 1, 64, 32, DT[dt], seed=1, device="cuda")
    x["k_weight"][21] = float("inf")
    bad = (~torch.isfinite(_run(x)["k_out"])).flatten(0, 2).all(0).nonzero().flatten().tolist()
    assert bad == [5, 21] and torch.equal(torch.isfinite(_run(x)["k_out"]).cpu(), torch.isfinite(rot_ref_grads(x, EPS, False)["k_out"]))


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_row_of_zeros_without_eps(dt, il):
    """0 / 0 in that head alone: its outputs, its gradient, and the weight's
    gradient, to which it adds."""
    x = rot_inputs(2, 4, 3, 2, 64, 48, DT[dt], seed=1, device="cuda")
    x["q"][1, 2, 1] = 0
    got, ref = _run(x, il, eps=0.0), rot_ref_grads(x, 0.0, il)
    for n, want in ref.items():
        fine = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got[n]).cpu(), fine), n
        if fine.any():
            assert rel(got[n][fine.cuda()], want[fine]) <= (2e-6 if n.startswith("d_") else TOL[got[n].dtype]), n
    assert not torch.isfinite(ref["q_out"]).all() and not torch.isfinite(ref["d_q_weight"]).any()
