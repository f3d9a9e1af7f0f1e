"""The block operators' calls with the caller's workspace, short windows
through the decode call, column views of one projection, and wide rows.
Tolerances as in the operators' own tests."""

import pytest
import torch

from delta_util import delta_inputs, delta_ref, rel
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.bfloat16: 4e-3, torch.float32: 2e-5}
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _delta_dims(x, l2norm=1):
    B, T, Hv, dv = x["v"].shape
    Hk, dk = x["k"].shape[2:]
    return binding.M3DeltaDims(B, T, Hk, Hv, dk, dv, 0, 0, 0, 0, 0, 0, 0.0, l2norm)


@pytest.mark.parametrize("B,T,H,dt", [(2, 100, 2, "bf16"), (1, 1100, 2, "bf16"), (8, 130, 20, "bf16"), (2, 70, 2, "f32")])
def test_delta_in_the_callers_workspace(B, T, H, dt):
    """The planned sizes are enough, nothing past them is written, the results
    are the bits of calls with scratch of their own, and the status is normal."""
    x = delta_inputs(B, T, H, H, 64, 64, DT[dt], seed=T, device="cuda")
    args = [x[n] for n in NAMES]
    pl = binding.m3scan_delta_plan(_delta_dims(x), binding._act_code(x["v"]))

    def both(fw, bw):
        o, st, ck = binding.m3scan_delta_fwd(*args, state=x["state"], qk_l2norm=True, want_ckpt=True, workspace=fw)
        return {"o": o, "st": st, **binding.m3scan_delta_bwd(*args, ck, x["d_o"], d_state_out=x["d_state_out"], want_d_state=True,
                                                           qk_l2norm=True, workspace=bw)}

    want = both(None, None)
    ws = []
    for n in (pl.fwd_workspace_bytes, pl.workspace_bytes):
        w = binding.Workspace(n + 4096, "cuda")
        w.nbytes = n
        w.buf[n:] = 0xA5
        ws.append(w)
    got = both(*ws)
    for n, t in want.items():
        assert torch.equal(got[n], t), n
    for w in ws:
        assert (w.buf[w.nbytes:] == 0xA5).all()
        assert binding.m3scan_get_status(w) == 0
        w.nbytes -= 1
    with pytest.raises(binding.M3Error) as e:
        both(ws[0], ws[1])
    assert e.value.status == 5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(3, 64), (1300, 512), (77, 1001)])
def test_norm_in_the_callers_workspace(rows, dim, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn(rows, dim, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    w = torch.randn(dim, generator=g, device="cuda")
    _, _, mean, rstd = binding.m3scan_norm_fwd(x, w)
    n = binding.m3scan_norm_plan(binding.M3NormDims(rows, dim, 0.0, 0), binding._act_code(x)).workspace_bytes
    want = binding.m3scan_norm_bwd(dy, x, w, mean, rstd)
    ws = binding.Workspace(n + 4096, "cuda")
    ws.nbytes = n
    ws.buf[n:] = 0xA5
    got = binding.m3scan_norm_bwd(dy, x, w, mean, rstd, workspace=ws)
    for k in ("dx", "d_weight", "d_bias"):
        assert torch.equal(got[k], want[k]), k
    assert (ws.buf[n:] == 0xA5).all() and binding.m3scan_get_status(ws) == 0
    ws.nbytes = n - 1
    with pytest.raises(binding.M3Error) as e:
        binding.m3scan_norm_bwd(dy, x, w, mean, rstd, workspace=ws)
    assert e.value.status == 5


def test_status_of_a_workspace_whose_wait_ran_out():
    """A wait that ran out shows in the workspace's status, once; the next call
    with it is right."""
    x = delta_inputs(1, 100, 2, 2, 64, 64, torch.bfloat16, device="cuda")
    args = [x[n] for n in NAMES]
    pl = binding.m3scan_delta_plan(_delta_dims(x), binding.M3_BF16)
    ws = binding.Workspace(pl.workspace_bytes, "cuda")
    want, _, _ = binding.m3scan_delta_fwd(*args, qk_l2norm=True)
    binding.m3scan_selftest_wait_timeout(workspace=ws)
    assert binding.m3scan_get_status(ws) == 7 and binding.m3scan_get_status(ws) == 0
    binding.m3scan_device_status()
    got, _, _ = binding.m3scan_delta_fwd(*args, qk_l2norm=True, workspace=ws)
    assert torch.equal(got, want) and binding.m3scan_get_status(ws) == 0


@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("T", [2, 5, 16, 17, 40])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_of_short_windows(dt, T, l2norm):
    """More than one token through the decode call, q, k and v as columns of
    one projection; then a single token of the same buffer."""
    x = delta_inputs(3, T + 1, 2, 4, 64, 72, DT[dt], seed=T, device="cuda", packed=True)
    if not l2norm:
        row = x["q"]._base if x["q"]._base is not None else x["q"]
        row *= 0.1
    ref, rst = delta_ref(*[x[n].double().cpu() for n in NAMES], x["state"].double().cpu(), 64 ** -0.5, l2norm)
    S = x["state"].clone()
    outs = []
    for lo, hi in ((0, T), (T, T + 1)):
        # a window of its own rows: the projection's output is made per call
        w = torch.cat([x[n][:, lo:hi].flatten(2) for n in ("q", "k", "v")], 2)
        q, k, v = w.split([128, 128, 288], -1)
        outs.append(binding.m3scan_delta_decode(q.unflatten(2, (2, 64)), k.unflatten(2, (2, 64)), v.unflatten(2, (4, 72)),
                                                x["g"][:, lo:hi].contiguous(), x["beta"][:, lo:hi].contiguous(), S, qk_l2norm=l2norm))
    assert rel(torch.cat(outs, 1), ref) <= TOL[DT[dt]]
    assert rel(S, rst) <= 2e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [40, 1000])
def test_norm_of_the_widest_rows(rows, dt):
    """16384 columns (eight vectors per thread in the backward), with fewer and
    with more rows than blocks."""
    dim = 16384
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy, res, dres, w, b = r(rows, dim).to(DT[dt]), r(rows, dim).to(DT[dt]), r(rows, dim), r(rows, dim), r(dim), r(dim)
    y, h, mean, rstd = binding.m3scan_norm_fwd(x, w, b, residual=res)
    got = binding.m3scan_norm_bwd(dy, h, w, mean, rstd, d_residual_out=dres)
    d = lambda t: t.double()
    z = d(x) + d(res)
    var, mu = torch.var_mean(z, 1, correction=0, keepdim=True)
    rs = (var + 1e-5).rsqrt()
    xh = (z - mu) * rs
    e = d(dy) * d(w)
    dz = rs * (e - e.mean(1, keepdim=True) - xh * (e * xh).mean(1, keepdim=True)) + d(dres)
    tol = {torch.bfloat16: 2e-3, torch.float32: 1e-5}[DT[dt]]
    assert rel(y, (xh * d(w) + d(b)).cpu()) <= tol and rel(got["dx"], dz.cpu()) <= tol
    assert rel(got["d_residual"], dz.cpu()) <= 1e-5
    assert rel(got["d_weight"], (d(dy) * xh).sum(0).cpu()) <= 1e-5 and rel(got["d_bias"], d(dy).sum(0).cpu()) <= 1e-5
