"""Layer norm on the GPU against float64.  Tolerances as 2-norm ratios:
bf16 outputs are one rounding (2^-9 per element) of f32 results: 2e-3; f32
outputs are sums of f32 terms: 1e-5."""

import pytest
import torch

from delta_util import rel
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.bfloat16: 2e-3, torch.float32: 1e-5}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()


def _inputs(rows, dim, dt, residual, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return {"x": r(rows, dim).to(DT[dt]), "w": 1 + 0.2 * r(dim), "b": 0.3 * r(dim), "dy": r(rows, dim).to(DT[dt]),
            "res": 2 * r(rows, dim) + 3 * r(dim) if residual else None, "dres": r(rows, dim) if residual else None}


def _ref(x, eps):
    h = (x["x"].double() + (x["res"].double() if x["res"] is not None else 0)).cpu().requires_grad_()
    w, b = x["w"].double().cpu().requires_grad_(), x["b"].double().cpu().requires_grad_()
    var, mean = torch.var_mean(h, 1, correction=0)
    rstd = (var + eps).rsqrt()
    y = (h - mean[:, None]) * rstd[:, None] * w + b
    loss = (y * x["dy"].double().cpu()).sum()
    if x["dres"] is not None:
        loss = loss + (h * x["dres"].double().cpu()).sum()
    gh, gw, gb = torch.autograd.grad(loss, (h, w, b))
    return {"y": y.detach(), "r": h.detach(), "mean": mean.detach(), "rstd": rstd.detach(), "dh": gh, "dw": gw, "db": gb}


CASES = [(1, 1), (1, 7), (3, 8), (5, 64), (2, 1003), (300, 96), (77, 768), (33, 1001), (64, 2560), (1300, 512),
         (9, 4097), (5, 5120), (3, 8191), (2, 8192), (3, 16384), (2000, 24)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", CASES)
def test_forward_and_gradients(rows, dim, dt, residual):
    if dim == 1:
        pytest.skip("a row of one value has no spread: rstd is 1/sqrt(eps) and the gradient zero; see the test below")
    x = _inputs(rows, dim, dt, residual, seed=rows + dim)
    y, r, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"], residual=x["res"], eps=1e-5)
    normed = r if residual else x["x"]
    g = binding.m3scan_norm_bwd(x["dy"], normed, x["w"], mean, rstd, d_residual_out=x["dres"])
    ref = _ref(x, 1e-5)
    assert rel(y, ref["y"]) <= TOL[y.dtype]
    assert rel(mean, ref["mean"]) <= 1e-5 + 1e-6 / max(ref["mean"].norm().item() / rows ** 0.5, 1e-6)
    assert rel(rstd, ref["rstd"]) <= 1e-5
    if residual:
        assert rel(r, ref["r"]) <= 1e-6
        assert rel(g["d_residual"], ref["dh"]) <= 1e-5
    assert rel(g["dx"], ref["dh"]) <= TOL[g["dx"].dtype]
    assert rel(g["d_weight"], ref["dw"]) <= 1e-5
    assert rel(g["d_bias"], ref["db"]) <= 1e-5


def test_one_column():
    x = _inputs(4, 1, "f32", False)
    y, _, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"])
    assert torch.equal(y, x["b"].expand(4, 1)) and torch.equal(mean, x["x"][:, 0])
    g = binding.m3scan_norm_bwd(x["dy"], x["x"], x["w"], mean, rstd)
    assert torch.equal(g["dx"], torch.zeros_like(g["dx"]))


def test_large_offset_keeps_the_variance():
    """Rows around 1000 with spread 1: the variance comes from deviations."""
    x = _inputs(50, 1024, "f32", False, seed=1)
    x["x"] += 1000.0
    y, _, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"])
    ref = _ref(x, 1e-5)
    # x itself is rounded at 2^-14 of its spread; f32 sums of 1024 values near 1000 are off by a few 1e-5
    assert rel(rstd, ref["rstd"]) <= 1e-5
    assert rel(y, ref["y"]) <= 2e-4


def test_unaligned_rows_and_views():
    """Pointers off the 16-byte boundary take the scalar kernels."""
    base = torch.randn(40 * 512 + 1, device="cuda").to(torch.bfloat16)
    x = _inputs(40, 512, "bf16", False)
    x["x"] = base[1:].view(40, 512)
    y, _, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"])
    g = binding.m3scan_norm_bwd(x["dy"], x["x"], x["w"], mean, rstd)
    ref = _ref(x, 1e-5)
    assert rel(y, ref["y"]) <= 2e-3 and rel(g["dx"], ref["dh"]) <= 2e-3 and rel(g["d_weight"], ref["dw"]) <= 1e-5


def test_no_rows_and_accumulation():
    x = _inputs(0, 64, "bf16", False)
    y, _, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"])
    g = binding.m3scan_norm_bwd(x["dy"], x["x"], x["w"], mean, rstd)
    assert y.shape == (0, 64) and not g["d_weight"].any() and not g["d_bias"].any()
    x = _inputs(100, 64, "f32", False)
    _, _, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"])
    once = binding.m3scan_norm_bwd(x["dy"], x["x"], x["w"], mean, rstd)
    acc = {"d_weight": torch.ones(64, device="cuda"), "d_bias": torch.ones(64, device="cuda")}
    binding.m3scan_norm_bwd(x["dy"], x["x"], x["w"], mean, rstd, accumulate_param_grads=True, out=acc)
    assert torch.equal(acc["d_weight"], once["d_weight"] + 1) and torch.equal(acc["d_bias"], once["d_bias"] + 1)


def test_same_bits_every_call():
    x = _inputs(5000, 768, "bf16", True)
    _, r, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], x["b"], residual=x["res"])
    a, b = (binding.m3scan_norm_bwd(x["dy"], r, x["w"], mean, rstd, d_residual_out=x["dres"]) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_without_bias_and_statistics():
    x = _inputs(10, 256, "bf16", False)
    y, r, mean, rstd = binding.m3scan_norm_fwd(x["x"], x["w"], want_stats=False)
    assert r is None and mean is None and rstd is None
    x["b"] = torch.zeros_like(x["b"])
    assert rel(y, _ref(x, 1e-5)["y"]) <= 2e-3
