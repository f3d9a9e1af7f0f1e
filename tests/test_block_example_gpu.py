"""The example block end to end: its gradients against autograd through the
float64 definitions, and decoding against the full pass."""

import importlib.util
import os

import pytest
import torch

from delta_util import delta_ref, rel

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("gated_delta_block", os.path.join(ROOT, "examples", "gated_delta_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _ref(block, x, res, dy, dr):
    d = lambda t: t.detach().double().cpu().clone().requires_grad_()
    X, R = d(x), d(res)
    w = {n: d(getattr(block, n)) for n in ("norm_w", "norm_b", "w_in", "w_out", "a_log", "dt_bias")}
    r = X + R
    var, mean = torch.var_mean(r, -1, correction=0, keepdim=True)
    h = (r - mean) * (var + 1e-5).rsqrt() * w["norm_w"] + w["norm_b"]
    q, k, v, a, b = block._split(h @ w["w_in"])
    g = -torch.exp(w["a_log"]) * torch.nn.functional.softplus(a + w["dt_bias"])
    o, _ = delta_ref(q, k, v, g, torch.sigmoid(b), None, block.dk ** -0.5, True)
    y = o.flatten(2) @ w["w_out"]
    loss = (y * dy.double().cpu()).sum() + (r * dr.double().cpu()).sum()
    gr = torch.autograd.grad(loss, [X, R] + list(w.values()))
    return y.detach(), dict(zip(["x", "residual"] + list(w), gr))


def test_training_step_in_f32(ex):
    """f32 activations, f32 matrix products: 1e-4 covers their rounding
    through two projections and the block's sums."""
    torch.backends.cuda.matmul.allow_tf32 = False
    block = ex.GatedDeltaBlock(64, 2, 4, head_k=32, head_v=16, dtype=torch.float32, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, res, dy, dr = (torch.randn(2, 70, 64, generator=gen, device="cuda") for _ in range(4))
    y, r, _, saved = block.forward(x, residual=res, train=True)
    dx, d_res, grads = block.backward(saved, dy, dr)
    ry, ref = _ref(block, x, res, dy, dr)
    assert rel(y, ry) <= 1e-4
    assert rel(dx, ref["x"]) <= 1e-4 and rel(d_res, ref["residual"]) <= 1e-4
    for n, g in grads.items():
        assert rel(g, ref[n]) <= 1e-4, n


def test_decode_continues_the_prompt(ex):
    """bf16: the single-token kernels and the chunked ones round their outputs
    once each (2^-9), and a GEMM's row may be summed in another order: 1e-2."""
    block = ex.GatedDeltaBlock(256, 2, 4, head_k=64, head_v=64, seed=3)
    x = torch.randn(3, 150, 256, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(3, 150, 256, device="cuda")
    whole, r, _, _ = block.forward(x, residual=res)
    _, _, state, _ = block.forward(x[:, :140].contiguous(), residual=res[:, :140].contiguous())
    for t in range(140, 150):
        y, rt = block.decode(x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous(), state)
        assert rel(y, whole[:, t:t + 1].double().cpu()) <= 1e-2
        assert torch.equal(rt, r[:, t:t + 1])
