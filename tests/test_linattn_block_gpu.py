"""Norm, rotation and linear attention together, as the example block uses
them, and their calls' workspaces, streams and status."""

import importlib.util
import os

import pytest
import torch

from lin_util import lin_inputs, lin_ref, rel, rot_inputs, rot_ref
from mamba_selective_scan_gb300 import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba_selective_scan_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("linear_attention_block", os.path.join(ROOT, "examples", "linear_attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _ref(block, x, res, dy, dr, state, start):
    d = lambda t: t.detach().double().clone().requires_grad_()
    X, R = d(x), d(res)
    w = {n: d(getattr(block, n)) for n in ("norm_w", "norm_b", "w_in", "w_out", "q_weight", "k_weight")}
    r = X + R
    var, mean = torch.var_mean(r, -1, correction=0, keepdim=True)
    h = (r - mean) * (var + 1e-5).rsqrt() * w["norm_w"] + w["norm_b"]
    q, k, v = block._split(h @ w["w_in"])
    pos = torch.arange(start, start + x.shape[1], device=x.device)
    q, k = (rot_ref(t, w[n], pos, block.inv_freq, 1e-6, False) for t, n in ((q, "q_weight"), (k, "k_weight")))
    o, _ = lin_ref(q, k, v, block.log_decay.double(), state.double(), block.dk ** -0.5)
    y = o.flatten(2) @ w["w_out"]
    loss = (y * dy.double()).sum() + (r * dr.double()).sum()
    gr = torch.autograd.grad(loss, [X, R] + list(w.values()))
    return y.detach().cpu(), {n: g.cpu() for n, g in zip(["x", "residual"] + list(w), gr)}


def test_training_step_in_f32(ex):
    """f32 activations, f32 matrix products: 1e-4 covers their rounding
    through two projections and the block's sums."""
    torch.backends.cuda.matmul.allow_tf32 = False
    block = ex.LinearAttentionBlock(64, 2, 4, head_k=32, head_v=16, rot=24, dtype=torch.float32, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, res, dy, dr = (torch.randn(2, 70, 64, generator=gen, device="cuda") for _ in range(4))
    state = 0.3 * torch.randn(2, 4, 32, 16, generator=gen, device="cuda")
    y, r, _, saved = block.forward(x, residual=res, state=state, start=1234, train=True)
    dx, d_res, grads = block.backward(saved, dy, dr)
    ry, ref = _ref(block, x, res, dy, dr, state, 1234)
    assert rel(y, ry) <= 1e-4
    assert rel(dx, ref["x"]) <= 1e-4 and rel(d_res, ref["residual"]) <= 1e-4
    for n, g in grads.items():
        assert rel(g, ref[n]) <= 1e-4, n


def test_training_step_in_bf16(ex):
    """bf16: each of the block's seven tensors between calls is rounded once
    (1.7e-3 in the 2-norm), and so are three operands inside; as independent
    errors 6e-3, twice that for what adds up along a path."""
    block = ex.LinearAttentionBlock(128, 2, 4, head_k=64, head_v=64, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(2, 200, 128, generator=gen, device="cuda").bfloat16() for _ in range(2))
    res, dr = (torch.randn(2, 200, 128, generator=gen, device="cuda") for _ in range(2))
    state = 0.3 * torch.randn(2, 4, 64, 64, generator=gen, device="cuda")
    y, r, _, saved = block.forward(x, residual=res, state=state, train=True)
    dx, d_res, grads = block.backward(saved, dy, dr)
    ry, ref = _ref(block, x, res, dy, dr, state, 0)
    assert rel(y, ry) <= 1.2e-2
    assert rel(dx, ref["x"]) <= 1.2e-2 and rel(d_res, ref["residual"]) <= 1.2e-2
    for n, g in grads.items():
        assert rel(g, ref[n]) <= 1.2e-2, n


def test_decode_continues_the_prompt(ex):
    """bf16: the single-token kernels and the chunked ones round their outputs
    once each, the chunked ones two operands too, and a GEMM's row may be
    summed in another order: 1e-2."""
    block = ex.LinearAttentionBlock(256, 2, 4, head_k=64, head_v=64, seed=3)
    x = torch.randn(3, 150, 256, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(3, 150, 256, device="cuda")
    whole, r, _, _ = block.forward(x, residual=res)
    _, _, state, _ = block.forward(x[:, :140].contiguous(), residual=res[:, :140].contiguous())
    for t in range(140, 150):
        y, rt = block.decode(x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous(), state, torch.full((3, 1), t, device="cuda"))
        assert rel(y, whole[:, t:t + 1].double().cpu()) <= 1e-2
        assert torch.equal(rt, r[:, t:t + 1])


# ---------------------------------------------------------------------------
# workspaces, status, streams
# ---------------------------------------------------------------------------

def _lin_calls(x):
    args = [x[n] for n in ("q", "k", "v", "log_decay")]

    def run(**kw):
        o, st = binding.m3scan_linattn_fwd(*args, state=x["state"], **kw)
        return {"o": o, "state": st, **binding.m3scan_linattn_bwd(*args, x["d_o"], state=x["state"], d_state_out=x["d_state_out"], want_d_state=True, **kw)}
    return run


def _rot_calls(x):
    rest = [x[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")]

    def run(workspace=None, **kw):
        q, k = binding.m3scan_qkrot_fwd(*rest, **kw)
        return {"qo": q, "ko": k, **binding.m3scan_qkrot_bwd(x["dq_out"], x["dk_out"], *rest, workspace=workspace, **kw)}
    return run


CALLS = {
    "one-walk": lambda s: _lin_calls(lin_inputs(2, 200, 2, 2, 64, 64, torch.bfloat16, seed=s, device="cuda")),
    "shared": lambda s: _lin_calls(lin_inputs(2, 200, 1, 3, 64, 72, torch.bfloat16, seed=s, device="cuda")),
    "segments": lambda s: _lin_calls(lin_inputs(1, 1500, 1, 2, 128, 64, torch.bfloat16, seed=s, device="cuda")),
    "shares": lambda s: _lin_calls(lin_inputs(9, 130, 20, 20, 64, 64, torch.bfloat16, seed=s, device="cuda")),
    "f32": lambda s: _lin_calls(lin_inputs(2, 90, 2, 4, 64, 64, torch.float32, seed=s, device="cuda")),
    "rotation": lambda s: _rot_calls(rot_inputs(3, 70, 4, 2, 64, 64, torch.bfloat16, seed=s, device="cuda")),
}
LIN_DIMS = {"one-walk": (2, 200, 2, 2, 64, 64), "shared": (2, 200, 1, 3, 64, 72), "segments": (1, 1500, 1, 2, 128, 64),
            "shares": (9, 130, 20, 20, 64, 64), "f32": (2, 90, 2, 4, 64, 64)}


def _need(name):
    if name == "rotation":
        d = binding.M3QkrotDims(3, 70, 4, 2, 64, 64, *[0] * 9, 1e-6, 0, 0, 0)
        return binding.m3scan_qkrot_plan(d, binding.M3_BF16).workspace_bytes
    d = binding.M3LinattnDims(*LIN_DIMS[name], *[0] * 6, 0.0, 0)
    return binding.m3scan_linattn_plan(d, binding.M3_F32 if name == "f32" else binding.M3_BF16).workspace_bytes


@pytest.mark.parametrize("name", list(CALLS))
def test_in_the_callers_workspace(ex, name):
    """Exactly the planned bytes are enough, nothing behind them is written,
    what an earlier call left in them does not matter, and fewer are refused."""
    run = CALLS[name](1)
    want = run()
    n = _need(name)
    ws = binding.Workspace(n + 4096, "cuda")
    ws.nbytes = n
    ws.buf[binding.STATUS_BYTES:] = 0xA5
    for _ in range(2):
        got = run(workspace=ws)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    assert (ws.buf[n:] == 0xA5).all() and binding.m3scan_get_status(ws) == 0
    ws.nbytes = n - 1
    with pytest.raises(binding.M3Error) as e:
        run(workspace=ws)
    assert e.value.status == 5


@pytest.mark.parametrize("name", list(CALLS))
def test_on_a_stream_beside_another(ex, name):
    """Two streams at once, each with inputs and workspaces of its own."""
    runs = [CALLS[name](s) for s in (1, 2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = [r(stream=s) for r, s in zip(runs, streams)]
    for s in streams:
        s.synchronize()
    for g, w in zip(got, want):
        for k in w:
            assert torch.equal(g[k], w[k]), k


def test_memory_of_the_stream_it_runs_on(ex):
    """With stream= a call's results and scratch are that stream's memory: work
    still queued on the current stream does not see them overwritten."""
    run = CALLS["segments"](1)
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.empty(64 << 20, device="cuda")
    for _ in range(8):
        busy.normal_()
        tmp = torch.full((1 << 20,), 3.0, device="cuda")
        total = tmp.sum()
        del tmp
        got = run(stream=s)
        assert total.item() == 3 * (1 << 20)
    s.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_status_of_a_workspace_whose_wait_ran_out(ex):
    run = CALLS["one-walk"](3)
    want = run()
    ws = binding.Workspace(_need("one-walk"), "cuda")
    binding.m3scan_selftest_wait_timeout(workspace=ws)
    assert binding.m3scan_get_status(ws) == 7 and binding.m3scan_get_status(ws) == 0
    binding.m3scan_device_status()
    got = run(workspace=ws)
    assert torch.equal(got["o"], want["o"]) and binding.m3scan_get_status(ws) == 0 and binding.m3scan_device_status() == 0


@pytest.mark.parametrize("T", [2, 5, 16, 17, 40])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_decode_of_short_windows(ex, dt, T):
    """More than one token through the decode call, q, k and v as columns of
    one projection; then a single token."""
    x = lin_inputs(3, T + 1, 2, 4, 64, 72, dt, seed=T, device="cuda", packed=True)
    ref, rst = lin_ref(*[x[n].double() for n in "qkv"], x["log_decay"].double(), x["state"].double(), 64 ** -0.5)
    S = x["state"].clone()
    outs = []
    for lo, hi in ((0, T), (T, T + 1)):
        w = torch.cat([x[n][:, lo:hi].flatten(2) for n in "qkv"], 2)
        q, k, v = w.split([128, 128, 288], -1)
        outs.append(binding.m3scan_linattn_decode(q.unflatten(2, (2, 64)), k.unflatten(2, (2, 64)), v.unflatten(2, (4, 72)), x["log_decay"], S))
    assert rel(torch.cat(outs, 1), ref.cpu()) <= (4e-3 if dt is torch.bfloat16 else 2e-5)
    assert rel(S, rst.cpu()) <= 2e-5


def test_a_batch_of_padded_prompts(ex):
    """Prompts of different lengths in one batch: with keys of zero behind its
    end a prompt's state only fades, and its outputs are those of the prompt
    alone."""
    lens, T = [70, 200, 131], 200
    x = lin_inputs(3, T, 2, 2, 64, 64, torch.bfloat16, seed=4, device="cuda")
    for b, n in enumerate(lens):
        x["k"][b, n:] = 0
    o, st = binding.m3scan_linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"])
    for b, n in enumerate(lens):
        ref, rst = lin_ref(*[x[m][b:b + 1, :n].double() for m in "qkv"], x["log_decay"].double(), x["state"][b:b + 1].double(), 64 ** -0.5)
        fade = torch.exp(x["log_decay"].double() * (T - n))[:, None, None]
        assert rel(o[b:b + 1, :n], ref.cpu()) <= 6e-3 and rel(st[b:b + 1], (fade * rst).cpu()) <= 2e-5
