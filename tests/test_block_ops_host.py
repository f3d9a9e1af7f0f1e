"""Host-side checks of the layer norm and gated delta rule entry points: their
plans and refusals (no GPU; every call with addresses fails validation)."""

import ctypes

import pytest
import torch

from delta_util import delta_inputs, delta_ref, delta_ref_grads
from mamba_selective_scan_gb300 import binding, build

F32, BF16 = binding.M3_F32, binding.M3_BF16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _delta(**kw):
    d = dict(batch=2, seq_len=100, k_heads=2, v_heads=4, head_k=64, head_v=128)
    d.update(kw)
    return binding.M3DeltaDims(**d)


def _delta_plan(dims, act=BF16):
    out = binding.M3DeltaPlan()
    return binding.load().m3scan_delta_plan(ctypes.byref(dims), act, ctypes.byref(out)), out


def test_delta_plan_sizes(lib):
    st, p = _delta_plan(_delta())
    assert st == 0 and p.n_chunks == -(-100 // p.chunk)
    assert p.ckpt_bytes == 2 * 4 * p.n_chunks * 99456  # bf16: state and update tiles padded to 128, T, P, factors
    assert p.workspace_bytes >= p.fwd_workspace_bytes >= binding.STATUS_BYTES and p.fwd_launches >= 1 and p.bwd_launches >= 1
    st, p = _delta_plan(_delta(seq_len=0))
    assert st == 0 and p.n_chunks == 0 and p.ckpt_bytes == 0 and p.fwd_launches == 0 and p.bwd_launches == 0
    # sizes past 32 bits
    st, p = _delta_plan(_delta(batch=8, seq_len=1 << 20, v_heads=64, k_heads=64, head_k=128))
    assert st == 0 and p.ckpt_bytes == 8 * 64 * p.n_chunks * 99456
    st, p = _delta_plan(_delta(), act=F32)
    assert st == 0 and p.ckpt_bytes == 2 * 4 * p.n_chunks * 64 * 128 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 2), (dict(seq_len=-1), 2), (dict(k_heads=0), 2), (dict(v_heads=0), 2), (dict(batch=70000), 2),
    (dict(v_heads=3), 3), (dict(head_k=0), 3), (dict(head_k=12), 3), (dict(head_k=136), 3), (dict(head_v=136), 3),
    (dict(head_v=4), 3), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(qk_l2norm=2), 2),
    (dict(q_stride=127), 2), (dict(q_stride=132), 4), (dict(v_stride=511), 2), (dict(dk_stride=-8), 2),
])
def test_delta_refuses(lib, kw, status):
    assert _delta_plan(_delta(**kw))[0] == status


def test_delta_refuses_other_types_and_null(lib):
    assert _delta_plan(_delta(), act=5)[0] == 3
    assert lib.m3scan_delta_plan(None, BF16, ctypes.byref(binding.M3DeltaPlan())) == 1
    d = _delta()
    n = [None] * 10
    assert lib.m3scan_delta_fwd(ctypes.byref(d), BF16, *n, 0, None) == 1
    assert lib.m3scan_delta_bwd(ctypes.byref(d), BF16, *([None] * 15), 0, None) == 1
    assert lib.m3scan_delta_decode(ctypes.byref(d), BF16, *([None] * 8)) == 1
    # misaligned q, then a missing and a small workspace
    a = 1 << 20
    assert lib.m3scan_delta_fwd(ctypes.byref(d), BF16, a + 8, a, a, a, a, None, a, None, None, None, 0, None) == 4
    assert lib.m3scan_delta_fwd(ctypes.byref(d), BF16, a, a, a, a, a, None, a, None, None, None, 0, None) == 5
    assert lib.m3scan_delta_fwd(ctypes.byref(d), BF16, a, a, a, a, a, None, a, None, None, a, 16, None) == 5
    assert lib.m3scan_delta_bwd(ctypes.byref(d), BF16, a, a, a, a, a, a, a, None, a, a, a, a, a, None, None, 0, None) == 5


@pytest.mark.parametrize("rows,dim,eps,act,status", [
    (-1, 8, 1e-5, BF16, 2), (1, -8, 1e-5, BF16, 2), (1, 8, -1.0, BF16, 2), (1, 8, float("nan"), BF16, 2),
    (1, 8, 1e-5, 7, 3), (1, 16392, 1e-5, BF16, 3), (1, 8193, 1e-5, F32, 3), (1 << 31, 8, 1e-5, F32, 2),
])
def test_norm_refuses(lib, rows, dim, eps, act, status):
    d = binding.M3NormDims(rows, dim, eps, 0)
    assert lib.m3scan_norm_plan(ctypes.byref(d), act, ctypes.byref(binding.M3NormPlan())) == status
    assert lib.m3scan_norm_fwd(ctypes.byref(d), act, *([None] * 9)) == status


def test_norm_refuses_pointers(lib):
    d = binding.M3NormDims(4, 16, 1e-5, 0)
    a = 1 << 20
    assert lib.m3scan_norm_fwd(ctypes.byref(d), BF16, *([None] * 9)) == 1
    assert lib.m3scan_norm_fwd(ctypes.byref(d), BF16, a + 1, None, a, a, a, None, None, None, None) == 4
    assert lib.m3scan_norm_fwd(ctypes.byref(d), BF16, a, a + 2, a, a, a, None, None, None, None) == 4
    assert lib.m3scan_norm_bwd(ctypes.byref(d), BF16, a, a, BF16, a, a, a, None, a, None, a, a, None, 0, None) == 5
    assert lib.m3scan_norm_bwd(ctypes.byref(d), F32, a, a, BF16, a, a, a, None, a, None, a, a, a, 1 << 20, None) == 3
    # 16384 columns only with rows on 16 bytes
    d = binding.M3NormDims(4, 16384, 1e-5, 0)
    assert lib.m3scan_norm_fwd(ctypes.byref(d), BF16, a + 2, None, a, a, a, None, None, None, None) == 4


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    x = delta_inputs(1, 4, 1, 2, 16, 16, torch.float32)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError):
        binding.m3scan_delta_fwd(*args)
    with pytest.raises(ValueError):
        binding.m3scan_norm_fwd(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(TypeError):
        binding.m3scan_norm_fwd(torch.zeros(2, 8, dtype=torch.float16), torch.ones(8))


def test_reference_gradients_against_differences():
    """The float64 definition's autograd gradients against central differences."""
    x = {k: v.double() for k, v in delta_inputs(1, 9, 1, 2, 8, 8, torch.float32, seed=3).items()}
    ref = delta_ref_grads(x, 0.3, True)

    def loss(y):
        o, S = delta_ref(y["q"], y["k"], y["v"], y["g"], y["beta"], y["state"], 0.3, True)
        return ((o * x["d_o"]).sum() + (S * x["d_state_out"]).sum()).item()

    gen = torch.Generator().manual_seed(0)
    for n in ("q", "k", "v", "g", "beta", "state"):
        d = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        num = (loss({**x, n: x[n] + eps * d}) - loss({**x, n: x[n] - eps * d})) / (2 * eps)
        ana = (ref["d_state" if n == "state" else "d" + n] * d).sum().item()
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), n


@pytest.mark.parametrize("shape,view", [
    ((1, 1, 2, 64), lambda t: t.expand(1, 100, 2, 64)),   # one key for all tokens
    ((1, 1, 2, 64), lambda t: t.expand(2, 100, 2, 64)),   # and for all sequences
    ((1, 1, 2, 64), lambda t: t.expand(3, 1, 2, 64)),     # a single token shared by a batch
    ((1, 710), lambda t: t.as_strided((1, 10, 2, 64), (0, 64, 64, 1))),  # tokens that overlap
    ((1, 710), lambda t: t.as_strided((4, 1, 2, 64), (120, 64, 64, 1))),
])
def test_token_stride_refuses_overlapping_tokens(shape, view):
    """A token stride below a token's width (0 in a broadcast view) is not
    passed on: 0 is the C ABI's word for dense."""
    t = view(torch.zeros(shape))
    with pytest.raises(ValueError):
        binding._token_stride(t, "k", t.dtype, -1, t.shape)


@pytest.mark.parametrize("B,T", [(1, 1), (1, 5), (3, 1), (2, 5), (0, 4), (2, 0)])
def test_token_stride_of_views_and_dense_tensors(B, T):
    assert binding._token_stride(torch.zeros(B, T, 2, 64), "k", torch.float32, -1, (B, T, 2, 64)) == 0
    row = torch.zeros(B, T, 400)
    for t in (row[..., :128], row[..., 128:256], row[..., 272:]):
        t = t.unflatten(2, (2, 64))
        want = 0 if t.is_contiguous() else 400 if B * T > 1 else 128
        assert binding._token_stride(t, "k", torch.float32, -1, (B, T, 2, 64)) == want


class _Cuda:
    """Stands in for torch.cuda on a machine with several devices."""

    def __init__(self):
        self.now = (0, None)

    def _on(self, place):
        import contextlib

        @contextlib.contextmanager
        def on():
            was, self.now = self.now, place
            yield
            self.now = was
        return on()

    def current_device(self):
        return self.now[0]

    def device(self, index):
        return self._on((index, None))

    def stream(self, s):
        return self._on((s.device.index, s))


WRAPPERS = ("m3scan_fwd", "m3scan_fwd_state", "m3scan_bwd", "m3scan_bwd_state", "m3scan_decode", "m3scan_bwd_two_phase",
            "m3scan_norm_fwd", "m3scan_norm_bwd", "m3scan_delta_fwd", "m3scan_delta_bwd", "m3scan_delta_decode")


@pytest.mark.parametrize("name", WRAPPERS)
def test_calls_run_on_their_tensors_device(name, monkeypatch):
    """The library launches on the current device, so a wrapper makes its
    tensors' device current (and its stream); a stream of another device is
    refused."""
    from types import SimpleNamespace as NS

    cuda, seen = _Cuda(), []
    monkeypatch.setattr(binding, "_TORCH", NS(cuda=cuda))
    tensor = lambda index: NS(get_device=lambda: index)

    def probe(x, stream=None):
        seen.append((cuda.now, stream))
        return "done"

    placed = binding._placed(probe)
    assert placed(tensor(0)) == "done" and placed(tensor(1)) == "done" and placed(x=tensor(2)) == "done"
    assert [s[0][0] for s in seen] == [0, 1, 2] and cuda.now == (0, None)
    s1 = NS(device=NS(index=1))
    assert placed(tensor(1), stream=s1) == "done" and seen[-1] == ((1, s1), s1)
    with pytest.raises(ValueError):
        placed(tensor(0), stream=s1)
    assert placed(tensor(-1)) == "done"  # (a host tensor: the call itself says what is wrong)
    assert getattr(binding, name).__code__ is placed.__code__  # this wrapper is placed like the probe
