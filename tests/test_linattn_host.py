"""Host-side checks of linear attention with a decay per head and of the norm
and rotation of queries and keys: plans and refusals (no GPU; every call with
addresses fails validation), and the float64 definitions themselves."""

import ctypes

import pytest
import torch

from lin_util import lin_inputs, lin_ref, lin_ref_chunked, lin_ref_grads, rel, rot_inputs, rot_ref, rot_ref_grads
from mamba_selective_scan_gb300 import binding, build

F32, BF16 = binding.M3_F32, binding.M3_BF16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _lin(**kw):
    d = dict(batch=2, seq_len=100, k_heads=2, v_heads=4, head_k=64, head_v=128)
    d.update(kw)
    return binding.M3LinattnDims(**d)


def _lin_plan(dims, act=BF16):
    out = binding.M3LinattnPlan()
    return binding.load().m3scan_linattn_plan(ctypes.byref(dims), act, ctypes.byref(out)), out


def _rot(**kw):
    d = dict(batch=2, seq_len=100, q_heads=4, k_heads=2, head_dim=64, rot_dim=32, eps=1e-6)
    d.update(kw)
    return binding.M3QkrotDims(**d)


def _rot_plan(dims, act=BF16):
    out = binding.M3QkrotPlan()
    return binding.load().m3scan_qkrot_plan(ctypes.byref(dims), act, ctypes.byref(out)), out


@pytest.mark.parametrize("act", [BF16, F32])
def test_linattn_plan(lib, act):
    st, p = _lin_plan(_lin(), act)
    assert st == 0 and p.workspace_bytes >= binding.STATUS_BYTES and p.fwd_workspace_bytes == 0
    assert p.fwd_launches == 1 and p.bwd_launches >= 1
    # segments of a long sequence, shares of many heads
    st, p = _lin_plan(_lin(batch=1, seq_len=20000), act)
    assert st == 0 and p.workspace_bytes >= p.fwd_workspace_bytes > binding.STATUS_BYTES and p.fwd_launches == 3
    st, p = _lin_plan(_lin(batch=100), act)
    assert st == 0 and p.fwd_launches == 1
    assert p.fwd_workspace_bytes > binding.STATUS_BYTES if act == BF16 else p.fwd_workspace_bytes == 0
    st, p = _lin_plan(_lin(seq_len=0), act)
    assert st == 0 and p.fwd_launches == 0 and p.bwd_launches == 0
    # sizes past 32 bits: the shares of shared heads' dq and dk
    st, p = _lin_plan(_lin(batch=8, seq_len=1 << 20, k_heads=1, v_heads=64, head_k=128), act)
    assert st == 0 and p.workspace_bytes >= 2 * 8 * (1 << 20) * 64 * 128 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 2), (dict(seq_len=-1), 2), (dict(k_heads=0), 2), (dict(v_heads=0), 2), (dict(batch=70000), 2),
    (dict(v_heads=3), 3), (dict(head_k=0), 3), (dict(head_k=12), 3), (dict(head_k=136), 3), (dict(head_v=136), 3),
    (dict(head_v=4), 3), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(reserved=1), 2),
    (dict(q_stride=127), 2), (dict(q_stride=132), 4), (dict(v_stride=511), 2), (dict(dk_stride=-8), 2),
    (dict(seq_len=(1 << 30) + 1), 2), (dict(batch=8, seq_len=1 << 30, k_heads=1, v_heads=64), 2),
])
def test_linattn_refuses(lib, kw, status):
    assert _lin_plan(_lin(**kw))[0] == status


def test_linattn_refuses_pointers(lib):
    assert _lin_plan(_lin(), act=5)[0] == 3
    assert lib.m3scan_linattn_plan(None, BF16, ctypes.byref(binding.M3LinattnPlan())) == 1
    d, a = _lin(batch=1, seq_len=20000), 1 << 20
    ref = ctypes.byref(d)
    assert lib.m3scan_linattn_plan(ref, BF16, None) == 1
    assert lib.m3scan_linattn_fwd(ref, BF16, *([None] * 8), 0, None) == 1
    assert lib.m3scan_linattn_bwd(ref, BF16, *([None] * 12), 0, None) == 1
    assert lib.m3scan_linattn_decode(ref, BF16, *([None] * 7)) == 1
    # misaligned q, state and decays, then a missing, a small and a misaligned workspace
    assert lib.m3scan_linattn_fwd(ref, BF16, a + 8, a, a, a, None, a, None, None, 0, None) == 4
    assert lib.m3scan_linattn_fwd(ref, BF16, a, a, a, a, a + 4, a, None, None, 0, None) == 4
    assert lib.m3scan_linattn_fwd(ref, BF16, a, a, a, a + 2, None, a, None, None, 0, None) == 4
    assert lib.m3scan_linattn_fwd(ref, BF16, a, a, a, a, None, a, None, None, 0, None) == 5
    assert lib.m3scan_linattn_fwd(ref, BF16, a, a, a, a, None, a, None, a, 16, None) == 5
    assert lib.m3scan_linattn_fwd(ref, BF16, a, a, a, a, None, a, None, a + 16, 1 << 40, None) == 4
    assert lib.m3scan_linattn_bwd(ref, BF16, a, a, a, a, None, a, None, a, a, a, None, None, 0, None) == 5
    assert lib.m3scan_linattn_decode(ref, BF16, a, a, a, a, None, a, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 2), (dict(seq_len=-1), 2), (dict(q_heads=0), 2), (dict(k_heads=0), 2), (dict(head_dim=0), 2), (dict(head_dim=1, rot_dim=0), 2),
    (dict(head_dim=257), 3), (dict(rot_dim=-2), 2), (dict(rot_dim=66), 2), (dict(rot_dim=31), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(interleaved=2), 2), (dict(accumulate_param_grads=3), 2), (dict(q_stride=255), 2),
    (dict(dk_out_stride=-1), 2), (dict(position_stride=99), 2), (dict(position_stride=-100), 2), (dict(reserved=1), 2),
])
def test_qkrot_refuses(lib, kw, status):
    assert _rot_plan(_rot(**kw))[0] == status


def test_qkrot_refuses_pointers(lib):
    st, p = _rot_plan(_rot())
    assert st == 0 and p.workspace_bytes >= binding.STATUS_BYTES + 64 * 8
    assert _rot_plan(_rot(), act=5)[0] == 3
    assert lib.m3scan_qkrot_plan(None, BF16, ctypes.byref(binding.M3QkrotPlan())) == 1
    d, a = _rot(), 1 << 20
    ref = ctypes.byref(d)
    assert lib.m3scan_qkrot_plan(ref, BF16, None) == 1
    assert lib.m3scan_qkrot_fwd(ref, BF16, *([None] * 9)) == 1
    assert lib.m3scan_qkrot_fwd(ref, BF16, a, a, None, None, None, None, a, a, None) == 1  # rotation without positions
    assert lib.m3scan_qkrot_fwd(ref, BF16, a + 1, a, a, a, a, a, a, a, None) == 4
    assert lib.m3scan_qkrot_fwd(ref, BF16, a, a, a + 2, a, a, a, a, a, None) == 4
    assert lib.m3scan_qkrot_fwd(ref, BF16, a, a, a, a, a + 4, a, a, a, None) == 4
    assert lib.m3scan_qkrot_bwd(ref, BF16, a, a, a, a, a, a, a, a, a, a, a, a, None, 0, None) == 5
    assert lib.m3scan_qkrot_bwd(ref, BF16, a, a, a, a, a, a, a, a, a, a, a, a, a + 16, 1 << 30, None) == 4


def test_binding_refuses(lib):
    x = lin_inputs(1, 4, 1, 2, 16, 16, torch.float32)
    args = [x[n] for n in ("q", "k", "v", "log_decay")]
    for call in (lambda: binding.m3scan_linattn_fwd(*args), lambda: binding.m3scan_linattn_bwd(*args, x["d_o"]),
                 lambda: binding.m3scan_linattn_decode(*args, x["state"])):
        with pytest.raises(ValueError):
            call()
    y = rot_inputs(1, 4, 2, 1, 16, 16, torch.float32)
    rest = [y[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")]
    with pytest.raises(ValueError):
        binding.m3scan_qkrot_fwd(*rest)
    with pytest.raises(ValueError):
        binding.m3scan_qkrot_bwd(y["dq_out"], y["dk_out"], *rest)
    with pytest.raises(TypeError):
        binding.m3scan_qkrot_fwd(*[t.half() if i < 2 else t for i, t in enumerate(rest)])


@pytest.mark.parametrize("pos,error", [
    (torch.zeros(2, 5, dtype=torch.int32), TypeError), (torch.zeros(2, 4, dtype=torch.int64), ValueError),
    (torch.zeros(5, 2, dtype=torch.int64).t(), ValueError), (torch.arange(6).as_strided((2, 5), (1, 1)), ValueError),
    (torch.zeros(2, 1, dtype=torch.int64).expand(2, 5), ValueError),
])
def test_positions_refused(pos, error):
    with pytest.raises(error):
        binding._qkrot_positions(pos, 2, 5, -1, torch)


def test_positions_taken():
    t = torch.arange(20).view(2, 10)
    assert binding._qkrot_positions(t, 2, 10, -1, torch) == (t.data_ptr(), 10)
    assert binding._qkrot_positions(t[:, :5], 2, 5, -1, torch) == (t.data_ptr(), 10)
    assert binding._qkrot_positions(t[0], 2, 10, -1, torch) == (t.data_ptr(), 0)
    assert binding._qkrot_positions(t[:1].expand(2, 10), 2, 10, -1, torch) == (t.data_ptr(), 0)
    assert binding._qkrot_positions(None, 2, 10, -1, torch) == (None, 0)


@pytest.mark.parametrize("name", ["m3scan_qkrot_fwd", "m3scan_qkrot_bwd", "m3scan_linattn_fwd", "m3scan_linattn_bwd", "m3scan_linattn_decode"])
def test_calls_run_on_their_tensors_device(name):
    assert getattr(binding, name).__code__ is binding._placed(lambda x: x).__code__


def test_definitions_against_differences():
    """The float64 definitions' autograd gradients against central differences."""
    gen = torch.Generator().manual_seed(0)
    x = {n: v.double() for n, v in lin_inputs(1, 9, 1, 2, 8, 8, torch.float32, seed=3).items()}
    ref = lin_ref_grads(x, 0.3)

    def lin_loss(y):
        o, S = lin_ref(y["q"], y["k"], y["v"], y["log_decay"], y["state"], 0.3)
        return ((o * x["d_o"]).sum() + (S * x["d_state_out"]).sum()).item()

    z = {n: v.double() if v.is_floating_point() else v for n, v in rot_inputs(1, 3, 2, 1, 8, 6, torch.float32, seed=3).items()}
    rref = rot_ref_grads(z, 1e-6, True)

    def rot_loss(y):
        return sum((rot_ref(y[n], y[n + "_weight"], y["positions"], y["inv_freq"], 1e-6, True) * z[f"d{n}_out"]).sum() for n in "qk").item()

    for loss, at, want, names in (
            (lin_loss, x, ref, {"q": "dq", "k": "dk", "v": "dv", "state": "d_state"}),
            (rot_loss, z, rref, {"q": "dq", "k": "dk", "q_weight": "d_q_weight", "k_weight": "d_k_weight"})):
        for n, g in names.items():
            d = torch.randn(at[n].shape, generator=gen, dtype=torch.float64)
            eps = 1e-5
            num = (loss({**at, n: at[n] + eps * d}) - loss({**at, n: at[n] - eps * d})) / (2 * eps)
            ana = (want[g] * d).sum().item()
            assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), n


def test_definition_by_chunks():
    """Whole and short chunks against the recurrence, gradients too; in 64 bits
    both are sums of a few hundred roundings of 2^-53."""
    for T in (64, 130, 9):
        x = lin_inputs(2, T, 2, 4, 16, 24, torch.float32, seed=1)
        a, b = lin_ref_grads(x, 0.3), lin_ref_grads(x, 0.3, lin_ref_chunked)
        assert all(rel(b[n], a[n]) <= 1e-13 for n in a)


def test_linattn_workspace_of_many_heads(lib):
    """With more heads than SMs what a workspace holds for the heads handed on
    does not grow with them: a state of 64 KB per SM and direction, and for the
    backward a copy of d_state."""
    for B, T in ((256, 512), (64, 4096), (1024, 130)):
        st, p = _lin_plan(_lin(batch=B, seq_len=T, k_heads=40, v_heads=40, head_k=128))
        hand = 152 * (64 << 10) + (64 << 10)
        assert st == 0 and p.fwd_workspace_bytes <= hand
        assert p.workspace_bytes <= 2 * hand + B * 40 * 128 * 128 * 4
