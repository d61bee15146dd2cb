"""Refusals of the attention and of the rotation of queries and keys, their
sizes and frequencies, without a device (nothing is launched), and the 64-bit
reference against differences and automatic differentiation."""
import ctypes
import math

import pytest
import torch

import attention_reference as ref
import implicit_gemm_dgrad_gb300 as cdg

INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, NO_DEVICE = 1, 2, 3, 4, 7
P = [1 << 26 << i for i in range(1, 20)]  # far-apart aligned addresses


def status(fn, *args, **kw):
    with pytest.raises(cdg.CdgError) as e:
        fn(*args, **kw)
    return e.value.status


@pytest.mark.parametrize("change,expect", [
    (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(heads=6, kv_heads=4), INVALID), (dict(dim=0), INVALID),
    (dict(dtype=3), INVALID), (dict(window=-1), INVALID), (dict(causal=False, window=5), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(dtype="f32"), UNSUPPORTED), (dict(dim=12), UNSUPPORTED),
    (dict(dim=136), UNSUPPORTED), (dict(heads=2048, kv_heads=2048), UNSUPPORTED)])
def test_plan_refusals(change, expect):
    a = dict(heads=4, kv_heads=2, dim=64)
    a.update(change)
    assert status(cdg.attention_plan_host, **a) == expect


def test_plan_without_a_place_for_it():
    assert cdg.load_library().cdg_attention_plan_host(4, 2, 64, 1, 1, 0, 0.1, None) == INVALID
    h = ctypes.c_void_p(1)
    assert cdg.load_library().cdg_attention_plan_host(4, 3, 64, 1, 1, 0, 0.1, ctypes.byref(h)) == INVALID
    assert not h.value
    cdg.load_library().cdg_attention_destroy(None)


def attend(**kw):
    a = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], workspace=P[5], q_tokens=100, k_tokens=200, q_offsets=P[6],
             k_offsets=P[7], sequences=3)
    a.update(kw)
    return status(cdg.attention_plan_host(4, 2, 64).attend, **a)


COMMON = [
    (dict(), NO_DEVICE), (dict(q_tokens=-1), INVALID), (dict(k_tokens=1 << 30), INVALID), (dict(sequences=0), INVALID),
    (dict(sequences=(1 << 20) + 1), INVALID), (dict(q_offsets=None), INVALID), (dict(k_offsets=None), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(workspace=None), INVALID), (dict(ld_q=255), INVALID), (dict(ld_k=127), INVALID),
    (dict(ld_q=260), ALIGNMENT), (dict(ld_v=1 << 31), UNSUPPORTED), (dict(q=P[0] + 8), ALIGNMENT),
    (dict(v=P[2] + 2), ALIGNMENT), (dict(lse=P[4] + 2), ALIGNMENT), (dict(workspace=P[5] + 128), ALIGNMENT),
    (dict(q_offsets=P[6] + 4), ALIGNMENT), (dict(q_offsets=None, k_offsets=None, sequences=1), NO_DEVICE),
    # q, k and v side by side in one buffer
    (dict(q=P[0], k=P[0] + 512, v=P[0] + 768, ld_q=512, ld_k=512, ld_v=512, k_tokens=100), NO_DEVICE)]


@pytest.mark.parametrize("change,expect", COMMON + [
    (dict(o=P[0]), ALIAS), (dict(o=P[1] + 1024), ALIAS), (dict(lse=P[3]), ALIAS), (dict(workspace=P[2]), ALIAS),
    (dict(o=P[6] - 16), ALIAS), (dict(workspace=P[4]), ALIAS),
    # o beside q in its rows, and over it
    (dict(q=P[0], o=P[0] + 512, ld_q=512, ld_o=512), NO_DEVICE), (dict(q=P[0], o=P[0] + 256, ld_q=512, ld_o=512), ALIAS)])
def test_attend_refusals(change, expect):
    assert attend(**change) == expect


@pytest.mark.parametrize("change,expect", COMMON + [
    (dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(ld_do=255), INVALID), (dict(ld_dk=120), INVALID), (dict(dv=P[11] + 4), ALIGNMENT), (dict(dq=P[0]), ALIAS),
    (dict(dk=P[1]), ALIAS), (dict(dv=P[10]), ALIAS), (dict(dq=P[8]), ALIAS), (dict(dk=P[3] + 32), ALIAS),
    (dict(workspace=P[9]), ALIAS), (dict(dv=P[4]), ALIAS), (dict(dq=P[7]), ALIAS),
    (dict(dq=P[9], dk=P[9] + 512, dv=P[9] + 768, ld_dq=512, ld_dk=512, ld_dv=512, k_tokens=100), NO_DEVICE)])
def test_attend_grad_refusals(change, expect):
    a = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], workspace=P[5], q_tokens=100, k_tokens=200, q_offsets=P[6],
             k_offsets=P[7], sequences=3, do=P[8], dq=P[9], dk=P[10], dv=P[11])
    a.update(change)
    assert status(cdg.attention_plan_host(4, 2, 64).attend_grad, **a) == expect


def test_workspaces():
    p = cdg.attention_plan_host(8, 2, 128)
    assert p.workspace_bytes(0, 0, 1) >= 16 and p.grad_workspace_bytes(0, 0, 1) >= 16
    # enough items for every SM: no parts; one short query against many keys: parts
    assert p.workspace_bytes(8192, 8192, 1) == 256 < p.workspace_bytes(1, 8192, 1)
    assert p.grad_workspace_bytes(100, 100, 4) >= 100 * 8 * 8
    for sizes in ((-1, 5, 1), (5, -1, 1), (5, 5, 0), (1 << 30, 5, 1)):
        assert status(p.workspace_bytes, *sizes) == INVALID
        assert status(p.grad_workspace_bytes, *sizes) == INVALID
    assert cdg.load_library().cdg_attention_device_status(p.handle, None) == NO_DEVICE


def rope(**kw):
    a = dict(q=P[0], k=P[1], positions=P[2], inv_freq=P[3], q_out=P[4], k_out=P[5], tokens=10, heads=4, kv_heads=2,
             dim=64, norm=True, w_q=P[6], w_k=P[7])
    a.update(kw)
    return status(cdg.qk_rope, **a)


ROPE = [
    (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(heads=0, kv_heads=0), INVALID), (dict(dim=0), INVALID),
    (dict(dtype=5), INVALID), (dict(rot=65), INVALID), (dict(rot=7), INVALID), (dict(rot=-2), INVALID),
    (dict(factor=math.nan), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID),
    (dict(inv_freq=None), INVALID), (dict(norm=False), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(ld_q=255), INVALID), (dict(ld_k=100), INVALID), (dict(dim=258), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(heads=70000), UNSUPPORTED), (dict(ld_q=1 << 31), UNSUPPORTED), (dict(q=P[0] + 1), ALIGNMENT), (dict(positions=P[2] + 4), ALIGNMENT),
    (dict(inv_freq=P[3] + 2), ALIGNMENT), (dict(w_q=P[6] + 1), ALIGNMENT)]


@pytest.mark.parametrize("change,expect", ROPE + [
    (dict(q_out=None), INVALID), (dict(k_out=None), INVALID), (dict(q_out=P[0] + 2), ALIAS), (dict(q_out=P[1]), ALIAS),
    (dict(k_out=P[4]), ALIAS), (dict(q_out=P[0], ld_qo=512), ALIAS), (dict(q_out=P[2]), ALIAS), (dict(k_out=P[6]), ALIAS)])
def test_rope_refusals(change, expect):
    assert rope(**change) == expect


@pytest.mark.parametrize("change,expect", ROPE + [
    (dict(dq_out=None), INVALID), (dict(dk=None), INVALID), (dict(workspace=None), INVALID),
    (dict(norm=False, w_q=None, w_k=None), INVALID), (dict(workspace=P[12] + 8), ALIGNMENT), (dict(dw_q=P[13] + 2), ALIGNMENT),
    (dict(dq=P[0]), ALIAS), (dict(dq=P[8] + 2), ALIAS), (dict(dk=P[8]), ALIAS), (dict(dk=P[10]), ALIAS),
    (dict(workspace=P[1]), ALIAS), (dict(dw_q=P[14]), ALIAS), (dict(dw_k=P[12]), ALIAS), (dict(dq=P[3]), ALIAS)])
def test_rope_grad_refusals(change, expect):
    a = dict(q=P[0], k=P[1], positions=P[2], inv_freq=P[3], tokens=10, heads=4, kv_heads=2, dim=64, norm=True, w_q=P[6],
             w_k=P[7], dq_out=P[8], dk_out=P[9], dq=P[10], dk=P[11], workspace=P[12], dw_q=P[13], dw_k=P[14])
    a.update(change)
    assert status(cdg.qk_rope_grad, **a) == expect


def test_no_tokens_is_no_error():
    cdg.qk_rope(P[0], P[1], P[2], P[3], P[4], P[5], 0, 4, 2, 64)
    cdg.qk_rope(P[0], None, None, P[3], P[4], None, 0, 4, 0, 64)
    for sizes in ((-1, 4, 2, 64), (10, 0, 0, 64), (10, 4, 2, 300)):
        assert status(cdg.qk_rope_grad_workspace_bytes, *sizes) == INVALID


class Cuda:
    """Stands in for a CUDA tensor that says its type."""
    is_cuda, dtype = True, "torch.float32"

    def __init__(self, n):
        self.n = n

    def numel(self):
        return self.n

    def element_size(self):
        return 4

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return True


def test_tensors_of_other_types_and_sizes_are_refused():
    p = cdg.attention_plan_host(4, 2, 64)
    args = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], workspace=P[5], q_tokens=10, k_tokens=10)
    with pytest.raises(ValueError):
        p.attend(**dict(args, q=Cuda(10 * 256)))  # fp32 where bf16 is needed
    with pytest.raises(ValueError):
        p.attend(**dict(args, lse=Cuda(39)))
    with pytest.raises(ValueError):
        p.attend(**dict(args, q_offsets=Cuda(2)))
    with pytest.raises(ValueError):
        cdg.qk_rope(P[0], P[1], P[2], Cuda(31), P[4], P[5], 10, 4, 2, 64)
    with pytest.raises(ValueError):
        p.attend(**dict(args, q=torch.zeros(10, 256, dtype=torch.bfloat16)))  # not on a GPU
    with pytest.raises(ValueError):
        p.attend(**dict(args, q_offsets=torch.tensor([0, 10]), k_offsets=torch.tensor([0, 10], dtype=torch.int32)))


def test_frequencies():
    assert cdg.rope_frequencies(0) == []
    plain = cdg.rope_frequencies(64, base=500.0)
    for i, f in enumerate(plain):
        assert abs(f - 500.0 ** (-2 * i / 64)) <= 2.0 ** -24 * f
    assert cdg.rope_frequencies(64, base=500.0, stretch=4.0) == pytest.approx([f / 4 for f in plain], rel=2.0 ** -23)
    got = cdg.rope_frequencies(64, base=500.0, stretch=4.0, trained=1000, low=2.0, high=20.0)
    for f, g in zip(plain, got):
        turns = 1000 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 2) / 18))
        assert g == pytest.approx(f * (keep + (1 - keep) / 4), rel=1e-6)
    for bad in (dict(rot=3), dict(rot=-2), dict(base=0.0), dict(stretch=0.0), dict(trained=-1), dict(trained=5, low=3.0, high=3.0),
                dict(base=math.inf), dict(rot=258)):
        assert status(cdg.rope_frequencies, **dict(dict(rot=64), **bad)) == INVALID


@pytest.mark.parametrize("n,m,causal,window", [(5, 7, False, 0), (6, 6, True, 0), (7, 4, True, 0), (6, 9, True, 3)])
def test_reference_gradient_against_differences(n, m, causal, window):
    g = torch.Generator().manual_seed(n * 10 + m)
    q, k, v, do = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((n, 8), (m, 8), (m, 8), (n, 8)))
    f = lambda *a: (ref.forward(*a, causal, window, 0.4, "f32")[0] * do).sum()  # noqa: E731
    o, lse, _, _ = ref.forward(q, k, v, causal, window, 0.4, "f32")
    grads, _ = ref.gradient(q, k, v, o, lse, do, causal, window, 0.4, "f32")
    for i, got in enumerate(grads):
        for at in ((0, 0), (got.shape[0] // 2, 3), (got.shape[0] - 1, 7)):
            ends = []
            for h in (1e-5, -1e-5):
                args = [q.clone(), k.clone(), v.clone()]
                args[i][at] += h
                ends.append(f(*args))
            assert abs((ends[0] - ends[1]) / 2e-5 - got[at]) < 1e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_keeps_lengths_and_relative_positions(interleaved):
    g = torch.Generator().manual_seed(1)
    x, y = torch.randn(2, 1, 1, 32, generator=g, dtype=torch.float64)
    f = torch.tensor(cdg.rope_frequencies(32))
    turn = lambda z, p: ref.rotate(z, torch.tensor([p]), f, 32, interleaved, 1.0, False, 0.0, None)  # noqa: E731
    assert torch.allclose(turn(x, 7).norm(), x.norm())
    assert torch.allclose((turn(x, 7) * turn(y, 3)).sum(), (turn(x, 104) * turn(y, 100)).sum(), rtol=1e-9)
