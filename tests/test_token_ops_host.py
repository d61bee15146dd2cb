"""Refusals of the token operators and the weight update: every argument that
the C ABI or the binding checks, without a device (nothing is launched)."""
import ctypes
import math

import pytest

import implicit_gemm_dgrad_gb300 as cdg

INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, NO_DEVICE = 1, 2, 3, 4, 7
P = [1 << 24 << i for i in range(1, 14)]  # far-apart 16-byte aligned addresses


def status(fn, *args, **kw):
    with pytest.raises(cdg.CdgError) as e:
        fn(*args, **kw)
    return e.value.status


def logprobs(**kw):
    a = dict(logits=P[0], targets=P[1], logp=P[2], lse=P[3], rows=4, vocab=100, dtype="bf16", scale=1.0, entropy=P[4],
             top=2, top_ids=P[5], top_logp=P[6])
    a.update(kw)
    return status(cdg.token_logprobs, **a)


@pytest.mark.parametrize("change,expect", [
    (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(dtype=3), INVALID), (dict(ld=99), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(top=33), INVALID), (dict(top=-1), INVALID),
    (dict(vocab=1, top=2), INVALID), (dict(logits=None), INVALID), (dict(targets=None), INVALID),
    (dict(logp=None), INVALID), (dict(top_ids=None), INVALID), (dict(top_logp=None), INVALID),
    (dict(top=0), INVALID), (dict(rows=1 << 30), UNSUPPORTED), (dict(logits=P[0] + 1), ALIGNMENT),
    (dict(logits=P[0] + 2, dtype="f32"), ALIGNMENT), (dict(targets=P[1] + 4), ALIGNMENT),
    (dict(lse=P[3] + 2), ALIGNMENT), (dict(lse=P[2] + 8), ALIAS), (dict(entropy=P[0] + 4), ALIAS),
    (dict(logp=P[1]), ALIAS), (dict(top_ids=P[6]), ALIAS),
    (dict(targets=None, logp=None, lse=None, entropy=None, top=0, top_ids=None, top_logp=None), INVALID)])
def test_logprobs_refusals(change, expect):
    assert logprobs(**change) == expect


def test_no_rows_or_tokens_is_no_error():
    cdg.token_logprobs(P[0], P[1], P[2], P[3], 0, 100)
    cdg.token_logprobs_grad(P[0], P[1], P[2], None, P[3], None, P[4], 0, 100)
    cdg.embed(P[0], P[1], P[2], 0, 10, 16)


@pytest.mark.parametrize("change,expect", [
    (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(dtype=7), INVALID), (dict(ld=9), INVALID),
    (dict(ld_d=9), INVALID), (dict(scale=-2.0), INVALID), (dict(targets=None), INVALID), (dict(lse=None), INVALID),
    (dict(g_logp=None), INVALID), (dict(entropy=None), INVALID), (dict(dlogits=None), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(dlogits=P[6] + 1), ALIGNMENT), (dict(g_logp=P[4] + 1), ALIGNMENT),
    (dict(dlogits=P[0] + 32), ALIAS), (dict(dlogits=P[0], ld_d=101), ALIAS), (dict(dlogits=P[2]), ALIAS)])
def test_logprobs_grad_refusals(change, expect):
    a = dict(logits=P[0], targets=P[1], lse=P[2], entropy=P[3], g_logp=P[4], g_entropy=P[5], dlogits=P[6], rows=4,
             vocab=100, dtype="bf16")
    a.update(change)
    assert status(cdg.token_logprobs_grad, **a) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(count=-1), INVALID), (dict(vocab=0), INVALID), (dict(dim=0), INVALID), (dict(dtype=3), INVALID),
    (dict(ld_table=15), INVALID), (dict(ld_out=15), INVALID), (dict(scale=math.nan), INVALID), (dict(table=None), INVALID),
    (dict(tokens=None), INVALID), (dict(out=None), INVALID), (dict(count=1 << 31), UNSUPPORTED),
    (dict(table=P[0] + 1), ALIGNMENT), (dict(tokens=P[1] + 4), ALIGNMENT), (dict(out=P[0] + 64), ALIAS),
    (dict(out=P[1]), ALIAS)])
def test_embed_refusals(change, expect):
    a = dict(table=P[0], tokens=P[1], out=P[2], count=4, vocab=10, dim=16, dtype="f16")
    a.update(change)
    assert status(cdg.embed, **a) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(count=-1), INVALID), (dict(count=1 << 30), INVALID), (dict(vocab=0), INVALID), (dict(dim=0), INVALID),
    (dict(dtype=3), INVALID), (dict(ld_dout=15), INVALID), (dict(ld_dtable=15), INVALID), (dict(scale=math.inf), INVALID),
    (dict(dout=None), INVALID), (dict(tokens=None), INVALID), (dict(dtable=None), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace=P[3] + 8), ALIGNMENT), (dict(dtable=P[2] + 2, out_f32=True), ALIGNMENT),
    (dict(dtable=P[0]), ALIAS), (dict(workspace=P[2] + 16), ALIAS), (dict(workspace=P[1]), ALIAS)])
def test_embed_grad_refusals(change, expect):
    a = dict(dout=P[0], tokens=P[1], dtable=P[2], workspace=P[3], count=4, vocab=10, dim=16, dtype="bf16")
    a.update(change)
    assert status(cdg.embed_grad, **a) == expect


def test_embed_grad_workspace():
    with pytest.raises(cdg.CdgError):
        cdg.embed_grad_workspace_bytes(-1, 10, 16)
    sizes = [cdg.embed_grad_workspace_bytes(n, 1000, 64) for n in (0, 1, 100, 5000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] >= 16 and sizes[-1] >= 2 * 4 * 100000


def test_out_of_range_index_width():
    lib = cdg.load_library()
    assert lib.cdg_embed(P[0], 16, P[1], 2, 4, 10, 16, 0, 1.0, P[2], 16, None) == INVALID
    assert lib.cdg_token_logprobs(P[0], 100, P[1], 1, 4, 100, 0, 1.0, 0, P[2], None, None, None, None, None) == INVALID


@pytest.mark.parametrize("change,expect", [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(batch=0), INVALID), (dict(dtype=3), INVALID),
    (dict(steps=0), INVALID), (dict(steps=33), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.nan), INVALID),
    (dict(coefficients=(math.inf, 0, 0)), INVALID), (dict(coefficients=(9.0, 0.0, 0.0)), INVALID),
    (dict(coefficients=(3.0, 5.0, 0.0)), INVALID), (dict(batch=65536), UNSUPPORTED),
    (dict(rows=32769, cols=40000), UNSUPPORTED), (dict(cols=(1 << 21) + 1), UNSUPPORTED)])
def test_muon_plan_refusals(change, expect):
    a = dict(rows=64, cols=576)
    a.update(change)
    assert status(cdg.muon_plan_host, **a) == expect


def test_muon_plan_shapes():
    wide, tall = cdg.muon_plan_host(64, 576, batch=3), cdg.muon_plan_host(576, 64, batch=3)
    assert (wide.info()["m"], wide.info()["n"], wide.info()["transposed"]) == (64, 576, 0)
    assert (tall.info()["m"], tall.info()["n"], tall.info()["transposed"]) == (64, 576, 1)
    assert wide.workspace_bytes == tall.workspace_bytes > 0
    assert status(wide.orthogonalize, P[0], P[1], P[2]) == NO_DEVICE
    assert status(wide.step, P[0], P[1], P[2], P[3], P[4], P[5], lr=0.1) == NO_DEVICE
    assert status(wide.orthogonalize, None, P[1], P[2]) == INVALID
    assert status(wide.step, P[0], P[1], P[2], P[3], P[4], P[5], lr=math.nan) == INVALID
    assert cdg.load_library().cdg_muon_device_status(wide.handle, None) == NO_DEVICE
    assert cdg.load_library().cdg_muon_plan_host(1, 8, 8, 0, 5, 1.5, -0.5, 0.0, 1e-7, 148, None) == INVALID
    h = ctypes.c_void_p(1)
    assert cdg.load_library().cdg_muon_plan_host(0, 8, 8, 0, 5, 1.5, -0.5, 0.0, 1e-7, 148, ctypes.byref(h)) == INVALID
    assert not h.value


class FakeCuda:
    """Stands in for a dense CUDA tensor: size, element size and an aligned address."""
    is_cuda = True

    def __init__(self, n, esize, floating=True):
        self.n, self.esize, self.floating = n, esize, floating

    def numel(self):
        return self.n

    def element_size(self):
        return self.esize

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.floating

    def data_ptr(self):
        return 1 << 24


def test_binding_checks_sizes_and_types():
    t = FakeCuda(4, 8, floating=False)
    f = lambda n: FakeCuda(n, 4)  # noqa: E731
    with pytest.raises(ValueError, match="logits"):
        cdg.token_logprobs(FakeCuda(399, 2), t, f(4), None, 4, 100)
    with pytest.raises(ValueError, match="logits"):
        cdg.token_logprobs(FakeCuda(400, 4), t, f(4), None, 4, 100)       # fp32 elements for bf16
    with pytest.raises(ValueError, match="targets"):
        cdg.token_logprobs(FakeCuda(400, 2), FakeCuda(3, 8, False), f(4), None, 4, 100)
    with pytest.raises(ValueError, match="int32 or int64"):
        cdg.token_logprobs(FakeCuda(400, 2), FakeCuda(4, 8), f(4), None, 4, 100)
    with pytest.raises(ValueError, match="logp"):
        cdg.token_logprobs(FakeCuda(400, 2), t, f(3), None, 4, 100)
    with pytest.raises(ValueError, match="top_ids"):
        cdg.token_logprobs(FakeCuda(400, 2), t, f(4), None, 4, 100, top=2, top_ids=FakeCuda(7, 4, False), top_logp=f(8))
    with pytest.raises(ValueError, match="dlogits"):
        cdg.token_logprobs_grad(FakeCuda(400, 2), t, f(4), None, f(4), None, FakeCuda(399, 2), 4, 100)
    with pytest.raises(ValueError, match="table"):
        cdg.embed(FakeCuda(159, 2), t, FakeCuda(64, 2), 4, 10, 16)
    with pytest.raises(ValueError, match="workspace"):
        cdg.embed_grad(FakeCuda(64, 2), t, FakeCuda(160, 2), FakeCuda(15, 1), 4, 10, 16)
    with pytest.raises(ValueError, match="dtable"):
        cdg.embed_grad(FakeCuda(64, 2), t, FakeCuda(160, 2), FakeCuda(1 << 20, 1), 4, 10, 16, out_f32=True)
    p = cdg.muon_plan_host(8, 16)
    with pytest.raises(ValueError, match="U"):
        p.orthogonalize(FakeCuda(127, 2), FakeCuda(128, 2), FakeCuda(1 << 20, 1))
    with pytest.raises(ValueError, match="workspace"):
        p.orthogonalize(FakeCuda(128, 2), FakeCuda(128, 2), FakeCuda(15, 1))
    with pytest.raises(ValueError, match="M_out"):
        p.step(f(128), FakeCuda(128, 2), f(128), f(128), f(127), FakeCuda(1 << 20, 1), lr=0.1)


def test_binding_rejects_cpu_and_strided_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros(4, 100)
    with pytest.raises(ValueError, match="CUDA"):
        cdg.token_logprobs(z, P[1], P[2], None, 4, 100, "f32")
    with pytest.raises(ValueError, match="column stride"):
        cdg.token_logprobs(torch.zeros(100, 4).t(), P[1], P[2], None, 4, 100, "f32")
    with pytest.raises(ValueError, match="call needs"):
        cdg.token_logprobs(torch.zeros(4, 120)[:, :101], P[1], P[2], None, 4, 100, "f32")
    with pytest.raises(ValueError, match="overlapping rows"):
        cdg.token_logprobs(torch.zeros(4, 100).as_strided((4, 100), (0, 1)), P[1], P[2], None, 4, 100, "f32")
