"""GPU tests of the weight update where its header states a bound or a
guarantee: a zero update whatever eps is, the accuracy of fp32 plans in both
calls, and products whose K is split over clusters of up to eight CTAs.

Bounds: 16-bit plans within 2e-3 of the iteration in exact arithmetic, fp32
plans within 1e-5 (relative, Frobenius), plus the rounding of the output.  A
step's U is itself rounded to fp32 (two roundings of 2^-24, amplified by at most
a^5 = 485 relative to a result of norm sqrt(m): 6e-5/sqrt(m))."""
import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg
from test_gpu_muon import ROUND, guarded, intact, iterate, make, workspace

pytestmark = pytest.mark.gpu

BAR = {"f16": 2e-3, "bf16": 2e-3, "f32": 1e-5}


def _dt(dtype):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def off(got, ref):
    import torch
    return float((torch.linalg.vector_norm(got.double() - ref, dim=(1, 2)) /
                  torch.linalg.vector_norm(ref, dim=(1, 2)).clamp_min(1e-30)).max())


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-25, 1e-7])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(70, 90), (64, 576), (200, 300), (300, 200)])
def test_zero_update_of_any_eps(rows, cols, dtype, eps):
    """A zero U gives a zero O whatever eps is, and leaves the other matrices alone."""
    import torch
    U = make(3, rows, cols, "gauss", 4).to(_dt(dtype))
    U[1] = 0
    p = cdg.muon_plan(rows, cols, batch=3, dtype=dtype, eps=eps)
    O, ws = torch.empty_like(U), workspace(p)
    p.orthogonalize(U, O, ws)
    assert p.device_status() == 0
    assert not O[1].any()
    ref = iterate(U[[0, 2]], eps=eps)
    assert off(O[[0, 2]], ref) <= BAR[dtype] + ROUND[dtype]
    # a weight whose gradient and momentum are zero only decays
    W, M = make(3, rows, cols, "gauss", 5), make(3, rows, cols, "gauss", 6)
    M[1] = 0
    W_out, M_out = torch.empty_like(W), torch.empty_like(M)
    p.step(W, U, M, W_out, M_out, ws, lr=0.1, weight_decay=0.25)
    keep = float(np.float32(1.0 - np.float64(np.float32(0.1)) * 0.25))
    assert torch.equal(W_out[1], W[1] * keep) and not M_out[1].any()
    assert torch.isfinite(W_out).all() and torch.isfinite(M_out).all()


F32_SHAPES = [(3, 64, 576), (1, 128, 128), (2, 130, 257), (1, 511, 513), (1, 300, 1000), (1, 1000, 300), (1, 1100, 1300),
              (1, 200, 4608), (1, 200, 9000), (1, 9000, 200)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("batch,rows,cols", F32_SHAPES)
def test_fp32_step_keeps_fp32_accuracy(batch, rows, cols, kind, nesterov):
    """The update of an fp32 plan's step is as exact as its orthogonalize."""
    import torch
    G, M = make(batch, rows, cols, kind, 20), make(batch, rows, cols, "gauss", 21)
    W = torch.zeros_like(G)
    mu = float(np.float32(0.9))
    m = mu * M.double() + G.double()
    o = iterate(G.double() + mu * m if nesterov else m)
    p = cdg.muon_plan(rows, cols, batch=batch, dtype="f32")
    bw, W_out = guarded(W.shape, torch.float32)
    M_out = torch.empty_like(M)
    p.step(W, G, M, W_out, M_out, workspace(p), lr=1.0, momentum=0.9, nesterov=nesterov)
    torch.cuda.synchronize()
    assert p.device_status() == 0 and intact(bw)
    assert off(-W_out, o) <= BAR["f32"] + 6e-5 / min(rows, cols) ** 0.5 + 2.0 ** -24


def test_fp32_plans_say_how_they_run():
    """No fp32 plan takes the Gram form, whose error exceeds its bound."""
    small, wide = cdg.muon_plan_host(64, 576, dtype="f32").info(), cdg.muon_plan_host(300, 576, dtype="f32").info()
    assert small["gram"] == 0 and small["launches"] == wide["launches"] == 17
    assert cdg.muon_plan_host(64, 576, dtype="bf16").info()["gram"] == 1


def spectrum(kind, rows, cols, seed):
    """U with the singular values of `kind` between random orthonormal bases."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n = min(rows, cols), max(rows, cols)
    q = torch.linalg.qr(torch.randn(n, m, generator=g, device="cuda", dtype=torch.float64))[0]
    p = torch.linalg.qr(torch.randn(m, m, generator=g, device="cuda", dtype=torch.float64))[0]
    i = torch.arange(m, device="cuda", dtype=torch.float64)
    s = {"flat": torch.ones_like(i), "few": torch.where(i < max(1, m // 8), 1.0, 0.02), "decay": 1.0 / (i + 1) ** 2,
         "wide": 10.0 ** (-4.0 * i / max(1, m - 1))}[kind]
    u = (p * s) @ q.mT
    return (u if rows <= cols else u.mT).float()[None].contiguous()


@pytest.mark.parametrize("kind", ["flat", "few", "decay", "wide"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(64, 576), (128, 128), (256, 256), (512, 512), (511, 513), (512, 2048), (1100, 1300),
                                       (200, 4608), (200, 9000), (9000, 200)])
def test_orthogonalize_is_within_its_stated_bound(rows, cols, dtype, kind):
    """Spectra other than random matrices'; rows of up to 512 with long K split it
    over two, four and eight CTAs of a cluster, in one-part and in three-part products."""
    import torch
    U = spectrum(kind, rows, cols, rows).to(_dt(dtype))
    p = cdg.muon_plan(rows, cols, dtype=dtype)
    ws = workspace(p)
    buf, O = guarded(U.shape, U.dtype)
    p.orthogonalize(U, O, ws)
    torch.cuda.synchronize()
    assert p.device_status() == 0 and intact(buf)
    assert off(O, iterate(U)) <= BAR[dtype] + ROUND[dtype]
    again = torch.empty_like(U)
    ws.fill_(255)
    p.orthogonalize(U, again, ws)
    assert torch.equal(again, O), "not the same bits again"


@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("batch,rows,cols", F32_SHAPES)
def test_fp32_orthogonalize_on_all_paths(batch, rows, cols, kind):
    import torch
    U = make(batch, rows, cols, kind, 22)
    p = cdg.muon_plan(rows, cols, batch=batch, dtype="f32")
    O = torch.empty_like(U)
    p.orthogonalize(U, O, workspace(p))
    assert off(O, iterate(U)) <= BAR["f32"]
