"""GPU tests of the orthogonalised weight update against the iteration in 64
bits.

Tolerance: the products take fp16 operands (2^-12 relative each); a 64-bit
simulation of what is rounded where, over Gaussian, low-rank and decaying
spectra of 64 to 1024 rows, is within 9e-4 of the exact iteration (relative,
Frobenius).  The bar is twice that, plus the rounding of the output."""
import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu

BAR = 1.8e-3
ROUND = {"f16": 2.0 ** -12, "bf16": 2.0 ** -9, "f32": 2.0 ** -24}
A, B, C = cdg.MUON_COEFFICIENTS
GUARD = 256


def _dt(dtype):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def iterate(u, steps=5, eps=1e-7, coefficients=(A, B, C)):
    import torch
    a, b, c = coefficients
    x = u.double()
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + eps)
    for _ in range(steps):
        if x.shape[1] > x.shape[2]:
            g = x.mT @ x
            x = a * x + x @ (b * g + c * g @ g)
        else:
            g = x @ x.mT
            x = a * x + (b * g + c * g @ g) @ x
    return x


def make(batch, rows, cols, kind, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randn(batch, rows, cols, generator=g, device="cuda")
    if kind == "gauss":
        return n
    r = max(1, min(rows, cols) // 8)
    low = torch.randn(batch, rows, r, generator=g, device="cuda") @ torch.randn(batch, r, cols, generator=g, device="cuda")
    return 0.05 * n + low / r ** 0.5


def guarded(shape, dt):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), -77.0, device="cuda").to(dt)
    return buf, buf[GUARD:GUARD + n].view(*shape)


def intact(buf):
    return bool((buf[:GUARD] == -77).all() and (buf[-GUARD:] == -77).all())


def workspace(p):
    import torch
    return torch.full((p.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")


def assert_near(got, ref, dtype, what=""):
    import torch
    err = torch.linalg.vector_norm(got.double() - ref, dim=(1, 2))
    size = torch.linalg.vector_norm(ref, dim=(1, 2))
    worst = float((err / size.clamp_min(1e-30)).max())
    assert worst <= BAR + ROUND[dtype], f"{what}: {worst:.3g}"


SHAPES = [(1, 1, 1), (2, 1, 9), (1, 9, 1), (3, 5, 7), (1, 16, 16), (2, 33, 20), (3, 64, 576), (1, 100, 64), (2, 127, 129),
          (1, 128, 128), (2, 130, 257), (1, 256, 64), (1, 300, 1000), (1, 1000, 300), (1, 511, 513), (2, 640, 640),
          (1, 17, 4608), (1, 1100, 1300)]


@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_orthogonalize(batch, rows, cols, dtype, kind):
    import torch
    U = make(batch, rows, cols, kind, rows + cols).to(_dt(dtype))
    p = cdg.muon_plan(rows, cols, batch=batch, dtype=dtype)
    ws = workspace(p)
    buf, O = guarded(U.shape, U.dtype)
    p.orthogonalize(U, O, ws)
    torch.cuda.synchronize()
    assert p.device_status() == 0
    assert intact(buf), "write outside O"
    assert_near(O, iterate(U), dtype, p.info())
    again = torch.empty_like(U)
    p.orthogonalize(U, again, ws)
    assert torch.equal(again, O), "not the same bits again"


@pytest.mark.parametrize("dtype,size", [("bf16", 1e-12), ("bf16", 1e12), ("f32", 1e-6), ("f32", 1e15), ("f16", 1e-3), ("f16", 1e3)])
def test_size_of_the_update(dtype, size):
    """X is scaled by a power of two first: very small and very large updates keep their digits."""
    import torch
    U = (make(1, 96, 200, "gauss", 1) * size).to(_dt(dtype))
    p = cdg.muon_plan(96, 200, dtype=dtype, eps=0.0)
    O = torch.empty_like(U)
    p.orthogonalize(U, O, workspace(p))
    assert_near(O, iterate(U, eps=0.0), dtype)


@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("batch,rows,cols", [(2, 5, 7), (1, 64, 576), (1, 300, 1000), (1, 640, 512)])
def test_fp32_update_keeps_fp32_accuracy(batch, rows, cols, kind):
    """fp32 plans take every operand as two fp16 parts (22 bits): the simulated
    iteration is then within 2e-6 of the exact one, an fp32 one within 1e-5.
    The bar is the latter."""
    import torch
    U = make(batch, rows, cols, kind, 10)
    p = cdg.muon_plan(rows, cols, batch=batch, dtype="f32")
    O = torch.empty_like(U)
    p.orthogonalize(U, O, workspace(p))
    ref = iterate(U)
    err = torch.linalg.vector_norm(O.double() - ref, dim=(1, 2)) / torch.linalg.vector_norm(ref, dim=(1, 2))
    assert float(err.max()) <= 1e-5, err


def test_steps_and_coefficients():
    import torch
    U = make(1, 200, 96, "gauss", 2)
    for steps, co in ((1, (A, B, C)), (2, (2.0, -1.5, 0.5)), (8, (1.875, -1.25, 0.375)), (5, (1.5, -0.5, 0.0))):
        p = cdg.muon_plan(200, 96, dtype="f32", steps=steps, coefficients=co)
        O = torch.empty_like(U)
        p.orthogonalize(U, O, workspace(p))
        assert_near(O, iterate(U, steps, coefficients=co), "f32", (steps, co))
    # a convergent map: the result's rows or columns are orthonormal (a random U's small singular
    # values need more steps than these, so the test takes a well-conditioned one)
    q = (torch.linalg.qr(make(1, 200, 96, "gauss", 3).double())[0].float() * 3.0).contiguous()
    p = cdg.muon_plan(200, 96, dtype="f32", steps=16, coefficients=(1.875, -1.25, 0.375))
    O = torch.empty_like(q)
    p.orthogonalize(q, O, workspace(p))
    assert float((O[0].double() - q[0].double() / 3.0).abs().max()) < 2e-3


def test_zero_and_non_finite_updates_stay_in_their_matrix():
    import torch
    U = make(4, 70, 90, "gauss", 4).bfloat16()
    U[0] = 0
    U[1, 3, 5] = float("nan")
    U[2, 69, 89] = float("inf")
    p = cdg.muon_plan(70, 90, batch=4, dtype="bf16")
    O = torch.empty_like(U)
    p.orthogonalize(U, O, workspace(p))
    assert not O[0].any() and torch.isnan(O[1]).all() and torch.isnan(O[2]).all()
    assert_near(O[3:], iterate(U[3:]), "bf16")


def test_single_element_and_rank_one():
    import torch
    U = torch.zeros(1, 40, 60, device="cuda")
    U[0, 7, 11] = -1e-3  # all of the norm in one element
    p = cdg.muon_plan(40, 60, dtype="f32")
    O = torch.empty_like(U)
    p.orthogonalize(U, O, workspace(p))
    assert_near(O, iterate(U), "f32")


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (2, 37, 21), (1, 64, 576), (1, 200, 130), (2, 130, 200)])
def test_step(batch, rows, cols, dtype, nesterov):
    """W_out's update is within the bar of the exact one; M_out is elementwise fp32."""
    import torch
    G = make(batch, rows, cols, "gauss", 5).to(_dt(dtype))
    M = make(batch, rows, cols, "lowrank", 6)
    W = make(batch, rows, cols, "gauss", 7)
    lr, mu, wd, sc = 0.02, 0.9, 0.1, 1.7
    m = mu * M.double() + G.double()
    o = iterate(G.double() + mu * m if nesterov else m)
    p = cdg.muon_plan(rows, cols, batch=batch, dtype=dtype)
    ws = workspace(p)
    bw, W_out = guarded(W.shape, torch.float32)
    bm, M_out = guarded(W.shape, torch.float32)
    p.step(W, G, M, W_out, M_out, ws, lr=lr, momentum=mu, weight_decay=wd, update_scale=sc, nesterov=nesterov)
    torch.cuda.synchronize()
    assert p.device_status() == 0 and intact(bw) and intact(bm)
    assert bool(((M_out.double() - m).abs() <= 2.0 ** -23 * (mu * M.double().abs() + G.double().abs()) + 1e-30).all())
    update = (W.double() * (1 - lr * wd) - W_out.double()) / (lr * sc)
    err = torch.linalg.vector_norm(update - o, dim=(1, 2)) / torch.linalg.vector_norm(o, dim=(1, 2))
    # W_out's own rounding, seen through the division by lr * update_scale
    seen = torch.linalg.vector_norm(W.double(), dim=(1, 2)) * 2.0 ** -22 / (lr * sc) / torch.linalg.vector_norm(o, dim=(1, 2))
    assert bool((err <= BAR + seen).all()), (err, seen)
    Wi, Mi = W.clone(), M.clone()  # in place
    p.step(Wi, G, Mi, Wi, Mi, ws, lr=lr, momentum=mu, weight_decay=wd, update_scale=sc, nesterov=nesterov)
    assert torch.equal(Wi, W_out) and torch.equal(Mi, M_out)


def test_plans_workspaces_and_streams():
    """Two plans, one workspace each, on two streams; one plan moved to another workspace."""
    import torch
    U1, U2 = make(1, 90, 300, "gauss", 8).bfloat16(), make(1, 300, 90, "gauss", 9).bfloat16()
    p1, p2 = cdg.muon_plan(90, 300), cdg.muon_plan(300, 90)
    O1, O2, O3 = torch.empty_like(U1), torch.empty_like(U2), torch.empty_like(U1)
    w1, w2, w3 = workspace(p1), workspace(p2), workspace(p1)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    p1.orthogonalize(U1, O1, w1, stream=s1)
    p2.orthogonalize(U2, O2, w2, stream=s2)
    p1.orthogonalize(U1, O3, w3, stream=s1)
    torch.cuda.synchronize()
    assert_near(O1, iterate(U1), "bf16")
    assert_near(O2, iterate(U2), "bf16")
    assert torch.equal(O1, O3)


@pytest.mark.parametrize("coefficients,steps,gram", [((A, B, C), 5, 1), ((A, B, C), 8, 0), ((1.875, -1.25, 0.375), 8, 1)])
@pytest.mark.parametrize("rows,cols", [(48, 700), (128, 128), (90, 31)])
def test_small_matrices_on_both_paths(rows, cols, coefficients, steps, gram):
    """Up to 128 rows the steps run on X X^T where the amplification of small
    singular values stays within 1000 (a^5 = 485; a^8 = 19818 does not), else on X."""
    import torch
    p = cdg.muon_plan(rows, cols, batch=2, dtype="bf16", steps=steps, coefficients=coefficients)
    assert p.info()["gram"] == gram
    for kind in ("gauss", "lowrank"):
        U = make(2, rows, cols, kind, 12).bfloat16()
        O = torch.empty_like(U)
        p.orthogonalize(U, O, workspace(p))
        torch.cuda.synchronize()
        assert p.device_status() == 0
        assert_near(O, iterate(U, steps, coefficients=coefficients), "bf16", kind)


@pytest.mark.parametrize("batch,rows,cols", [(1, 2100, 2300), (1, 2300, 2101), (6, 700, 801), (1, 200, 4608), (1, 4608, 333)])
def test_large_and_long_matrices(batch, rows, cols):
    """Products in CTA pairs, alone and mixed with single CTAs, with partial tiles on both sides; K split over clusters."""
    import torch
    for kind in ("gauss", "lowrank"):
        U = make(batch, rows, cols, kind, 14).bfloat16()
        p = cdg.muon_plan(rows, cols, batch=batch)
        ws = workspace(p)
        buf, O = guarded(U.shape, U.dtype)
        p.orthogonalize(U, O, ws)
        torch.cuda.synchronize()
        assert p.device_status() == 0 and intact(buf)
        assert_near(O, iterate(U), "bf16", kind)
        again = torch.empty_like(U)
        p.orthogonalize(U, again, ws)
        assert torch.equal(again, O), "not the same bits again"


def test_large_step_in_place():
    import torch
    rows, cols = 2100, 2200
    G, M, W = make(1, rows, cols, "gauss", 15).bfloat16(), make(1, rows, cols, "lowrank", 16), make(1, rows, cols, "gauss", 17)
    lr, mu = 0.02, 0.9
    m = mu * M.double() + G.double()
    o = iterate(G.double() + mu * m)
    p = cdg.muon_plan(rows, cols)
    Wi, Mi = W.clone(), M.clone()
    p.step(Wi, G, Mi, Wi, Mi, workspace(p), lr=lr, momentum=mu)
    torch.cuda.synchronize()
    assert p.device_status() == 0
    update = (W.double() - Wi.double()) / lr
    err = float(torch.linalg.vector_norm(update - o) / torch.linalg.vector_norm(o))
    seen = float(torch.linalg.vector_norm(W.double()) * 2.0 ** -22 / lr / torch.linalg.vector_norm(o))
    assert err <= BAR + seen, (err, seen)
    assert bool(((Mi.double() - m).abs() <= 2.0 ** -23 * (mu * M.double().abs() + G.double().abs()) + 1e-30).all())
