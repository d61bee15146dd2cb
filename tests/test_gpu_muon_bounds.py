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
