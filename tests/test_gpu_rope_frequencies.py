"""Frequencies that are not finite: their pairs are NaN, as the definition's are, others of the rotated part are NaN or
unchanged, and the rest of the head is unchanged."""
import math

import pytest
import torch

from test_gpu_rope import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 32), (96, 48), (34, 18)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("positions", ["far", None])
def test_frequencies_that_are_not_finite(dtype, dim, rot, interleaved, norm, positions):
    a, b = (Case(9, 3, 2, dim, rot, dtype, norm, interleaved, positions=positions, seed=dim) for _ in range(2))
    at = {1: math.inf, 4: math.nan, rot // 2 - 1: -math.inf}
    for i, f in at.items():
        b.inv_freq[i] = f
    for c in (a, b):
        c.forward()
        c.backward()
    bad = torch.zeros(dim, dtype=torch.bool, device="cuda")
    for i in at:
        bad[[2 * i, 2 * i + 1] if interleaved else [i, i + rot // 2]] = True
    pairs = [*zip(a.y, b.y)] + ([] if norm else [*zip(a.dx, b.dx)])  # (with the norm a NaN of dz reaches its head's dx)
    for x, y in pairs:
        x, y = (m.reshape(9, -1, dim) for m in (x, y))
        assert torch.isnan(y[..., bad]).all()
        assert (torch.isnan(y) | (x == y)).all()
        assert torch.equal(x[..., rot:], y[..., rot:])
