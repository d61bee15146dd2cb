"""The norms with eps = 0: rows that are not zero have finite results and
weights' gradients, at numbers of heads that leave lanes without one."""
import pytest

import test_gpu_rope as rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 2), (9, 3), (17, 1), (8, 4)])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 32), (40, 40), (256, 64), (33, 6)])
def test_zero_eps(monkeypatch, dtype, heads, kv_heads, dim, rot):
    monkeypatch.setattr(rope, "EPS", 0.0)
    c = rope.Case(21, heads, kv_heads, dim, rot, dtype, seed=heads + dim)
    c.forward()
    c.backward()
    c.check()
