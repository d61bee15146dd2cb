"""Windows that hide nothing, up to the largest number, give the bits of no window."""
import pytest
import torch

import implicit_gemm_dgrad_gb300 as cdg
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,klens", [([300], [300]), ([300], [5]), ([5], [300]), ([130, 0, 257], [7, 64, 600]), ([1], [3000])])
@pytest.mark.parametrize("window", [None, (1 << 30) - 1, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 1, 1 << 70])
def test_a_window_past_every_key_hides_nothing(lens, klens, window):
    """None: one number more than the keys."""
    plain, far = (Case(lens, klens, 2, 1, 64, "bf16", window=w, seed=5) for w in (0, sum(klens) + 1 if window is None else window))
    plain.run()
    far.run()
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), plain.outputs(), far.outputs()):
        assert torch.equal(a, b), name
    plain.check()


def test_the_widest_window_that_hides_a_key():
    for window in (299, 300):
        c = Case([300], None, 2, 1, 64, "bf16", window=window, seed=6)
        c.run()
        c.check()
