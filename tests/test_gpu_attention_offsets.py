"""Lists of offsets that end in many empty sequences, as a list of fixed length has."""
import pytest
import torch

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before,after", [(0, 20000), (9000, 9000), (3, 40)])
def test_empty_sequences_cost_little(before, after):
    """What the tail costs is the list read once by a CTA and the numbers of CTAs taken over: a few milliseconds at most,
    where a search of the whole list for each of them takes tens."""
    c = Case([0] * before + [1500, 2, 700] + [0] * after, None, 4, 2, 64, "bf16", seed=3)
    c.run()
    c.check(skip={*range(before), *range(before + 3, before + 3 + after)})
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(2):
        ends[0].record()
        c.forward()
        c.backward()
        ends[1].record()
        torch.cuda.synchronize()
    assert c.plan.device_status() == 0
    assert ends[0].elapsed_time(ends[1]) < 10.0
