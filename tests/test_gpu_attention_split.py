"""The kernels that take a part of an item's steps, and those that join the
parts, in every type, with windows, and with rows that no part sees."""
import math

import pytest
import torch

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,klens,heads,kv_heads,dim,causal,window", [
    ([2100], [2400], 2, 1, 128, False, 0),
    ([2500], [2500], 1, 1, 64, True, 0),
    ([2300], [2300], 2, 1, 64, True, 1000),    # a window that ends in other parts for each tile
    ([2300], [2300], 1, 1, 128, True, 1100),
    ([3000], [2100], 1, 1, 64, True, 0),       # the first 900 queries see no key
    ([3000], [2100], 2, 2, 128, True, 950),
    ([2600, 1900], [2050, 2450], 1, 1, 40, True, 0),
])
def test_parts(dtype, lens, klens, heads, kv_heads, dim, causal, window):
    c = Case(lens, klens, heads, kv_heads, dim, dtype, causal, window, seed=dim + window, behind=2)
    # two parts at least of o, and of dq and of dk and dv beside the statistics
    assert c.ws.numel() >= 2 * c.nq * heads * (dim + 1) * 4
    assert c.gws.numel() >= c.nq * heads * 8 + 2 * c.nq * heads * dim * 4 + 2 * 2 * c.nk * kv_heads * dim * 4
    for w in (c.ws, c.gws):
        w.fill_(0xFF)  # NaN: what no part has written reaches nothing
    c.run()
    c.check()
    empty = max(0, lens[0] - klens[0]) if causal else 0
    assert torch.isinf(c.lse[:, :empty]).all() and (c.o[:empty] == 0).all() and (c.dq[:empty] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window", [0, 2000])
def test_one_query_over_many_keys(dtype, window):
    c = Case([1, 3], [5000, 4000], 4, 1, 128, dtype, True, window, seed=2)
    assert c.ws.numel() > 256
    c.ws.fill_(0xFF)
    c.run()
    c.check()
    assert not math.isinf(float(c.lse.min()))
