"""One work item that takes longer than a wait inside an item may."""
import math

import pytest
import torch

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu


def test_an_item_of_seconds():
    """A query of each of 152 heads over 2^30 - 200 keys: the warps of an item's second tile, which has no rows, wait for all
    of it.  Keys and values are zeros, in one tensor of 17 GB: lse is the log of their number, o is 0."""
    keys, heads = (1 << 30) - 200, 152
    plan = cdg.attention_plan(heads, 1, 8, "bf16", causal=False)
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    q = torch.randn(1, heads * 8, device="cuda").to(torch.bfloat16)
    kv = torch.zeros(keys, 8, device="cuda", dtype=torch.bfloat16)
    o, lse = torch.full_like(q, 7.0), torch.full((heads, 1), 7.0, device="cuda")
    ws = torch.empty(plan.workspace_bytes(1, keys), device="cuda", dtype=torch.uint8)
    plan.attend(q, kv, kv, o, lse, ws, 1, keys)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert (o == 0).all()
    # the sum of ones is exact but for the last step's; the log and its scaling take a few roundings of 30 log(2)
    assert (lse.cpu().double() - math.log(keys)).abs().max() <= 8 * 2.0 ** -24 * 31
