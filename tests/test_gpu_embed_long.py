"""GPU tests of the table gradient for token lists above 262144, whose sort takes
tiles of 4096 keys instead of 1024.  Tolerances as for shorter lists: n values
added in fp32, n 2^-24 of the sum of magnitudes, the scale and one rounding."""
import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count,vocab,dim", [(262144, 1000, 8), (262145, 1000, 8), (300001, 300007, 8), (270000, 1, 8),
                                             (524289, 70, 12), (1000003, 40000, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_a_long_token_list(count, vocab, dim, accumulate):
    import torch
    rng = np.random.default_rng(count + vocab)
    t = rng.integers(-2, vocab + 2, count)
    t[rng.random(count) < 0.3] = vocab // 3
    d = rng.standard_normal((count, dim)).astype(np.float32)
    has = (t >= 0) & (t < vocab)
    n = np.bincount(t[has], minlength=vocab)
    ref = np.stack([np.bincount(t[has], d[has, c].astype(np.float64), minlength=vocab) for c in range(dim)], 1)
    mag = np.stack([np.bincount(t[has], np.abs(d[has, c]).astype(np.float64), minlength=vocab) for c in range(dim)], 1)
    scale = float(np.float32(0.3))
    base = rng.standard_normal((vocab, dim)).astype(np.float32) if accumulate else np.full((vocab, dim), np.nan, np.float32)
    out = torch.from_numpy(base).cuda()
    ws = torch.full((cdg.embed_grad_workspace_bytes(count, vocab, dim) + 256,), 255, dtype=torch.uint8, device="cuda")
    dev, tok = torch.from_numpy(d).cuda(), torch.from_numpy(t).cuda()
    cdg.embed_grad(dev, tok, out, ws[:-256], count, vocab, dim, "f32", scale=scale, accumulate=accumulate)
    got = out.double().cpu().numpy()
    assert (ws[-256:] == 255).all(), "write outside the workspace"
    before = base.astype(np.float64) if accumulate else 0.0
    want = ref * scale + before
    tol = (n[:, None] + 2) * 2.0 ** -24 * (mag * scale + np.abs(before)) + 2.0 ** -24 * np.abs(want) + 2.0 ** -126
    assert (np.abs(got - want) <= tol).all()
    again = torch.from_numpy(base).cuda()
    cdg.embed_grad(dev, tok.int(), again, ws[:-256], count, vocab, dim, "f32", scale=scale, accumulate=accumulate)
    assert torch.equal(again, out), "not the same bits again"
