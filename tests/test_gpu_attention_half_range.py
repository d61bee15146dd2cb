"""The gradient in fp16 where probabilities and their gradients are far below
fp16's smallest normal number: many keys, and small gradients of the output."""
import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention import Case, near

pytestmark = pytest.mark.gpu


def check(c, monkeypatch):
    """The reference's bounds with what fp16 keeps of p and ds: steps of 2^-24 of 2^11 p (half a step: 2^-36), and of ds times a
    power of two that brings max |do| max |v| + max |do o| above 2^10 (half a step: 2^-35 of that, which is no more than
    2 max |do| max |v| but for o's rounding), or of ds itself if it is larger."""
    group, dim = c.heads // c.kv_heads, c.dim
    monkeypatch.setitem(ref.TINY, "f16", 0.0)
    rows = slice(int(c.qe[0]), int(c.qe[-1])), slice(int(c.ke[0]), int(c.ke[-1]))
    norm = lambda x, at, h: float(x.cpu().double()[at].view(-1, h, dim).norm(dim=2).max())  # noqa: E731
    step = min(2.0 ** -25, 2 * norm(c.do, rows[0], c.heads) * norm(c.v, rows[1], c.kv_heads) * 1.001 * 2.0 ** -35)
    cols = lambda x, h: x.cpu().double()[:, h * dim:(h + 1) * dim]  # noqa: E731
    for b, (qs, ks) in enumerate(c.parts()):
        for kh in range(c.kv_heads):
            k, v = cols(c.k, kh)[ks], cols(c.v, kh)[ks]
            sums = [torch.zeros_like(k) for _ in range(4)]
            for h in range(kh * group, (kh + 1) * group):
                q, do = cols(c.q, h)[qs], cols(c.do, h)[qs]
                see = ref.visible(q.shape[0], k.shape[0], c.causal, c.window).double()
                (dq, dk, dv), (t_q, t_k, t_v) = ref.gradient(q, k, v, cols(c.o, h)[qs], c.lse.cpu().double()[h, qs], do, c.causal,
                                                            c.window, c.scale, "f16")
                near(cols(c.dq, h)[qs], dq, t_q + c.scale * step * (see @ k.abs()) + 2.0 ** -25, ("dq", b, h))
                for s, x in zip(sums, (dk, dv, t_k + c.scale * step * (see.T @ q.abs()), t_v + 2.0 ** -36 * (see.T @ do.abs()))):
                    s += x
            near(cols(c.dk, kh)[ks], sums[0], sums[2] + 2.0 ** -25, ("dk", b, kh))
            near(cols(c.dv, kh)[ks], sums[1], sums[3] + 2.0 ** -25, ("dv", b, kh))


@pytest.mark.parametrize("q_spread,k_spread", [(2.0 ** -12, 512.0), (512.0, 2.0 ** -12)])
def test_small_gradients_over_many_keys(monkeypatch, q_spread, k_spread):
    c = Case([96], [65536], 1, 1, 64, "f16", causal=False, seed=21, spread=q_spread)
    c.k.mul_(k_spread)
    c.do.mul_(1e-4)
    c.run()
    check(c, monkeypatch)


def test_probabilities_between_two_steps(monkeypatch):
    """Every p is 1 / 414252: 40.5 of fp16's smallest steps."""
    c = Case([5], [414252], 1, 1, 8, "f16", causal=False, seed=22)
    c.q.zero_()
    c.do.abs_()
    c.run()
    check(c, monkeypatch)


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("lens,klens,heads,kv_heads,dim,causal,window", [
    ([200, 1, 500], None, 6, 2, 64, True, 0), ([700], [2600], 2, 1, 128, True, 600), ([90, 40], [60, 300], 2, 2, 40, False, 0)])
def test_sizes_of_the_gradient(monkeypatch, size, lens, klens, heads, kv_heads, dim, causal, window):
    c = Case(lens, klens, heads, kv_heads, dim, "f16", causal, window, seed=23, behind=3)
    c.do.mul_(size)
    c.run()
    check(c, monkeypatch)


def test_nothing_to_scale(monkeypatch):
    for name in ("do", "v"):
        c = Case([100], None, 2, 1, 64, "f16", seed=24)
        getattr(c, name).zero_()
        c.run()
        assert (c.dq == 0).all() and (c.dk == 0).all()
        check(c, monkeypatch)


@pytest.mark.parametrize("bad", [math.nan, math.inf, 6e4])
def test_rows_that_no_sequence_holds_scale_nothing(bad):
    a, b = (Case([130, 77], None, 2, 1, 64, "f16", seed=25, behind=200) for _ in range(2))
    for x in (b.q, b.k, b.v, b.do):
        x[207:] = bad
    for c in (a, b):
        c.do.mul_(1e-4)
        c.run()
    for x, y in zip(a.outputs(), b.outputs()):
        assert torch.equal(x, y)


def test_a_sequence_that_is_not_finite_scales_nothing():
    a, b = (Case([130, 77, 200], None, 2, 1, 64, "f16", seed=26) for _ in range(2))
    for c in (a, b):
        c.do[:130] *= 2  # the largest rows are the first sequence's
        c.v[:130] *= 2
        c.do.mul_(1e-4)
    for x in (b.q, b.k, b.v, b.do):
        x[130:207] = math.nan
        x[150] = math.inf
    a.run()
    b.run()
    rows = torch.ones(407, dtype=torch.bool, device="cuda")
    rows[130:207] = False
    for x, y in zip(a.outputs(), b.outputs()):
        x, y = (x.T, y.T) if x.shape[0] == a.heads else (x, y)
        assert torch.equal(x[rows], y[rows])
