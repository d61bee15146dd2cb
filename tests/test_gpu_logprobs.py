"""GPU tests of the token log probabilities and their gradient against the
definitions in 64 bits.

Tolerances, from the arithmetic (u32 = 2^-24, y = scale * logits):
  * lse, logp, top_logp: y and its reference are rounded products (2 u32 |y|),
    the exponential is within 2^-22, a thread adds up to vocab/128 terms before
    the joins: |err| <= 2^-21 (8 + max|y|) + u32 (vocab/128 + 64);
  * entropy = log s - e/s with |e/s| <= log vocab + max|y| of the terms that count:
    the same, times (1 + log vocab);
  * gradient: p is within 2^-20 (4 + max|y|) relative, the result is rounded once to
    the logits' type.
"""
import math

import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu

HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}
GUARD = 64


def _dt(dtype):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def definition(z, targets, scale, top):
    """64-bit lse, logp, entropy, ids and log probabilities of numpy float64
    logits; scale as the call takes it, an fp32 number."""
    y = z * float(np.float32(scale))
    m = y.max(1, keepdims=True)
    ms = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = (ms + np.log(np.exp(y - ms).sum(1, keepdims=True)))[:, 0]
        lp = y - lse[:, None]
        lp[np.isneginf(lse)] = -np.inf
        p = np.exp(lp)
        entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(1)
    has = (targets >= 0) & (targets < z.shape[1])
    logp = np.where(has, lp[np.arange(len(z)), np.where(has, targets, 0)], 0.0)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top]
    return dict(lse=lse, logp=logp, entropy=entropy, lp=lp, p=p, ids=ids, top=np.take_along_axis(lp, ids, 1), has=has)


def forward(z, targets, dtype, scale=1.0, top=0, pad=0, offset=0, index=None):
    """Runs token_logprobs on logits inside a wider buffer (row stride vocab +
    pad, first row at element `offset`), outputs in guarded buffers."""
    import torch
    rows, vocab = z.shape
    ld = vocab + pad
    buf = torch.full((offset + rows * ld + 16,), 1e4, dtype=torch.float32, device="cuda").to(_dt(dtype))
    lg = buf[offset:offset + rows * ld].view(rows, ld)[:, :vocab]
    lg.copy_(torch.from_numpy(z))
    tg = torch.from_numpy(targets).cuda().to(index or torch.int64)
    outs = {}

    def guarded(n, dt):
        t = torch.full((n + 2 * GUARD,), -77, dtype=dt, device="cuda")
        return t, t[GUARD:GUARD + n]

    full = {k: guarded(n, dt) for k, n, dt in (("logp", rows, torch.float32), ("lse", rows, torch.float32),
                                               ("entropy", rows, torch.float32),
                                               ("top_ids", rows * top, torch.int32),
                                               ("top_logp", rows * top, torch.float32))}
    outs = {k: v[1] for k, v in full.items()}
    cdg.token_logprobs(lg, tg, outs["logp"], outs["lse"], rows, vocab, dtype, scale=scale, entropy=outs["entropy"],
                       top=top, top_ids=outs["top_ids"] if top else None, top_logp=outs["top_logp"] if top else None)
    torch.cuda.synchronize()
    for k, (whole, _) in full.items():
        g = whole.cpu().numpy()
        assert (g[:GUARD] == -77).all() and (g[-GUARD:] == -77).all(), f"write outside {k}"
    res = {k: v.cpu().numpy().astype(np.float64 if v.dtype == torch.float32 else np.int64) for k, v in outs.items()}
    res["top_ids"] = res["top_ids"].reshape(rows, top)
    res["top_logp"] = res["top_logp"].reshape(rows, top)
    res["z"] = lg.double().cpu().numpy()
    return res


def close(got, ref, tol, what):
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), what
    f = np.isfinite(ref)
    assert np.array_equal(got[~f & ~np.isnan(ref)], ref[~f & ~np.isnan(ref)]), what
    if f.any():
        t = np.broadcast_to(tol, ref.shape)
        worst = np.max(np.abs(got - ref)[f] / t[f])
        assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def check(z, targets, dtype, **kw):
    scale, top = kw.get("scale", 1.0), kw.get("top", 0)
    got = forward(z, targets, dtype, **kw)
    ref = definition(got["z"], targets, scale, top)
    y = got["z"] * scale
    big = np.max(np.abs(y[np.isfinite(y)])) if np.isfinite(y).any() else 0.0
    vocab = z.shape[1]
    tol = 2.0 ** -21 * (8 + big) + 2.0 ** -24 * (vocab / 128 + 64)
    close(got["lse"], ref["lse"], tol, "lse")
    close(got["logp"], ref["logp"], tol, "logp")
    close(got["entropy"], ref["entropy"], tol * (1 + math.log(vocab)), "entropy")
    assert np.array_equal(got["top_ids"], ref["ids"])
    close(got["top_logp"], ref["top"], tol, "top_logp")
    return got


def draw(rng, rows, vocab, banned=0.0, spread=2.5):
    z = rng.standard_normal((rows, vocab)) * spread
    targets = rng.integers(0, vocab, rows)
    if banned:
        z[rng.random((rows, vocab)) < banned] = -np.inf
    targets[rng.random(rows) < 0.2] = -100
    return z, targets


# rows, vocab, top, pad, offset: row starts at every alignment, vocabularies below
# a vector, about a CTA's reach (128 and 512 threads), split rows
SHAPES = [(1, 1, 1, 0, 0), (3, 2, 2, 1, 1), (5, 7, 5, 2, 3), (2, 31, 20, 0, 5), (17, 33, 32, 7, 0), (4, 256, 8, 1, 7),
          (9, 1000, 5, 0, 0), (3, 1029, 32, 3, 2), (2, 8192, 20, 1, 1), (2, 8193, 20, 0, 1), (1, 20011, 8, 0, 3),
          (1, 131072, 20, 0, 0), (40, 32003, 4, 5, 6), (300, 9001, 1, 0, 0), (200, 50021, 0, 1, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,top,pad,offset", SHAPES)
def test_matches_definition(rows, vocab, top, pad, offset, dtype):
    rng = np.random.default_rng(rows * 7919 + vocab)
    z, t = draw(rng, rows, vocab)
    check(z, t, dtype, top=top, pad=pad, offset=offset)


@pytest.mark.parametrize("scale", [1e-3, 0.7, 1.25, 40.0])
@pytest.mark.parametrize("rows,vocab", [(2, 777), (3, 30000)])
def test_scale(rows, vocab, scale):
    z, t = draw(np.random.default_rng(3), rows, vocab)
    check(z, t, "bf16", scale=scale, top=6)


def test_int32_targets_and_large_values():
    import torch
    z, t = draw(np.random.default_rng(4), 5, 4099)
    check(z, t, "f32", top=3, index=torch.int32)
    check(z * 1e4, t, "f32", top=3)      # a single token has all the probability
    check(z - 3e4, t, "f16", top=3)      # all far below zero
    check(np.where(z > 0, 6e4, -6e4), t, "f16", top=32)


@pytest.mark.parametrize("vocab", [5, 200, 9000, 70001])
@pytest.mark.parametrize("banned", [0.001, 0.5, 0.999])
def test_banned_tokens(vocab, banned):
    z, t = draw(np.random.default_rng(vocab), 6, vocab, banned)
    z[0] = -np.inf                       # a row whose mask leaves nothing
    z[1, 1:] = -np.inf                   # one token left
    z[1, 0] = -3.0
    z[2] = np.finfo(np.float32).min if vocab % 2 else -np.inf  # the type's lowest value
    t[:3] = [0, 0, vocab - 1]
    got = check(z, t, "f32", top=min(vocab, 20))
    assert got["lse"][0] == -np.inf and got["entropy"][0] == 0.0 and got["logp"][0] == -np.inf
    assert list(got["top_ids"][0]) == list(range(min(vocab, 20)))
    assert abs(got["logp"][1]) < 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 300), (2, 5000), (3, 12000), (1, 100003)])
def test_equal_logits_go_to_the_lowest_number(rows, vocab, dtype):
    rng = np.random.default_rng(vocab)
    t = rng.integers(0, vocab, rows)
    check(np.zeros((rows, vocab)), t, dtype, top=32)                                    # all equal
    check(rng.integers(0, 3, (rows, vocab)).astype(float), t, dtype, top=32)            # three values
    check(np.where(rng.random((rows, vocab)) < 0.002, 1.0, -0.0), t, dtype, top=32)     # few above, then ties
    check(np.round(rng.standard_normal((rows, vocab)) * 4) / 4, t, dtype, top=20)
    check(np.tile(np.arange(vocab)[None] / vocab, (rows, 1)), t, "f32", top=32)         # ascending
    check(np.tile(-np.arange(vocab)[None] / vocab, (rows, 1)), t, "f32", top=32)        # descending


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("vocab,at", [(50, 3), (9001, 9000), (40000, 12345)])
def test_rows_with_nan_or_infinity_answer_nan(vocab, at, bad):
    z, t = draw(np.random.default_rng(5), 3, vocab)
    t[:] = 1
    z[1, at] = bad
    got = forward(z, t, "f32", top=4)
    for k in ("lse", "logp", "entropy"):
        assert np.isnan(got[k][1]) and np.isfinite(got[k][[0, 2]]).all()
    assert np.isnan(got["top_logp"][1]).all() and (got["top_ids"][1] == -1).all()
    ref = definition(z[[0, 2]].astype(np.float32).astype(float), t[[0, 2]], 1.0, 4)
    assert np.array_equal(got["top_ids"][[0, 2]], ref["ids"])


def test_outputs_are_optional_and_repeat():
    import torch
    z = torch.randn(7, 20000, device="cuda")
    t = torch.randint(0, 20000, (7,), device="cuda")
    full = [torch.empty(7, device="cuda") for _ in range(3)]
    cdg.token_logprobs(z, t, full[0], full[1], 7, 20000, "f32", entropy=full[2])
    one = torch.empty(7, device="cuda")
    cdg.token_logprobs(z, t, one, None, 7, 20000, "f32")
    assert torch.equal(one, full[0])
    cdg.token_logprobs(z, None, None, one, 7, 20000, "f32")
    assert torch.equal(one, full[1])
    again = [torch.empty(7, device="cuda") for _ in range(3)]
    cdg.token_logprobs(z, t, again[0], again[1], 7, 20000, "f32", entropy=again[2])
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    cdg.token_logprobs(z[:0], t[:0], one[:0], None, 0, 20000, "f32")  # no rows


def test_another_stream():
    import torch
    s = torch.cuda.Stream()
    z = torch.randn(64, 50000, device="cuda")
    t = torch.randint(0, 50000, (64,), device="cuda")
    a, b = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    cdg.token_logprobs(z, t, a, None, 64, 50000, "f32")
    s.wait_stream(torch.cuda.current_stream())
    cdg.token_logprobs(z, t, b, None, 64, 50000, "f32", stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_row_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32 (fp32, row stride 2^27 + 3): the last row answers as alone."""
    import torch
    ld, vocab, rows = (1 << 27) + 3, 1003, 10
    buf = torch.empty(ld * (rows - 1) + vocab, device="cuda")
    z = torch.as_strided(buf, (rows, vocab), (ld, 1))
    z.copy_(torch.randn(rows, vocab, device="cuda"))
    t = torch.arange(rows, device="cuda")
    a, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    cdg.token_logprobs(z, t, a, lse, rows, vocab, "f32")
    ref = torch.log_softmax(z.double(), 1)[torch.arange(rows), t]
    assert torch.allclose(a.double(), ref, atol=1e-5, rtol=0)
    g = torch.ones(rows, device="cuda")
    cdg.token_logprobs_grad(z, t, lse, None, g, None, z, rows, vocab, "f32")
    assert abs(float(z.sum())) < 1e-2 and float(z[rows - 1, rows - 1]) > 0.5


# ---------------------------------------------------------------- gradient


def grad_definition(z, targets, lse, entropy, g, h, scale):
    scale = float(np.float32(scale))
    y = z * scale
    with np.errstate(invalid="ignore"):
        lp = y - lse[:, None]
    lp[np.isneginf(lse)] = -np.inf
    p = np.exp(lp)
    has = (targets >= 0) & (targets < z.shape[1]) & np.isfinite(lse)
    ge = np.where(has, g, 0.0)[:, None]
    inner = np.where(p > 0, np.where(p > 0, lp, 0.0) + entropy[:, None], 0.0)
    d = -ge * p - h[:, None] * p * inner
    d[np.arange(len(z)), np.where(has, targets, 0)] += ge[:, 0]
    size = p * (np.abs(ge) + np.abs(h[:, None]) * (np.abs(inner)))
    return scale * d, scale * size


def grad_case(z, targets, dtype, scale=1.0, with_entropy=True, pads=(0, 0), offsets=(0, 0), in_place=False):
    import torch
    rows, vocab = z.shape
    rng = np.random.default_rng(11)
    g, h = rng.standard_normal(rows), 0.3 * rng.standard_normal(rows) if with_entropy else np.zeros(rows)
    f = forward(z, targets, dtype, scale=scale)
    dt = _dt(dtype)

    def wide(pad, offset):
        ld = vocab + pad
        buf = torch.full((offset + rows * ld + GUARD,), -77.0, device="cuda").to(dt)
        return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :vocab]

    _, lg = wide(pads[0], offsets[0])
    lg.copy_(torch.from_numpy(f["z"]))
    buf, out = wide(pads[1], offsets[1])
    if in_place:
        out.copy_(lg)
        lg = out
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda()  # noqa: E731
    g32, h32, lse, ent = (np.asarray(a, dtype=np.float32) for a in (g, h, f["lse"], f["entropy"]))
    cdg.token_logprobs_grad(lg, torch.from_numpy(targets).cuda(), dev(lse), dev(ent) if with_entropy else None, dev(g32),
                            dev(h32) if with_entropy else None, out, rows, vocab, dtype, scale=scale)
    torch.cuda.synchronize()
    whole = buf.float().cpu().numpy()
    mask = np.ones(len(whole), bool)
    ld = vocab + pads[1]
    for r in range(rows):
        mask[offsets[1] + r * ld: offsets[1] + r * ld + vocab] = False
    assert (whole[mask] == -77).all(), "write outside dlogits"
    got = out.double().cpu().numpy()
    ref, size = grad_definition(f["z"], targets, lse.astype(float), ent.astype(float), g32.astype(float),
                                h32.astype(float), scale)
    y = f["z"] * scale
    big = np.max(np.abs(y[np.isfinite(y)])) if np.isfinite(y).any() else 0.0
    tol = size * 2.0 ** -20 * (4 + big) + HALF_ULP[dtype] * np.abs(ref) * 1.001 + 2 * TINY[dtype]
    close(got, ref, tol + 1e-300, "dlogits")
    return got


GRAD_SHAPES = [(1, 1, 0, 0, 0, 0), (3, 5, 1, 2, 1, 0), (7, 33, 0, 0, 3, 3), (2, 1000, 0, 0, 0, 0), (5, 1001, 0, 0, 0, 0),
               (3, 1001, 2, 2, 5, 5), (2, 4099, 1, 0, 2, 1), (3, 8200, 0, 0, 0, 0), (2, 20011, 0, 3, 0, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,pad,pad_d,off,off_d", GRAD_SHAPES)
def test_gradient_matches_formula(rows, vocab, pad, pad_d, off, off_d, dtype):
    z, t = draw(np.random.default_rng(vocab), rows, vocab)
    grad_case(z, t, dtype, scale=1.3, pads=(pad, pad_d), offsets=(off, off_d))
    grad_case(z, t, dtype, with_entropy=False, pads=(pad, pad_d), offsets=(off, off_d))
    grad_case(z, t, dtype, pads=(pad, pad), offsets=(off, off), in_place=True)


def test_gradient_of_masked_rows():
    z, t = draw(np.random.default_rng(8), 5, 3001, banned=0.4)
    z[0] = -np.inf
    z[1, 1:] = -np.inf
    z[1, 0] = 2.0
    t[:2] = [7, 0]
    got = grad_case(z, t, "f32")
    assert (got[0] == 0).all() and np.abs(got[1]).max() < 1e-5
    assert (got[:, :][np.isneginf(z) & (np.arange(3001)[None] != t[:, None])] == 0).all()


def test_gradient_matches_differences():
    """<dlogits, v> against central differences of the 64-bit definition."""
    import torch
    rng = np.random.default_rng(9)
    rows, vocab, scale = 4, 211, 0.8
    z, t = draw(rng, rows, vocab, spread=1.5)
    z = z.astype(np.float32).astype(np.float64)
    g, h = rng.standard_normal(rows), rng.standard_normal(rows)

    def value(a):
        d = definition(a, t, scale, 0)
        return float((g * d["logp"] + h * d["entropy"]).sum())

    f = forward(z, t, "f32", scale=scale)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda()  # noqa: E731
    out = torch.empty(rows, vocab, device="cuda")
    cdg.token_logprobs_grad(dev(z), torch.from_numpy(t).cuda(), dev(f["lse"]), dev(f["entropy"]), dev(g), dev(h), out,
                            rows, vocab, "f32", scale=scale)
    d = out.double().cpu().numpy()
    for _ in range(8):
        v = rng.standard_normal((rows, vocab))
        eps = 1e-4
        diff = (value(z + eps * v) - value(z - eps * v)) / (2 * eps)
        # differences: O(eps^2) third derivatives; the gradient: fp32 throughout
        assert abs(diff - float((d * v).sum())) <= 1e-5 * (1 + abs(diff)) + 1e-5 * np.abs(d * v).sum()


# many rows of a small vocabulary: a warp takes a row
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab,top,pad,offset", [(1, 1, 0, 0), (7, 7, 1, 3), (33, 32, 0, 1), (256, 20, 0, 0),
                                                  (1001, 5, 2, 5), (4096, 32, 0, 0)])
def test_many_rows_of_a_small_vocabulary(vocab, top, pad, offset, dtype):
    rng = np.random.default_rng(vocab)
    rows = 1003
    z, t = draw(rng, rows, vocab, banned=0.05 if vocab > 7 else 0.0)
    z[5] = -np.inf                                              # nothing left
    z[6] = 0.0                                                  # all equal
    z[7] = np.round(z[7] * 2) / 2                               # many equal
    z[8] = np.where(np.arange(vocab) < vocab // 2, -np.inf, 1.0)
    t[5:9] = [0, vocab - 1, 0, vocab - 1]
    check(z, t, dtype, top=top, pad=pad, offset=offset)
    check(z, t, dtype, pad=pad, offset=offset)


def test_many_rows_with_the_types_lowest_value_and_nan():
    rng = np.random.default_rng(21)
    z, t = draw(rng, 1000, 300)
    t[:] = 3
    z[11] = np.finfo(np.float32).min
    check(z, t, "f32", top=4)
    z[12, 7], z[13, 9] = np.nan, np.inf
    got = forward(z, t, "f32", top=4)
    bad = np.isnan(got["lse"])
    assert list(np.flatnonzero(bad)) == [12, 13] and (got["top_ids"][[12, 13]] == -1).all()
    assert np.isnan(got["logp"][[12, 13]]).all() and np.isfinite(got["logp"][~bad]).all()
