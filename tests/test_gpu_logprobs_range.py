"""GPU tests of the token log probabilities over the whole range of their
logits: rows far from zero, and finite values at the type's limits beside
ordinary ones.  Against the definition in 64 bits.

Tolerances (u = 2^-24, L = lse - max y, D = the mean of max y - y under p): the
sums hold exponentials within 2^-22 of exponents within 2 u D, added in trees of
vocab/512 + 16 terms; one rounding of the result, half a unit of its last
place, and for logp one of z - max z, u |logp - L|.  The entropy is a difference
of two such sums, of size up to 1 + log vocab."""
import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu

# rows, vocab: a warp a row, a CTA a row, a row over a cluster of CTAs
FORMS = [(1000, 300), (5, 3000), (2, 20011)]


def _dt(dtype):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def lowest(dtype):
    import torch
    return torch.finfo(_dt(dtype)).min


def run(z, targets, dtype, scale=1.0, top=0):
    """Answers as float64, and the logits as the type holds them."""
    import torch
    rows, vocab = z.shape
    lg = torch.from_numpy(z).to(_dt(dtype)).cuda()
    f32 = dict(device="cuda", dtype=torch.float32)
    out = {k: torch.empty(rows, **f32) for k in ("logp", "lse", "entropy")}
    ids, tl = torch.empty(rows, top, device="cuda", dtype=torch.int32), torch.empty(rows, top, **f32)
    cdg.token_logprobs(lg, torch.from_numpy(targets).cuda(), out["logp"], out["lse"], rows, vocab, dtype, scale=scale,
                       entropy=out["entropy"], top=top, top_ids=ids if top else None, top_logp=tl if top else None)
    res = {k: v.cpu().numpy().astype(np.float64) for k, v in out.items()}
    return dict(res, top_ids=ids.cpu().numpy(), top=tl.cpu().numpy().astype(np.float64), z=lg.double().cpu().numpy())


def definition(z, targets, scale, top):
    y = z * float(np.float32(scale))
    m = y.max(1, keepdims=True)
    with np.errstate(under="ignore"):
        w = np.exp(y - m)
        L = np.log(w.sum(1))
        p = w / w.sum(1, keepdims=True)
        D = (p * (m - y)).sum(1)
    lp = (y - m) - L[:, None]
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top]
    has = (targets >= 0) & (targets < z.shape[1])
    return dict(lse=m[:, 0] + L, L=L, D=D, logp=np.where(has, lp[np.arange(len(z)), np.where(has, targets, 0)], 0.0), ids=ids,
                top=np.take_along_axis(lp, ids, 1), entropy=L + D)


def half_unit(x):
    """Half a unit of the last place of fp32 numbers of x's size."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 24)


def within(got, ref, tol, what):
    with np.errstate(over="ignore"):
        held = ref.astype(np.float32).astype(np.float64)
    far = np.isinf(held)  # past fp32
    assert np.array_equal(got[far], held[far]), what
    worst = np.max(np.abs(got - ref)[~far] / np.broadcast_to(tol, ref.shape)[~far], initial=0.0)
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def check(z, targets, dtype, scale=1.0, top=0, what=("lse", "entropy", "logp", "top")):
    got = run(z, targets, dtype, scale, top)
    ref = definition(got["z"], targets, scale, top)
    u, vocab = 2.0 ** -24, z.shape[1]
    sums = u * (vocab / 512 + 16) + 2.0 ** -22 + 2 * u * ref["D"] + half_unit(ref["L"]) + 2.0 ** -24
    if "lse" in what:
        within(got["lse"], ref["lse"], sums + half_unit(ref["lse"]), "lse")
    if "entropy" in what:
        within(got["entropy"], ref["entropy"], sums * (3 + np.log(vocab)), "entropy")
    if "logp" in what:
        within(got["logp"], ref["logp"], sums + half_unit(ref["logp"]) + 2 * u * (np.abs(ref["logp"]) + ref["L"]), "logp")
    if "top" in what:
        assert np.array_equal(got["top_ids"], ref["ids"])
        within(got["top"], ref["top"], sums[:, None] + half_unit(ref["top"]) + 2 * u * (np.abs(ref["top"]) + ref["L"][:, None]),
               "top_logp")
    return got


@pytest.mark.parametrize("offset", [20.0, 90.0, -500.0, 3000.0])
@pytest.mark.parametrize("rows,vocab", [(2000, 1000), (600, 2000), (8, 30000)])
def test_lse_of_rows_far_from_zero(rows, vocab, offset):
    """lse takes one rounding, whatever the size of the logits."""
    rng = np.random.default_rng(int(abs(offset)))
    z = rng.standard_normal((rows, vocab)) * 1.5 + offset
    t = rng.integers(0, vocab, rows)
    check(z, t, "f32", what=("lse", "entropy"))
    check(z, t, "f32", scale=0.7, what=("lse", "entropy"))


def masked(rng, rows, vocab, value):
    """Ordinary logits with entries at a mask's value: some of each row, and in
    every fifth row all but three; targets masked or not."""
    z = rng.standard_normal((rows, vocab)) * 2.5
    z[rng.random((rows, vocab)) < 0.3] = value
    z[::5, 3:] = value
    z[:, 1] = 0.5
    targets = rng.integers(0, vocab, rows)
    targets[::5] = vocab - 1
    return z, targets


@pytest.mark.parametrize("scale", [1.0, 0.7, 0.3, 1.3])
@pytest.mark.parametrize("dtype,value", [("f32", v) for v in (None, -1e30, -1e20, -1e10, -1e9, -2e7, -1e4)] +
                         [("bf16", v) for v in (None, -1e30, -1e10, -1e9, -1e4)] + [("f16", None), ("f16", -1e4)])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_masks_of_any_value_and_scale(rows, vocab, dtype, value, scale):
    """Masked entries, however large, leave ordinary rows as they are; a row of
    nothing but masks shares its probability among them."""
    z, t = masked(np.random.default_rng(vocab), rows, vocab, lowest(dtype) if value is None else value)
    z[1] = z[0, 4]  # a mask alone
    t[1] = 2
    got = check(z, t, dtype, scale, what=("lse", "entropy"))
    assert abs(got["entropy"][1] - np.log(vocab)) < 1e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [20, 23, 24, 26, 30, 31, 40])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_rows_of_large_logits(rows, vocab, dtype, exponent):
    """Every logit about 2^exponent / log2(e), on either side of zero."""
    rng = np.random.default_rng(exponent)
    size = 2.0 ** exponent / 1.4426950408889634
    z = np.sign(rng.standard_normal((rows, 1))) * size * (1 + 2.0 ** -20 * rng.integers(-8, 9, (rows, vocab)))
    check(z, rng.integers(0, vocab, rows), dtype, what=("lse", "entropy"))


@pytest.mark.parametrize("offset", [20.0, 90.0, -500.0, 3000.0])
@pytest.mark.parametrize("rows,vocab", [(2000, 1000), (600, 2000), (8, 30000)])
def test_logp_of_rows_far_from_zero(rows, vocab, offset):
    rng = np.random.default_rng(int(abs(offset)))
    z = rng.standard_normal((rows, vocab)) * 1.5 + offset
    check(z, rng.integers(0, vocab, rows), "f32", scale=0.7, top=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_the_types_lowest_value_beside_ordinary_logits(rows, vocab, dtype):
    """A masked entry is as improbable as its logit says, not impossible."""
    z, t = masked(np.random.default_rng(vocab), rows, vocab, lowest(dtype))
    got = check(z, t, dtype, top=8)
    assert np.isfinite(got["logp"]).all() and np.isfinite(got["top"]).all()


@pytest.mark.parametrize("rows,vocab", FORMS)
def test_logits_further_apart_than_the_type_reaches(rows, vocab):
    """z - max z passes fp32; scale times it need not."""
    rng = np.random.default_rng(3)
    z = np.where(rng.random((rows, vocab)) < 0.5, 3e38, -3e38)
    z[:, :2] = [3e38, -3e38]
    t = rng.integers(0, vocab, rows)
    t[0] = 1
    for scale in (0.3, 1.0):
        check(z, t, "f32", scale, top=5)


@pytest.mark.parametrize("scale", [1.0, 0.7, 0.3, 1.3])
@pytest.mark.parametrize("dtype,value", [("f32", None), ("f32", -1e30), ("f32", -1e9), ("bf16", None), ("bf16", -1e10), ("f16", None)])
@pytest.mark.parametrize("rows,vocab", FORMS)
def test_logp_of_masked_tokens(rows, vocab, dtype, value, scale):
    """The answers are -inf only where scale times the logit passes fp32."""
    z, t = masked(np.random.default_rng(vocab), rows, vocab, lowest(dtype) if value is None else value)
    z[1] = z[0, 4]  # a mask alone
    t[1] = 2
    got = check(z, t, dtype, scale, top=8)
    assert abs(got["logp"][1] + np.log(vocab)) < 1e-5


@pytest.mark.parametrize("rows,vocab", FORMS)
def test_largest_scales(rows, vocab):
    """scale up to the largest fp32 number: the row's largest logits share the probability."""
    rng = np.random.default_rng(5)
    z = rng.integers(-3, 1, (rows, vocab)).astype(float) * 0.25
    z[:, 0] = 0.0
    t = rng.integers(0, vocab, rows)
    t[0] = 0
    for scale in (1e30, 3e38):
        got = check(z, t, "f32", scale, top=4)
        assert np.abs(got["entropy"] - np.log((z == 0.0).sum(1))).max() < 1e-5


@pytest.mark.parametrize("scale", [1.0, 0.7, 1.25, 1.3])
@pytest.mark.parametrize("dtype,value", [("f32", v) for v in (None, -1e30, -1e20, -1e10, -1e9)] + [("bf16", None), ("bf16", -1e10)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_rows_that_are_all_mask(dtype, value, scale, entropy):
    """lse does not hold such a row's probabilities (one unit of its last place
    is a large number), but the gradient stays that of probabilities in [0, 1]:
    zero where the row's gradients are zero, and else no larger than they are."""
    import torch
    rows, vocab = 6, 1003
    z = np.random.default_rng(1).standard_normal((rows, vocab))
    z[:4] = lowest(dtype) if value is None else value
    lg = torch.from_numpy(z).to(_dt(dtype)).cuda()
    t = torch.tensor([-100, 5, -100, 5, 5, -100], device="cuda")
    g = torch.tensor([0.0, 0.0, 0.5, 0.5, 0.5, 0.5], device="cuda")
    h = torch.tensor([0.0, 0.0, 0.0, 0.25, 0.25, 0.25], device="cuda") if entropy else None
    f32 = dict(device="cuda", dtype=torch.float32)
    logp, lse, H = (torch.empty(rows, **f32) for _ in range(3))
    cdg.token_logprobs(lg, t, logp, lse, rows, vocab, dtype, scale=scale, entropy=H)
    d = torch.empty_like(lg)
    cdg.token_logprobs_grad(lg, t, lse, H if entropy else None, g, h, d, rows, vocab, dtype, scale=scale)
    got = d.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (got[:3] == 0).all()  # no gradient, or no token
    assert np.abs(got[3]).max() <= 1.01 * scale * (0.5 + (0.25 * np.log(vocab) if entropy else 0.0))
    # the ordinary rows beside them
    zz = lg.double().cpu().numpy()[4:] * float(np.float32(scale))
    p = np.exp(zz - lse.double().cpu().numpy()[4:, None])
    ref = -p * np.array([[0.5], [0.0]])
    if entropy:
        ref -= 0.25 * p * (np.log(p) + H.double().cpu().numpy()[4:, None])
    ref[0, 5] += 0.5
    ref *= float(np.float32(scale))
    # p within 2^-20 (4 + max|y|), the result rounded to the type
    unit = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    tol = 2.0 ** -20 * (4 + np.abs(zz).max()) * scale * p * (0.5 + 0.25 * (np.abs(np.log(p)) + np.log(vocab)))
    assert (np.abs(got[4:] - ref) <= tol + unit * 1.001 * np.abs(ref) + 1e-30).all()
