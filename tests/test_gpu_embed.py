"""GPU tests of the embedding lookup and its gradient against 64-bit
definitions.  The lookup is one fp32 product, rounded once: half a unit of the
type.  The gradient adds n values in fp32: n 2^-24 of the sum of magnitudes,
then the scale and one rounding."""
import numpy as np
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu

HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "f32": 2.0 ** -126}
SENTINEL = -77.0


def _dt(dtype):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def wide(rows, cols, pad, offset, dt):
    """A rows x cols view of row stride cols + pad inside a sentinel-filled buffer."""
    import torch
    buf = torch.full((offset + rows * (cols + pad) + 64,), SENTINEL, device="cuda").to(dt)
    return buf, buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def untouched(buf, view, rows, cols, pad, offset):
    whole = buf.double().cpu().numpy().copy()
    for r in range(rows):
        whole[offset + r * (cols + pad): offset + r * (cols + pad) + cols] = SENTINEL
    return (whole == SENTINEL).all()


def tokens(rng, count, vocab, hot=0.3):
    t = rng.integers(-2, vocab + 2, count)  # some name no token
    t[rng.random(count) < hot] = vocab // 3  # one token very often
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("count,vocab,dim,pad,off", [(1, 1, 1, 0, 0), (5, 7, 3, 1, 1), (9, 11, 8, 0, 0), (4, 300, 64, 0, 0),
                                                     (70, 50, 129, 3, 2), (33, 20, 1000, 0, 0), (3, 9, 4096, 8, 8),
                                                     (2, 5, 9001, 0, 3), (3000, 100, 24, 0, 0), (40000, 64, 40, 0, 0)])
def test_lookup(count, vocab, dim, pad, off, dtype):
    import torch
    rng = np.random.default_rng(count + dim)
    dt = _dt(dtype)
    t = tokens(rng, count, vocab)
    _, table = wide(vocab, dim, pad, off, dt)
    table.copy_(torch.from_numpy(rng.standard_normal((vocab, dim))))
    buf, out = wide(count, dim, pad, off, dt)
    for index, scale in ((torch.int64, 1.0), (torch.int32, 1.7)):
        cdg.embed(table, torch.from_numpy(t).cuda().to(index), out, count, vocab, dim, dtype, scale=scale)
        torch.cuda.synchronize()
        has = (t >= 0) & (t < vocab)
        ref = np.where(has[:, None], table.double().cpu().numpy()[np.where(has, t, 0)] * np.float32(scale), 0.0)
        got = out.double().cpu().numpy()
        assert (np.abs(got - ref) <= HALF_ULP[dtype] * 1.001 * np.abs(ref) + TINY[dtype]).all()
        assert untouched(buf, out, count, dim, pad, off), "write outside out"


# counts about the sort's tile (4096) and below, one token's run longer than any
# part, vocabularies of one, of one digit and of two and three digits of the sort
GRAD = [(1, 1, 1, 0, 0), (7, 5, 3, 1, 1), (100, 1, 16, 0, 0), (300, 40, 129, 3, 2), (2048, 1000, 72, 0, 0),
        (4095, 700, 8, 0, 0), (4096, 511, 8, 0, 0), (4097, 512, 10, 0, 0), (20000, 5000, 33, 0, 1), (9000, 300000, 8, 0, 0),
        (64, 10, 5001, 0, 0), (5000, 37, 1024, 8, 8), (70000, 100, 16, 0, 0)]


@pytest.mark.parametrize("dtype,out_f32", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True), ("f32", False)])
@pytest.mark.parametrize("count,vocab,dim,pad,off", GRAD)
def test_gradient(count, vocab, dim, pad, off, dtype, out_f32):
    import torch
    rng = np.random.default_rng(count + vocab)
    t = tokens(rng, count, vocab)
    odt = "f32" if out_f32 else dtype
    _, dout = wide(count, dim, pad, off, _dt(dtype))
    dout.copy_(torch.from_numpy(rng.standard_normal((count, dim))))
    d64 = dout.double().cpu().numpy()
    has = (t >= 0) & (t < vocab)
    ref, mag, n = np.zeros((vocab, dim)), np.zeros((vocab, dim)), np.bincount(t[has], minlength=vocab)
    np.add.at(ref, t[has], d64[has])
    np.add.at(mag, t[has], np.abs(d64[has]))
    scale = np.float32(0.3)
    ws = torch.full((cdg.embed_grad_workspace_bytes(count, vocab, dim),), 255, dtype=torch.uint8, device="cuda")
    tok = torch.from_numpy(t).cuda()
    buf, out = wide(vocab, dim, pad, off, _dt(odt))
    base = np.random.default_rng(1).standard_normal((vocab, dim)).astype(np.float32)
    for accumulate in (False, True):
        if accumulate:
            out.copy_(torch.from_numpy(base))
        before = out.double().cpu().numpy()
        cdg.embed_grad(dout, tok, out, ws, count, vocab, dim, dtype, scale=float(scale), out_f32=out_f32,
                       accumulate=accumulate)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        want = ref * scale + (before if accumulate else 0.0)
        tol = (n[:, None] + 2) * 2.0 ** -24 * (mag * scale + (np.abs(before) if accumulate else 0.0))
        tol = tol + HALF_ULP[odt] * 1.001 * np.abs(want) + TINY[odt]
        assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))
        if accumulate:
            assert np.array_equal(got[n == 0], before[n == 0])
        else:
            assert (got[n == 0] == 0).all()
            first = got
        assert untouched(buf, out, vocab, dim, pad, off), "write outside dtable"
    cdg.embed_grad(dout, tok.to(torch.int32), out, ws, count, vocab, dim, dtype, scale=float(scale), out_f32=out_f32)
    assert np.array_equal(out.double().cpu().numpy(), first), "not the same bits again"


def test_gradient_is_the_adjoint_of_the_lookup():
    """<embed(E), d> = <E, embed_grad(d)> (both linear), to fp32 rounding."""
    import torch
    count, vocab, dim = 500, 91, 48
    g = torch.Generator(device="cuda").manual_seed(3)
    E = torch.randn(vocab, dim, generator=g, device="cuda")
    d = torch.randn(count, dim, generator=g, device="cuda")
    t = torch.randint(-1, vocab, (count,), generator=g, device="cuda")
    out, dE = torch.empty(count, dim, device="cuda"), torch.empty(vocab, dim, device="cuda")
    ws = torch.empty(cdg.embed_grad_workspace_bytes(count, vocab, dim), dtype=torch.uint8, device="cuda")
    cdg.embed(E, t, out, count, vocab, dim, "f32", scale=2.5)
    cdg.embed_grad(d, t, dE, ws, count, vocab, dim, "f32", scale=2.5)
    a, b = float((out.double() * d.double()).sum()), float((E.double() * dE.double()).sum())
    size = float((out.double() * d.double()).abs().sum())
    assert abs(a - b) <= 2.0 ** -20 * size


def test_no_tokens():
    import torch
    out = torch.full((5, 6), 3.0, device="cuda")
    ws = torch.empty(cdg.embed_grad_workspace_bytes(0, 5, 6), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    d = torch.empty(0, 6, device="cuda")
    cdg.embed_grad(d, none, out, ws, 0, 5, 6, "f32", accumulate=True)
    assert (out == 3.0).all()
    cdg.embed_grad(d, none, out, ws, 0, 5, 6, "f32")
    assert (out == 0.0).all()
    cdg.embed(out, none, d, 0, 5, 6, "f32")
    t = torch.full((4,), -1, device="cuda")
    d4 = torch.randn(4, 6, device="cuda")
    ws = torch.empty(cdg.embed_grad_workspace_bytes(4, 5, 6), dtype=torch.uint8, device="cuda")
    out.fill_(3.0)
    cdg.embed_grad(d4, t, out, ws, 4, 5, 6, "f32")
    assert (out == 0.0).all()


def test_table_offsets_past_32_bits():
    """A table of more than 2^32 bytes: its last rows are read and written as any other."""
    import torch
    vocab, dim, count = 70001, 32776, 6
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[-2:] = torch.randn(2, dim, device="cuda").bfloat16()
    t = torch.tensor([vocab - 1, 0, vocab - 2, -1, vocab, vocab - 1], device="cuda")
    out = torch.empty(count, dim, dtype=torch.bfloat16, device="cuda")
    cdg.embed(table, t, out, count, vocab, dim, "bf16")
    assert torch.equal(out[0], table[-1]) and torch.equal(out[2], table[-2]) and not out[[1, 3, 4]].any()
    want = (out[0].float() + out[5].float()).bfloat16()
    ws = torch.empty(cdg.embed_grad_workspace_bytes(count, vocab, dim), dtype=torch.uint8, device="cuda")
    cdg.embed_grad(out, t, table, ws, count, vocab, dim, "bf16")
    assert torch.equal(table[-1], want) and torch.equal(table[-2], out[2]) and not table[:-2].any()
