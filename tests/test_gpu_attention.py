"""GPU tests of the attention and its gradient against the 64-bit definitions,
within bounds that count roundings (attention_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref
import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu


class Case:
    """Packed sequences of a plan, and what the definitions say of them."""

    def __init__(self, lens, klens, heads, kv_heads, dim, dtype, causal=True, window=0, scale=None, packed=False, offsets=torch.int32,
                 behind=0, seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.klens = lens, klens or lens
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        self.causal, self.window, self.scale = causal, window, scale or dim ** -0.5
        nq, nk = sum(self.lens) + behind, sum(self.klens) + behind
        self.nq, self.nk = nq, nk
        t = ref.DTYPE[dtype]
        widths = [heads * dim, kv_heads * dim, kv_heads * dim]
        cast = lambda *s: torch.randn(*s, generator=g).to(t)  # noqa: E731
        if packed:
            self.q, self.k, self.v = cast(nq, sum(widths)).cuda().split(widths, 1)
        else:
            self.q, self.k, self.v = cast(nq, widths[0]).cuda(), cast(nk, widths[1]).cuda(), cast(nk, widths[2]).cuda()
        self.q.mul_(spread)
        self.do = cast(nq, widths[0]).cuda()
        self.packed = packed
        edges = lambda ns: torch.tensor([0] + ns).cumsum(0)  # noqa: E731
        self.qe, self.ke = edges(self.lens), edges(self.klens)
        self.qo, self.ko = (e.to(offsets).cuda() for e in (self.qe, self.ke)) if offsets else (None, None)
        self.plan = cdg.attention_plan(heads, kv_heads, dim, dtype, causal, window, self.scale)
        self.ws = torch.empty(self.plan.workspace_bytes(nq, nk, len(lens)), dtype=torch.uint8, device="cuda")
        self.gws = torch.empty(self.plan.grad_workspace_bytes(nq, nk, len(lens)), dtype=torch.uint8, device="cuda")
        full = dict(device="cuda", dtype=t)
        self.o = torch.full((nq, widths[0]), 7.0, **full)
        self.lse = torch.full((heads, nq), 7.0, device="cuda")
        if packed:
            self.dq, self.dk, self.dv = torch.full((nq, sum(widths)), 7.0, **full).split(widths, 1)
        else:
            self.dq, self.dk, self.dv = (torch.full((n, w), 7.0, **full) for n, w in zip((nq, nk, nk), widths))

    def forward(self, stream=None):
        self.plan.attend(self.q, self.k, self.v, self.o, self.lse, self.ws, self.nq, self.nk, q_offsets=self.qo, k_offsets=self.ko,
                         stream=stream)

    def backward(self, stream=None):
        self.plan.attend_grad(self.q, self.k, self.v, self.o, self.lse, self.do, self.dq, self.dk, self.dv, self.gws, self.nq, self.nk,
                              q_offsets=self.qo, k_offsets=self.ko, stream=stream)

    def run(self):
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        assert self.plan.device_status() == 0

    def outputs(self):
        return [self.o, self.lse, self.dq, self.dk, self.dv]

    def parts(self):
        """(query rows, key rows) of each sequence."""
        return [(slice(int(self.qe[b]), int(self.qe[b + 1])), slice(int(self.ke[b]), int(self.ke[b + 1]))) for b in range(len(self.lens))]

    def check(self, skip=()):
        cols = lambda x, h: x.cpu().double()[:, h * self.dim:(h + 1) * self.dim]  # noqa: E731
        group = self.heads // self.kv_heads
        how = (self.causal, self.window, self.scale, self.dtype)
        lse_got = self.lse.cpu().double()
        for b, (qs, ks) in enumerate(self.parts()):
            if b in skip:
                continue
            for kh in range(self.kv_heads):
                k, v = cols(self.k, kh)[ks], cols(self.v, kh)[ks]
                sums = [torch.zeros_like(k) for _ in range(4)]
                for h in range(kh * group, (kh + 1) * group):
                    q, do = cols(self.q, h)[qs], cols(self.do, h)[qs]
                    o, lse, tol_o, tol_lse = ref.forward(q, k, v, *how)
                    near(cols(self.o, h)[qs], o, tol_o, ("o", b, h))
                    got = lse_got[h, qs]
                    assert torch.equal(torch.isinf(got), torch.isinf(lse)), ("lse", b, h)
                    seen = ~torch.isinf(lse)
                    near(got[seen], lse[seen], tol_lse[seen], ("lse", b, h))
                    # the gradient of what the forward wrote
                    (dq, dk, dv), tol = ref.gradient(q, k, v, cols(self.o, h)[qs], got, do, *how)
                    near(cols(self.dq, h)[qs], dq, tol[0], ("dq", b, h))
                    for s, x in zip(sums, (dk, dv, tol[1], tol[2])):
                        s += x
                near(cols(self.dk, kh)[ks], sums[0], sums[2], ("dk", b, kh))
                near(cols(self.dv, kh)[ks], sums[1], sums[3], ("dv", b, kh))
        # rows that no sequence holds are left alone
        for x, n in ((self.o, self.qe[-1]), (self.dq, self.qe[-1]), (self.dk, self.ke[-1]), (self.dv, self.ke[-1])):
            assert (x[int(n):] == 7).all()
        assert (self.lse[:, int(self.qe[-1]):] == 7).all()


def near(got, want, tol, what):
    off = (got - want).abs() - tol
    assert got.shape == want.shape and (off <= 0).all(), (what, float(off.max()), float((got - want).abs().max()), int((off > 0).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 100)])
def test_ragged_sequences(dtype, dim, causal, window):
    c = Case([1, 127, 0, 128, 129, 2, 300], None, 4, 2, dim, dtype, causal, window, behind=3, seed=dim)
    c.run()
    c.check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (3, 3), (8, 1)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("offsets", [torch.int32, torch.int64])
def test_head_layouts_and_strides(heads, kv_heads, packed, offsets):
    c = Case([70, 257], None, heads, kv_heads, 64, "bf16", packed=packed, offsets=offsets, seed=heads)
    c.run()
    c.check()


@pytest.mark.parametrize("lens,klens", [([5], [300]), ([300], [5]), ([130, 1, 64, 0, 7], [129, 513, 0, 5, 7]), ([1], [1]), ([257], [1])])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 33)])
def test_other_numbers_of_keys(lens, klens, causal, window):
    """Among them rows that see nothing: o = 0, lse = -inf and no gradient."""
    c = Case(lens, klens, 4, 2, 64, "f16", causal, window, seed=len(lens))
    c.run()
    c.check()
    if causal and lens == [300]:
        assert torch.isinf(c.lse[:, :295]).all() and (c.o[:295] == 0).all() and (c.dq[:295] == 0).all()


@pytest.mark.parametrize("lens,klens,heads,kv_heads,dim,causal", [
    ([1], [5000], 4, 1, 128, True), ([2000], None, 1, 1, 128, False), ([2500], None, 2, 1, 64, True), ([300, 260], [2100, 3000], 2, 2, 40, True)])
def test_few_items_are_split(lens, klens, heads, kv_heads, dim, causal):
    c = Case(lens, klens, heads, kv_heads, dim, "bf16", causal, seed=dim)
    assert c.ws.numel() > 256  # the workspace of parts
    c.run()
    c.check()


def test_one_sequence_without_offsets():
    c = Case([333], None, 2, 1, 128, "bf16", offsets=None)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_that_grow_from_step_to_step(dtype):
    """The running maximum rises by far more than 2^8 at every step, and falls."""
    c = Case([640], None, 2, 2, 64, dtype, causal=False, seed=5)
    ramp = torch.tensor([0.1, 3.0, 9.0, 0.5, 20.0], device="cuda").repeat_interleave(128)[:, None].to(c.k.dtype)
    c.k.mul_(ramp)
    c.run()
    c.check()


def test_large_scale_and_flat_scores():
    for scale, spread in ((4.0, 3.0), (1e-6, 1.0)):
        c = Case([200, 140], None, 2, 1, 64, "bf16", scale=scale, spread=spread, seed=7)
        c.run()
        c.check()


def test_many_short_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 9, (150,), generator=g).tolist()
    c = Case(lens, None, 2, 1, 64, "bf16", seed=9)
    c.run()
    c.check()


def test_more_items_than_sms():
    c = Case([900, 1500, 64, 700], None, 16, 8, 64, "bf16", seed=11)
    c.run()
    c.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_neighbours_that_are_not_finite(dim):
    """A sequence of NaN and infinities between others, and behind the last, changes nothing of theirs."""
    a, b = (Case([130, 77, 200], None, 4, 2, dim, "bf16", behind=20, seed=2) for _ in range(2))
    for x, e in ((b.q, b.qe), (b.do, b.qe), (b.k, b.ke), (b.v, b.ke)):
        x[int(e[1]):int(e[2])] = math.nan
        x[int(e[-1]):] = math.inf
    a.run()
    b.run()
    a.check()
    b.check(skip=(1,))
    rows = torch.ones(a.nq, dtype=torch.bool, device="cuda")
    rows[130:207] = False
    for x, y in zip(a.outputs(), b.outputs()):
        x, y = (x.T, y.T) if x.shape[0] == a.heads else (x, y)
        assert torch.equal(x[rows], y[rows])
    assert torch.isnan(b.o[130:207]).all()


def test_a_head_that_is_not_finite():
    a, b = (Case([200], None, 4, 2, 64, "f16", seed=4) for _ in range(2))
    b.k[:, 64:] = math.nan  # the second key head: query heads 2 and 3
    a.run()
    b.run()
    for x, y in ((a.o[:, :128], b.o[:, :128]), (a.dq[:, :128], b.dq[:, :128]), (a.dk[:, :64], b.dk[:, :64]), (a.dv[:, :64], b.dv[:, :64])):
        assert torch.equal(x, y)


def test_offsets_are_cut_to_the_rows():
    c = Case([100, 60], None, 2, 1, 64, "bf16", seed=6)
    c.qo[2] = c.ko[2] = 10 ** 9
    c.run()
    c.check()
    c.qo[0] = c.ko[0] = -5
    c.run()
    c.check()
    c.qo.copy_(torch.tensor([160, 100, 0]))  # sequences that end before they begin
    for x in c.outputs():
        x.fill_(7.0)
    c.run()
    assert (c.o == 7).all() and (c.dq == 7).all()


def test_no_rows():
    p = cdg.attention_plan(4, 2, 64)
    b16 = dict(device="cuda", dtype=torch.bfloat16)
    q, k = torch.randn(10, 256, **b16), torch.randn(12, 128, **b16)
    o, lse = torch.full_like(q, 7.0), torch.full((4, 10), 7.0, device="cuda")
    ws = torch.empty(1 << 16, device="cuda", dtype=torch.uint8)
    none = k[:0]
    p.attend(q, none, none, o, lse, ws, 10, 0)
    assert (o == 0).all() and torch.isinf(lse).all()
    dq = torch.full_like(q, 7.0)
    p.attend_grad(q, none, none, o, lse, q, dq, none, none, ws, 10, 0)
    assert (dq == 0).all()
    dk, dv = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    p.attend_grad(q[:0], k, k, q[:0], lse[:, :0], q[:0], q[:0], dk, dv, ws, 0, 12)
    assert (dk == 0).all() and (dv == 0).all()
    p.attend(q[:0], k, k, q[:0], lse[:, :0], ws, 0, 12)
    torch.cuda.synchronize()
    assert p.device_status() == 0


def test_repeated_calls_give_the_same_bits():
    c = Case([500, 900], None, 8, 2, 128, "bf16", seed=8)
    c.run()
    first = [x.clone() for x in c.outputs()]
    for _ in range(5):
        for x in c.outputs():
            x.zero_()
        c.run()
        assert all(torch.equal(x, y) for x, y in zip(c.outputs(), first))


@pytest.mark.parametrize("lens,heads", [([77], 8), ([300, 700], 4), ([1800], 1)])
def test_captured_calls_replay(lens, heads):
    c = Case(lens, None, heads, 1, 64, "bf16", seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.forward()
        c.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.forward()
        c.backward()
    for seed in range(1, 4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x in (c.q, c.k, c.v, c.do):
            x.normal_(generator=g)
        c.run()
        want = [x.clone() for x in c.outputs()]
        for x in c.outputs():
            x.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert c.plan.device_status() == 0
        assert all(torch.equal(x, y) for x, y in zip(c.outputs(), want))


def test_two_calls_at_once():
    """One plan on two streams, a workspace each."""
    a, b = Case([900, 400], None, 8, 4, 128, "bf16", seed=12), Case([1300], None, 8, 4, 128, "bf16", seed=13)
    b.plan = a.plan
    a.run()
    b.run()
    want = [[x.clone() for x in c.outputs()] for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for c in (a, b):
        for x in c.outputs():
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip((a, b), streams):
            c.forward(stream=s)
            c.backward(stream=s)
    torch.cuda.synchronize()
    assert a.plan.device_status() == 0
    for c, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(c.outputs(), w))
