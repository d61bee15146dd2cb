"""GPU tests of the norms of queries and keys with the rotation, and their
gradient, against the 64-bit definitions."""
import math

import pytest
import torch

import attention_reference as ref
import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu
EPS = 1e-5


def angle_error(dtype):
    """An angle's own rounding and that of its cosine and sine: 16-bit results use the hardware's approximations."""
    return 2.0 ** -20 if dtype != "f32" else 2.0 ** -21


class Case:
    def __init__(self, tokens, heads, kv_heads, dim, rot, dtype, norm=True, interleaved=False, factor=1.0, positions="far", shift=0,
                 packed=False, weights=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.dtype, self.norm = (tokens, heads, kv_heads, dim), dtype, norm
        t = ref.DTYPE[dtype]
        self.how = dict(rot=rot, interleaved=interleaved, factor=factor, norm=norm, eps=EPS)
        widths = (heads * dim, kv_heads * dim)

        def pair():
            if packed:  # side by side, with something behind them
                m = torch.randn(tokens, sum(widths) + 24, generator=g).to(t).cuda()
                return m[:, :widths[0]], m[:, widths[0]:sum(widths)]
            out = []
            for w in widths:  # `shift` elements into a buffer
                flat = torch.randn(tokens * w + shift, generator=g).to(t).cuda()
                out.append(flat[shift:].view(tokens, w))
            return out

        self.x, self.dy, self.y, self.dx = pair(), pair(), pair(), pair()
        if positions == "far":
            self.positions = torch.randint(0, 1 << 20, (tokens,), generator=g).cuda()
        elif positions == "int32":
            self.positions = torch.randint(-5000, 5000, (tokens,), generator=g, dtype=torch.int32).cuda()
        elif positions == "huge":
            self.positions = torch.randint(-(1 << 40), 1 << 40, (tokens,), generator=g).cuda()
        else:
            self.positions = None
        self.inv_freq = torch.tensor(cdg.rope_frequencies(rot), device="cuda") if rot else None
        w = 1.0 + 0.3 * torch.randn(2, dim, generator=g)
        self.w = w.cuda().unbind(0) if norm and weights else (None, None)
        self.dw = tuple(torch.full((dim,), 7.0, device="cuda") for _ in range(2)) if norm else (None, None)
        self.ws = torch.empty(cdg.qk_rope_grad_workspace_bytes(tokens, heads, kv_heads, dim), dtype=torch.uint8, device="cuda")

    def forward(self):
        cdg.qk_rope(*self.x, self.positions, self.inv_freq, *self.y, *self.sizes, self.dtype, w_q=self.w[0], w_k=self.w[1], **self.how)

    def backward(self):
        cdg.qk_rope_grad(*self.x, self.positions, self.inv_freq, *self.dy, *self.dx, self.ws, *self.sizes, self.dtype, w_q=self.w[0],
                         w_k=self.w[1], dw_q=self.dw[0], dw_k=self.dw[1], **self.how)

    def check(self):
        tokens, heads, kv_heads, dim = self.sizes
        pos = torch.arange(tokens) if self.positions is None else self.positions.cpu()
        f = torch.zeros(0) if self.inv_freq is None else self.inv_freq.cpu()
        rot, inter, factor = self.how["rot"], self.how["interleaved"], self.how["factor"]
        # beside it: the reference's product of 64 bits, rounded by its size times 2^-53 (2^-13 radians at position 2^40), and
        # the kernel's frequency, cut to 2^-64 of a turn, times the position
        far = float(pos.abs().max()) if tokens else 0.0
        u, e_a = ref.U[self.dtype], angle_error(self.dtype) + far * (2.0 ** -53 + 4 * math.pi * 2.0 ** -64)
        e_n = (dim + 16) * ref.U32 if self.norm else 0.0  # the sum of squares, its root, and the product with the weight

        def swap(z):  # the other value of each rotated pair
            z = z.clone()
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
            z[..., a], z[..., b] = z[..., b].clone(), z[..., a].clone()
            z[..., rot:] = 0
            return z

        for i, h in enumerate((heads, kv_heads)):
            if h == 0:
                continue
            view = lambda m: m.cpu().double().reshape(tokens, h, dim)  # noqa: E731
            w = None if self.w[i] is None else self.w[i].cpu().double()
            x = view(self.x[i]).requires_grad_()
            wt = torch.ones(dim, dtype=torch.float64) if w is None else w
            wt.requires_grad_()
            y = ref.rotate(x, pos, f, rot, inter, factor, self.norm, EPS, wt)
            dy = view(self.dy[i])
            grads = torch.autograd.grad(y, [x, wt], dy, allow_unused=True)
            y = y.detach()
            scale = 1.0 / torch.sqrt(x.detach().pow(2).mean(-1, keepdim=True) + EPS) if self.norm else torch.ones(())
            z = (x.detach() * scale * wt.detach()) if self.norm else x.detach()
            mag = abs(factor) * (z.abs() + swap(z.abs()))
            mag[..., rot:] = z.abs()[..., rot:]
            near(view(self.y[i]), y, u * y.abs() + (e_n + e_a + 8 * ref.U32) * mag + ref.TINY[self.dtype], ("y", i))
            dz = abs(factor) * (dy.abs() + swap(dy.abs()))
            dz[..., rot:] = dy.abs()[..., rot:]
            e = 4 * e_n + e_a + 16 * ref.U32
            if self.norm:
                n = x.detach() * scale
                dn = dz * wt.detach().abs()
                big = scale * (dn + n.abs() * (dn * n.abs()).mean(-1, keepdim=True))
            else:
                big = dz
            near(view(self.dx[i]), grads[0], u * grads[0].abs() + e * big + ref.TINY[self.dtype], ("dx", i))
            if self.norm:
                terms = (dz * n.abs()).sum((0, 1))
                near(self.dw[i].cpu().double(), grads[1] if w is not None else torch.autograd.grad(ref.rotate(
                    x, pos, f, rot, inter, factor, True, EPS, wt), wt, dy)[0], (e + (tokens * h + 64) * ref.U32) * terms + 1e-30, ("dw", i))


def near(got, want, tol, what):
    off = (got - want).abs() - tol
    assert got.shape == want.shape and (off <= 0).all(), (what, float(off.max()), float((got - want).abs().max()), int((off > 0).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (64, 16), (256, 128), (80, 20), (96, 48), (40, 40), (34, 2), (2, 2), (33, 6), (1, 0), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_sizes_and_layouts(dtype, dim, rot, interleaved, norm):
    c = Case(37, 5, 2, dim, rot, dtype, norm, interleaved, seed=dim + rot)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("positions", ["int32", "huge", None])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [1.0, 1.3, -0.5])
def test_positions_and_factors(positions, dtype, factor):
    c = Case(60, 3, 1, 64, 64, dtype, True, False, factor, positions, seed=1)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("tokens", [1, 2, 255, 4100])
@pytest.mark.parametrize("heads,kv_heads", [(1, 0), (0, 3), (17, 3), (32, 8)])
def test_heads_and_lengths(tokens, heads, kv_heads):
    c = Case(tokens, heads, kv_heads, 64, 32, "bf16", seed=tokens)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rows_at_any_element(dtype, shift):
    c = Case(50, 4, 2, 64, 64, dtype, shift=shift, seed=shift)
    c.forward()
    c.backward()
    c.check()


def test_packed_rows_leave_the_rest_alone():
    c = Case(300, 6, 2, 64, 64, "bf16", packed=True, seed=3)
    behind = [m._base[:, 512:].clone() for m in (c.y[0], c.dx[0])]
    c.forward()
    c.backward()
    c.check()
    for m, b in zip((c.y[0], c.dx[0]), behind):
        assert torch.equal(m._base[:, 512:], b)


def test_without_weights_or_their_gradients():
    c = Case(100, 4, 2, 128, 128, "bf16", weights=False, seed=4)
    c.forward()
    c.backward()
    c.check()
    c.dw = (None, None)
    first = [m.clone() for m in c.dx]
    c.backward()
    assert all(torch.equal(a, b) for a, b in zip(c.dx, first))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    c = Case(200, 8, 2, 128, 64, dtype, seed=5)
    c.forward()
    c.backward()
    want = [m.clone() for m in (*c.y, *c.dx)]
    x = [m.clone() for m in c.x]
    c.dx = c.dy
    c.backward()
    c.y, c.x = x, x
    c.forward()
    assert all(torch.equal(a, b) for a, b in zip((*c.y, *c.dx), want))


def test_zero_rows_and_no_tokens():
    c = Case(20, 2, 1, 64, 64, "f32", seed=6)
    for m in c.x:
        m.zero_()
    c.forward()
    c.backward()
    c.check()
    c = Case(0, 2, 1, 64, 64, "f32", seed=6)
    c.forward()
    c.backward()
    assert all((w == 0).all() for w in c.dw)  # a sum of nothing


def test_a_row_that_is_not_finite_stays_there():
    a, b = Case(64, 4, 2, 64, 64, "bf16", seed=7), Case(64, 4, 2, 64, 64, "bf16", seed=7)
    b.x[0][9, 64:128] = math.inf
    for c in (a, b):
        c.forward()
    other = torch.ones(64, 256, dtype=torch.bool, device="cuda")
    other[9, 64:128] = False
    assert torch.equal(a.y[0][other], b.y[0][other]) and torch.equal(a.y[1], b.y[1])


def test_gradient_against_differences():
    """The kernel's own forward in fp32, along a direction; a central difference of h is off by h^2 and by the sums' rounding over h."""
    c = Case(40, 4, 2, 64, 32, "f32", seed=8)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(2):
        along = torch.randn(c.x[i].shape, generator=g, device="cuda")
        start, ends = c.x[i].clone(), []
        for h in (1e-2, -1e-2):
            c.x[i].copy_(start + h * along)
            c.forward()
            ends.append((c.y[i].double() * c.dy[i].double()).sum())
        c.x[i].copy_(start)
        got = (c.dx[i].double() * along.double()).sum()
        size = (c.dx[i].double() * along.double()).abs().sum()
        assert abs((ends[0] - ends[1]) / 2e-2 - got) < 1e-4 * size


def test_repeated_and_captured_calls_give_the_same_bits():
    c = Case(3000, 16, 4, 128, 128, "bf16", seed=9)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    outs = (*c.y, *c.dx, *c.dw)
    want = [m.clone() for m in outs]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.forward()
        c.backward()
    for _ in range(3):
        for m in outs:
            m.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_an_attention_block(dtype):
    """Rotation in the projection's buffer, attention, its gradient and the rotation's, against the chain in 64 bits."""
    lens, heads, kv_heads, dim = [150, 333, 1], 4, 2, 64
    n, widths = sum(lens), (heads * dim, kv_heads * dim, kv_heads * dim)
    t = ref.DTYPE[dtype]
    g = torch.Generator().manual_seed(11)
    qkv, do = torch.randn(n, sum(widths), generator=g).to(t).cuda(), torch.randn(n, widths[0], generator=g).to(t).cuda()
    pos = torch.cat([torch.arange(k) for k in lens]).cuda()
    freq = torch.tensor(cdg.rope_frequencies(dim), device="cuda")
    w_q, w_k = (1.0 + 0.1 * torch.randn(2, dim, generator=g)).cuda()
    plan = cdg.attention_plan(heads, kv_heads, dim, dtype)
    offsets = torch.tensor([0, 150, 483, 484], device="cuda", dtype=torch.int32)
    turned, dqkv = qkv.clone(), torch.empty_like(qkv)
    q, k, v = turned.split(widths, 1)
    dq, dk, dv = dqkv.split(widths, 1)
    sizes, how = (n, heads, kv_heads, dim, dtype), dict(norm=True, eps=EPS, w_q=w_q, w_k=w_k)
    o, lse = torch.empty_like(do), torch.empty(heads, n, device="cuda")
    ws = torch.empty(max(plan.workspace_bytes(n, n, 3), plan.grad_workspace_bytes(n, n, 3), cdg.qk_rope_grad_workspace_bytes(n, heads, kv_heads, dim)),
                     device="cuda", dtype=torch.uint8)
    dw_q, dw_k = torch.empty(2, dim, device="cuda")
    cdg.qk_rope(q, k, pos, freq, q, k, *sizes, **how)
    plan.attend(q, k, v, o, lse, ws, n, n, q_offsets=offsets, k_offsets=offsets)
    plan.attend_grad(q, k, v, o, lse, do, dq, dk, dv, ws, n, n, q_offsets=offsets, k_offsets=offsets)
    raw = qkv.split(widths, 1)
    cdg.qk_rope_grad(raw[0], raw[1], pos, freq, dq, dk, dq, dk, ws, *sizes, **how, dw_q=dw_q, dw_k=dw_k)
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    # the chain by automatic differentiation
    x = qkv.cpu().double().requires_grad_()
    wq, wk = (w.cpu().double().requires_grad_() for w in (w_q, w_k))
    xs = [m.reshape(n, -1, dim) for m in x.split(widths, 1)]
    rq, rk = (ref.rotate(m, pos.cpu(), freq.cpu(), dim, False, 1.0, True, EPS, w) for m, w in zip(xs, (wq, wk)))
    outs, at = [], 0
    for m in lens:
        s = slice(at, at + m)
        at += m
        kk, vv = (z[s].repeat_interleave(heads // kv_heads, 1) for z in (rk, xs[2]))
        z = torch.einsum("ihd,jhd->hij", rq[s], kk) * dim ** -0.5
        z = z.masked_fill(~ref.visible(m, m, True, 0), -math.inf)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), vv).flatten(1))
    y = torch.cat(outs)
    want = torch.autograd.grad(y, [x, wq, wk], do.cpu().double())
    # each of the chain's 16-bit tensors (turned q and k, p, o, ds, dq and dk) is off by u at most, elementwise: in the 2-norm
    # the results are off by no more than their sum
    for got, ref64 in ((o, y.detach()), (dqkv, want[0]), (dw_q, want[1]), (dw_k, want[2])):
        assert (got.cpu().double() - ref64).norm() <= 8 * ref.U[dtype] * ref64.norm()
