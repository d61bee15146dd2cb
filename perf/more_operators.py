"""Cases that measure the operators of an attention block in a training step:
attention over packed sequences and its gradient, and the norms of queries and
keys with the position rotation, and their gradient.

Every case names one operator and its sizes.  ``run`` makes one pass: the
operator's plain form in elementary torch operations where ``own`` is false,
the calls a user makes of this package where it is true.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6


def _attention(name, op, lens, heads, kv_heads, dim, dtype, causal=True, window=0, klens="", packed=False):
    """lens: the sequences' numbers of queries; klens: of keys, where these differ."""
    return dict(name=name, op=op, lens=lens, klens=klens, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                causal=causal, window=window, packed=packed)


def _rope(name, op, tokens, heads, kv_heads, dim, rot, dtype, norm=True, interleaved=False, far=0, factor=1.0,
          packed=True):
    """rot: the rotated part of a head; far: the largest first position of a sequence."""
    return dict(name=name, op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot, dtype=dtype,
                norm=norm, interleaved=interleaved, far=far, factor=factor, packed=packed)


def listed():
    return [
        # a short text through a small model: one CTA's worth of work a head, latency counts
        _attention("attention, short text", "attention", "77", 8, 2, 64, "f16"),
        # a packed batch of documents of uneven lengths, grouped heads, from one projection's buffer
        _attention("attention, packed documents", "attention", "1033,64,2500,777,1,4096,3001,129,2047,1536", 16, 4,
                   128, "bf16", packed=True),
        # a new part of a text against all that came before it, within a window
        _attention("attention, windowed part", "attention", "1000,3000", 12, 12, 64, "bf16", window=1024,
                   klens="5000,3000"),
        # one long sequence
        _attention("attention, long sequence", "attention", "8192", 16, 4, 128, "bf16", packed=True),
        # the gradient of a short batch of an odd head width without a causal mask, as an encoder has
        _attention("attention gradient, short batch", "attention_grad", "100,65,128,7", 8, 8, 80, "f16",
                   causal=False),
        # the gradient of the packed batch of documents
        _attention("attention gradient, documents", "attention_grad", "1033,64,2500,777,1,4096,3001,129,2047,1536",
                   16, 4, 128, "bf16", packed=True),
        # the gradient of one long sequence
        _attention("attention gradient, long", "attention_grad", "8192", 16, 4, 128, "bf16", packed=True),
        # one token that a model decodes at a far position
        _rope("qk rope, one token", "rope", 1, 32, 8, 128, 128, "bf16", far=100000),
        # a training step's queries and keys, normed and rotated out of the projection's buffer
        _rope("qk rope, training step", "rope", 32768, 32, 8, 128, 128, "bf16"),
        # neighbouring pairs in a quarter of each head, without norms, a stretched context
        _rope("qk rope, part of the head", "rope", 4099, 16, 16, 64, 16, "f16", norm=False, interleaved=True,
              far=30000, factor=1.2),
        # the gradient of a short fp32 step of odd sizes
        _rope("qk rope gradient, short", "rope_grad", 517, 9, 3, 96, 48, "f32", packed=False),
        # the gradient of the training step
        _rope("qk rope gradient, training step", "rope_grad", 32768, 32, 8, 128, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention_grad", "attention_grad", "rope", "rope_grad"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    if op in ("rope", "rope_grad"):
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        tokens = _log(rng, 1, min(32768, 32768 * 40 * 128 * 2 // ((heads + kv_heads) * dim * SIZE[dtype])))
        case = _rope("", op, tokens, heads, kv_heads, dim, rot, dtype, norm=rng.random() < 0.7,
                     interleaved=rng.random() < 0.3, far=rng.choice([0, 0, 4000, 1000000]),
                     factor=rng.choice([1.0, 1.0, 1.3]), packed=rng.random() < 0.6)
    else:
        dim = rng.choice([64, 64, 128, 128, 128, 40, 80, 96])
        how, causal = rng.random(), rng.random() < 0.7
        window = _log(rng, 16, 4096) if causal and rng.random() < 0.3 else 0
        dtype, packed = rng.choice(["bf16", "bf16", "f16"]), how >= 0.25 and rng.random() < 0.5
        count, longest = _log(rng, 1, 32), _log(rng, 1, 8192)
        while True:
            lens = [rng.randint(max(1, longest // 4), longest) for _ in range(count)]
            klens = ""
            if how < 0.15:  # keys from before the queries
                klens = ",".join(str(n + rng.randint(0, longest)) for n in lens)
            elif how < 0.25:  # fewer keys than queries: under a causal mask the first queries see none
                klens = ",".join(str(max(1, n - rng.randint(0, n))) for n in lens)
            case = _attention("", op, ",".join(map(str, lens)), heads, kv_heads, dim, dtype, causal=causal,
                              window=window, klens=klens, packed=packed)
            # no more than the long listed sequence takes, also when padded to the longest
            if heads * dim * _pairs(case) <= 16 * 128 * 8192 * 8193 // 2 and \
                    heads * count * longest * max(_lens(case)[1]) <= 16 * 8192 * 8192:
                break
            longest -= longest // 4
    del case["name"]
    return case


def _lens(case):
    q = [int(n) for n in case["lens"].split(",")]
    return q, [int(n) for n in case["klens"].split(",")] if case["klens"] else q


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(widths, tokens, packed, dtype, fill):
    """Matrices of `tokens` rows, side by side in one buffer where packed."""
    if packed:
        return list(fill(tokens, sum(widths)).to(dtype).split(widths, dim=1))
    return [fill(tokens, w).to(dtype) for w in widths]


def prepare(case, seed):
    g, dt, s = _gen(seed), DTYPES[case["dtype"]], dict(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] in ("rope", "rope_grad"):
        n, rot = case["tokens"], case["rot"]
        widths = [heads * dim, kv_heads * dim]
        s["q"], s["k"] = _rows(widths + [kv_heads * dim], n, case["packed"], dt, randn)[:2]
        # texts of 2048 tokens that start anywhere up to `far`
        first = torch.randint(0, case["far"] + 1, (n // 2048 + 1,), generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        s["positions"] = first[at // 2048] + at % 2048
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float32) / rot)
        s["w_q"], s["w_k"] = (1.0 + 0.2 * randn(2, dim)) if case["norm"] else (None, None)
        if case["op"] == "rope":
            s["q_out"], s["k_out"] = (torch.empty(n, w, device="cuda", dtype=dt) for w in widths)
        else:
            s["dq_out"], s["dk_out"] = (0.01 * x for x in _rows(widths, n, False, dt, randn))
            s["dq"], s["dk"] = _rows(widths, n, case["packed"], dt, lambda *shape: torch.empty(*shape, device="cuda"))
            if case["norm"]:
                s["dw_q"], s["dw_k"] = torch.empty(2, dim, device="cuda")
            if own:
                import implicit_gemm_dgrad_gb300 as cdg
                size = cdg.qk_rope_grad_workspace_bytes(n, heads, kv_heads, dim)
                s["workspace"] = torch.empty(size, device="cuda", dtype=torch.uint8)
        return s

    lens, klens = _lens(case)
    nq, nk = sum(lens), sum(klens)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["longest"], s["k_longest"] = max(lens), max(klens)
    for name, ns in (("q_offsets", lens), ("k_offsets", klens)):
        s[name] = torch.tensor([0] + list(np.cumsum(ns)), device="cuda", dtype=torch.int32)
    widths = [heads * dim, kv_heads * dim, kv_heads * dim]
    if case["packed"]:
        s["q"], s["k"], s["v"] = _rows(widths, nq, True, dt, randn)
    else:
        s["q"], s["k"], s["v"] = (randn(n, w).to(dt) for n, w in zip((nq, nk, nk), widths))
    # scores of some spread: a few keys of each row stand out
    s["q"].mul_(1.5)
    if case["op"] == "attention":
        s["o"] = torch.empty(nq, heads * dim, device="cuda", dtype=dt)
        s["lse"] = torch.empty(heads, nq, device="cuda")
    else:
        s.update(_plain_attention(s))  # o and lse, as the pass before left them
        s["do"] = (0.01 * randn(nq, heads * dim)).to(dt)
        if case["packed"]:
            s["dq"], s["dk"], s["dv"] = torch.empty(nq, sum(widths), device="cuda", dtype=dt).split(widths, dim=1)
        else:
            s["dq"], s["dk"], s["dv"] = (torch.empty(n, w, device="cuda", dtype=dt)
                                         for n, w in zip((nq, nk, nk), widths))
    if own:
        import implicit_gemm_dgrad_gb300 as cdg
        s["plan"] = cdg.attention_plan(heads, kv_heads, dim, dtype=case["dtype"], causal=case["causal"],
                                       window=case["window"], scale=s["scale"])
        need = s["plan"].workspace_bytes if case["op"] == "attention" else s["plan"].grad_workspace_bytes
        s["workspace"] = torch.empty(need(nq, nk, len(lens)), device="cuda", dtype=torch.uint8)
    return s


# ---- plain forms: elementary operations in 32 bits (angles in 64), rounded once at the end


def _padded(x, offsets, longest, heads, dim):
    """Packed rows as (sequence, head, place, dim); places past a sequence's end hold other rows."""
    at = (offsets[:-1, None] + torch.arange(longest, device="cuda")).clamp(max=x.shape[0] - 1)
    return x.float()[at].reshape(len(offsets) - 1, longest, heads, dim).transpose(1, 2)


def _packed(x, offsets, rows):
    """(sequence, head, place, dim) back to packed rows of heads * dim."""
    at = torch.arange(rows, device="cuda")
    which = torch.searchsorted(offsets.long(), at, right=True) - 1
    return x.transpose(1, 2)[which, at - offsets[which]].reshape(rows, -1)


def _visible(s):
    """(sequence, query, key): whether the query sees the key."""
    n, kn = s["q_offsets"].diff()[:, None, None], s["k_offsets"].diff()[:, None, None]
    i = torch.arange(s["longest"], device="cuda")[:, None]
    j = torch.arange(s["k_longest"], device="cuda")
    see = (i < n) & (j < kn)
    if s["causal"]:
        see = see & (j <= i + kn - n)
    if s["window"]:
        see = see & (j > i + kn - n - s["window"])
    return see[:, None]


def _scores(s):
    """Queries, keys and values by sequence and head (a group's keys repeated), and the masked scores."""
    group = s["heads"] // s["kv_heads"]
    q = _padded(s["q"], s["q_offsets"], s["longest"], s["heads"], s["dim"])
    k, v = (_padded(s[x], s["k_offsets"], s["k_longest"], s["kv_heads"], s["dim"]).repeat_interleave(group, 1)
            for x in ("k", "v"))
    scores = (q @ k.transpose(2, 3)) * s["scale"]
    return q, k, v, scores.masked_fill_(~_visible(s), -math.inf)


def _plain_attention(s):
    _, _, v, x = _scores(s)
    top = x.max(3, keepdim=True).values
    top = torch.where(top > -math.inf, top, torch.zeros((), device="cuda"))
    x = x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    o = (x @ v) / torch.where(total > 0, total, torch.ones((), device="cuda"))
    lse = top + torch.log(total)
    rows = s["q"].shape[0]
    return dict(o=_packed(o, s["q_offsets"], rows).to(s["q"].dtype),
                lse=_packed(lse, s["q_offsets"], rows).t().contiguous())


def _plain_attention_grad(s):
    q, k, v, p = _scores(s)
    rows, krows, dt = s["q"].shape[0], s["k"].shape[0], s["q"].dtype
    do, o = (_padded(s[x], s["q_offsets"], s["longest"], s["heads"], s["dim"]) for x in ("do", "o"))
    lse = _padded(s["lse"].t(), s["q_offsets"], s["longest"], s["heads"], 1)
    p = p.sub_(torch.where(lse > -math.inf, lse, torch.zeros((), device="cuda"))).exp_()
    ds = do @ v.transpose(2, 3)
    ds = ds.sub_((do * o).sum(3, keepdim=True)).mul_(p)
    dq = ds @ k * s["scale"]
    of_group = (len(s["k_offsets"]) - 1, s["kv_heads"], -1, s["k_longest"], s["dim"])
    dk = (ds.transpose(2, 3) @ q * s["scale"]).view(of_group).sum(2)
    dv = (p.transpose(2, 3) @ do).view(of_group).sum(2)
    return dict(dq=_packed(dq, s["q_offsets"], rows).to(dt), dk=_packed(dk, s["k_offsets"], krows).to(dt),
                dv=_packed(dv, s["k_offsets"], krows).to(dt))


def _turned(x, s, back):
    """The rotated part of x (token, head, dim) turned by its positions' angles, or back by them."""
    rot, half = s["rot"], s["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = (f.float()[:, None] * s["factor"] for f in (torch.cos(angle), torch.sin(angle)))
    sin = -sin if back else sin
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, half), slice(half, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope(s, x, w):
    y = x.float().reshape(x.shape[0], -1, s["dim"])
    if s["norm"]:
        y = y / torch.sqrt(y.square().mean(2, keepdim=True) + EPS) * w
    return _turned(y, s, False).flatten(1).to(x.dtype)


def _plain_rope_grad(s, x, dy, w):
    dz = _turned(dy.float().reshape(x.shape[0], -1, s["dim"]), s, True)
    if not s["norm"]:
        return dz.flatten(1).to(x.dtype), None
    n = x.float().reshape(dz.shape)
    scale = 1.0 / torch.sqrt(n.square().mean(2, keepdim=True) + EPS)
    n = n * scale
    dw = (dz * n).sum((0, 1))
    dn = dz * w
    return (scale * (dn - n * (dn * n).mean(2, keepdim=True))).flatten(1).to(x.dtype), dw


def _run_plain(s):
    if s["op"] == "attention":
        return _plain_attention(s)
    if s["op"] == "attention_grad":
        return _plain_attention_grad(s)
    if s["op"] == "rope":
        return dict(q=_plain_rope(s, s["q"], s["w_q"]), k=_plain_rope(s, s["k"], s["w_k"]))
    dq, dw_q = _plain_rope_grad(s, s["q"], s["dq_out"], s["w_q"])
    dk, dw_k = _plain_rope_grad(s, s["k"], s["dk_out"], s["w_k"])
    return dict(dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k)


def _run_own(s):
    import implicit_gemm_dgrad_gb300 as cdg
    op = s["op"]
    if op == "attention":
        s["plan"].attend(s["q"], s["k"], s["v"], s["o"], s["lse"], s["workspace"], s["q"].shape[0], s["k"].shape[0],
                         q_offsets=s["q_offsets"], k_offsets=s["k_offsets"])
        return dict(o=s["o"], lse=s["lse"])
    if op == "attention_grad":
        s["plan"].attend_grad(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"],
                              s["workspace"], s["q"].shape[0], s["k"].shape[0], q_offsets=s["q_offsets"],
                              k_offsets=s["k_offsets"])
        return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    sizes = (s["tokens"], s["heads"], s["kv_heads"], s["dim"], s["dtype"])
    how = dict(rot=s["rot"], interleaved=s["interleaved"], factor=s["factor"], norm=s["norm"], eps=EPS, w_q=s["w_q"],
               w_k=s["w_k"])
    if op == "rope":
        cdg.qk_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], *sizes, **how)
        return dict(q=s["q_out"], k=s["k_out"])
    cdg.qk_rope_grad(s["q"], s["k"], s["positions"], s["inv_freq"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                     s["workspace"], *sizes, **how, dw_q=s.get("dw_q"), dw_k=s.get("dw_k"))
    return dict(dq=s["dq"], dk=s["dk"], dw_q=s.get("dw_q"), dw_k=s.get("dw_k"))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _pairs(case):
    """Visible pairs of a query and a key, over the sequences."""
    total = 0
    for n, kn in zip(*_lens(case)):
        end = np.arange(n) + kn - n + 1 if case["causal"] else np.full(n, kn)
        first = end - case["window"] if case["window"] else np.zeros(n, int)
        total += int(np.clip(np.clip(end, 0, kn) - np.clip(first, 0, kn), 0, None).sum())
    return total


def work(case):
    """Bytes: every input read once and every output written once.  Flops of the
    attention: two products of 2 * dim a visible pair and head, five for the
    gradient (the scores again, dP, dV, dQ, dK)."""
    e, heads, kv_heads, dim = SIZE[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("rope", "rope_grad"):
        n = case["tokens"] * (heads + kv_heads) * dim
        moved = 2 if case["op"] == "rope" or not case["norm"] else 3
        return {"bytes": moved * n * e + 8 * case["tokens"], "flops": (10 if case["norm"] else 4) * n}
    lens, klens = _lens(case)
    q, kv = sum(lens) * heads * dim * e, sum(klens) * kv_heads * dim * e
    flops = 4 * dim * heads * _pairs(case)
    if case["op"] == "attention":
        return {"bytes": 2 * q + 2 * kv + 4 * sum(lens) * heads, "flops": flops}
    return {"bytes": 4 * q + 4 * kv + 4 * sum(lens) * heads, "flops": 5 * flops // 2}


# ---- the definitions in 64 bits


def _exact_rope(case, s, x, w):
    """The rotation as a product of complex numbers."""
    dim, rot = case["dim"], case["rot"]
    y = x.reshape(x.shape[0], -1, dim)
    if case["norm"]:
        y = y * torch.rsqrt(y.pow(2).sum(2, keepdim=True) / dim + EPS) * w.double()
    turned, rest = y[..., :rot], y[..., rot:]
    pairs = turned.unflatten(2, (rot // 2, 2)) if case["interleaved"] else turned.unflatten(2, (2, rot // 2)).mT
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, case["factor"]), angle)[:, None]
    pairs = torch.view_as_real(z)
    turned = pairs.flatten(2) if case["interleaved"] else pairs.mT.flatten(2)
    return torch.cat([turned, rest], 2).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    op, heads, kv_heads, dim = case["op"], case["heads"], case["kv_heads"], case["dim"]
    if op == "rope":
        return {n: _exact_rope(case, s, s[n].double(), s["w_" + n]) for n in ("q", "k")}
    if op == "rope_grad":
        out = {}
        for n in ("q", "k"):
            x = s[n].double().requires_grad_()
            w = s["w_" + n].double().requires_grad_() if case["norm"] else None
            y = _exact_rope(case, s, x, w)
            got = torch.autograd.grad(y, [x] + [w] * case["norm"], s[f"d{n}_out"].double())
            out["d" + n], out["dw_" + n] = got[0], got[1] if case["norm"] else None
        return out
    lens, klens = _lens(case)
    group, qs, ks = heads // kv_heads, np.cumsum([0] + lens), np.cumsum([0] + klens)
    if op == "attention":
        out = dict(o=torch.zeros(sum(lens), heads, dim, device="cuda", dtype=torch.float64),
                   lse=torch.full((heads, sum(lens)), -math.inf, device="cuda", dtype=torch.float64))
    else:
        out = {"d" + n: torch.zeros(s[n].shape[0], s[n].shape[1] // dim, dim, device="cuda", dtype=torch.float64)
               for n in ("q", "k", "v")}
    for b, (n, kn) in enumerate(zip(lens, klens)):
        at, kat = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
        behind = torch.arange(n, device="cuda")[:, None] + (kn - n) - torch.arange(kn, device="cuda")
        hidden = torch.zeros(n, kn, device="cuda", dtype=torch.bool)
        if case["causal"]:
            hidden |= behind < 0
        if case["window"]:
            hidden |= behind >= case["window"]
        for h in range(heads):
            c, kc = slice(h * dim, (h + 1) * dim), slice(h // group * dim, (h // group + 1) * dim)
            q, k, v = s["q"][at, c].double(), s["k"][kat, kc].double(), s["v"][kat, kc].double()
            z = torch.where(hidden, -math.inf, q @ k.T * s["scale"])
            if op == "attention":
                lse = torch.logsumexp(z, 1)
                out["lse"][h, at] = lse
                out["o"][at, h] = torch.where(hidden, 0.0, torch.exp(z - lse[:, None])) @ v
                continue
            p = torch.where(hidden, 0.0, torch.exp(z - s["lse"][h, at].double()[:, None]))
            do, o = s["do"][at, c].double(), s["o"][at, c].double()
            ds = p * (do @ v.T - torch.linalg.vecdot(do, o)[:, None]) * s["scale"]
            out["dq"][at, h] = ds @ k
            out["dk"][kat, h // group] += ds.T @ q
            out["dv"][kat, h // group] += p.T @ do
    return {n: x if n == "lse" else x.flatten(1) for n, x in out.items()}
