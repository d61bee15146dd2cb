"""Cases that measure the operators around a training step's gradients: token
log probabilities and their gradient, the embedding lookup and its gradient,
and the orthogonalised (Muon) weight update.

Every case names one operator and its sizes.  ``run`` makes one pass: the
operator's plain form in elementary torch operations where ``own`` is false,
the calls a user makes of this package where it is true.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}

# the quintic Newton-Schulz step X <- a X + b (X X^T) X + c (X X^T)^2 X
STEPS, NS_A, NS_B, NS_C, NS_EPS = 5, 3.4445, -4.7750, 2.0315, 1e-7
MOMENTUM, WEIGHT_DECAY, LR = 0.95, 0.1, 5e-4


def listed():
    return [
        # one sequence decoding its next token: 8 alternatives at temperature 0.8; latency counts
        dict(name="logprobs, one token", op="logprobs", rows=1, vocab=131072, dtype="bf16", top=8, scale=1.25,
             banned=0.0),
        # a served batch scored from fp32 logits of an odd vocabulary, some tokens banned (-inf)
        dict(name="logprobs, served batch", op="logprobs", rows=48, vocab=100003, dtype="f32", top=20, scale=1.0,
             banned=0.001),
        # the loss of a training step: 8192 positions, entropy for monitoring, no alternatives
        dict(name="logprobs, training step", op="logprobs", rows=8192, vocab=32000, dtype="bf16", top=0, scale=1.0,
             banned=0.0),
        # the gradient of a 1000-class head on a batch of 256 images
        dict(name="logprobs gradient, classes", op="logprobs_grad", rows=256, vocab=1000, dtype="f16", scale=1.0),
        # the gradient of a training step over an odd vocabulary: every row starts at another alignment
        dict(name="logprobs gradient, tokens", op="logprobs_grad", rows=6145, vocab=50021, dtype="bf16", scale=1.0),
        # one decoding step of 64 sequences
        dict(name="embed, decoding step", op="embed", count=64, vocab=131072, dim=2048, dtype="bf16"),
        # a long prompt, or the inputs of a training step
        dict(name="embed, long prompt", op="embed", count=32768, vocab=65536, dim=4096, dtype="f16"),
        # a short training step with an odd width, the table's gradient in fp32
        dict(name="embed gradient, short", op="embed_grad", count=2048, vocab=10007, dim=1000, dtype="bf16",
             out="f32"),
        # a long training step, the table's gradient in the table's type
        dict(name="embed gradient, long", op="embed_grad", count=65536, vocab=32768, dim=4096, dtype="bf16",
             out="same"),
        # the update of three 3x3 filters of 64 -> 64 channels (64 x 576 matrices)
        dict(name="orthogonalise, 3x3 filters", op="orthogonalize", batch=3, rows=64, cols=576, dtype="bf16"),
        # the whole weight update of a 3x3 filter of 512 -> 512 channels (a 512 x 4608 matrix)
        dict(name="weight update, wide filter", op="muon_step", batch=1, rows=512, cols=4608, dtype="bf16"),
        # a large square weight
        dict(name="orthogonalise, large", op="orthogonalize", batch=1, rows=4096, cols=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "embed", "embed_grad", "orthogonalize", "muon_step"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("logprobs", "logprobs_grad"):
        vocab = _log(rng, 1000, 131072)
        rows = _log(rng, 1, min(8192, 500_000_000 // (vocab * SIZE[dtype])))
        case = dict(op=op, rows=rows, vocab=vocab, dtype=dtype, scale=rng.choice([1.0, 1.0, 0.7, 1.5]))
        if op == "logprobs":
            case.update(top=rng.choice([0, 1, 5, 20, 32]) if rows <= 1024 else 0,
                        banned=rng.choice([0.0, 0.0, 0.001, 0.3]))
        return case
    if op in ("embed", "embed_grad"):
        dim, vocab, count = _log(rng, 64, 4096), _log(rng, 1000, 32768), _log(rng, 1, 65536)
        case = dict(op=op, count=count, vocab=vocab, dim=dim, dtype=dtype)
        if op == "embed_grad":
            case.update(out=rng.choice(["same", "f32"]))
        return case
    rows, cols = _log(rng, 16, 3000), _log(rng, 16, 4608)
    batch = rng.choice([1, 1, 2, 4]) if rows * cols <= 1 << 20 else 1
    return dict(op=op, batch=batch, rows=rows, cols=cols, dtype=dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(g, count, vocab):
    """Token numbers with the frequencies of text (about 1/rank), one in fifty
    of them a padding position (-1)."""
    u = torch.rand(count, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    t[torch.rand(count, generator=g, device="cuda") < 0.02] = -1
    return t


def _gradient(g, batch, rows, cols):
    """A weight gradient's shape: a decaying spectrum over a floor of noise."""
    r = max(1, min(rows, cols) // 2)
    s = 1.0 / torch.arange(1, r + 1, device="cuda")
    left = torch.randn(batch, rows, r, generator=g, device="cuda") * s
    right = torch.randn(batch, r, cols, generator=g, device="cuda")
    noise = torch.randn(batch, rows, cols, generator=g, device="cuda") / math.sqrt(max(rows, cols))
    return 1e-3 * (left @ right / math.sqrt(max(rows, cols)) + 0.5 * noise)


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    f32 = dict(device="cuda", dtype=torch.float32)
    if op in ("logprobs", "logprobs_grad"):
        rows, vocab = case["rows"], case["vocab"]
        s["logits"] = torch.randn(rows, vocab, generator=g, device="cuda", dtype=dt) * 2.5
        targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        # the model has learnt something: the target stands out in most rows
        at = torch.arange(rows, device="cuda")
        s["logits"][at, targets] += (8.0 * torch.rand(rows, generator=g, device="cuda")).to(dt)
        if case.get("banned"):
            ban = torch.rand(rows, vocab, generator=g, device="cuda") < case["banned"]
            s["logits"].masked_fill_(ban, -math.inf)
        if rows > 1:  # positions without a target, as prompts and padding have
            targets[torch.rand(rows, generator=g, device="cuda") < 0.1] = -100
        s["targets"] = targets
        if op == "logprobs":
            s.update(logp=torch.empty(rows, **f32), lse=torch.empty(rows, **f32), entropy=torch.empty(rows, **f32))
            if case["top"]:
                s.update(top_ids=torch.empty(rows, case["top"], device="cuda", dtype=torch.int32),
                         top_logp=torch.empty(rows, case["top"], **f32))
        else:
            z = s["logits"].double() * case["scale"]
            lse = torch.logsumexp(z, 1)
            s["lse"] = lse.float()
            s["entropy"] = (lse - (torch.exp(z - lse[:, None]) * z).sum(1)).float()
            # the mean negative log probability, with a bonus for entropy
            s["g_logp"] = torch.full((rows,), -1.0 / rows, **f32) * (0.5 + torch.rand(rows, generator=g, device="cuda"))
            s["g_entropy"] = torch.full((rows,), 0.01 / rows, **f32)
            s["dlogits"] = torch.empty(rows, vocab, device="cuda", dtype=dt)
    elif op in ("embed", "embed_grad"):
        count, vocab, dim = case["count"], case["vocab"], case["dim"]
        s["tokens"] = _tokens(g, count, vocab)
        s["scale"] = math.sqrt(dim)
        if op == "embed":
            s["table"] = torch.randn(vocab, dim, generator=g, device="cuda", dtype=dt) * 0.02
            s["out"] = torch.empty(count, dim, device="cuda", dtype=dt)
        else:
            s["dout"] = torch.randn(count, dim, generator=g, device="cuda", dtype=dt) * 0.01
            odt = torch.float32 if case["out"] == "f32" else dt
            s["dtable"] = torch.empty(vocab, dim, device="cuda", dtype=odt)
            if own:
                import implicit_gemm_dgrad_gb300 as cdg
                s["workspace"] = torch.empty(cdg.embed_grad_workspace_bytes(count, vocab, dim), device="cuda",
                                             dtype=torch.uint8)
    else:
        batch, rows, cols = case["batch"], case["rows"], case["cols"]
        s["G"] = _gradient(g, batch, rows, cols).to(dt)
        if op == "orthogonalize":
            s["O"] = torch.empty_like(s["G"])
        else:
            s["W"] = torch.randn(batch, rows, cols, generator=g, device="cuda") * math.sqrt(2.0 / cols)
            s["M"] = _gradient(g, batch, rows, cols) * 8.0
            s["W_out"], s["M_out"] = torch.empty_like(s["W"]), torch.empty_like(s["M"])
            s["update_scale"] = 0.2 * math.sqrt(max(rows, cols))
        if own:
            import implicit_gemm_dgrad_gb300 as cdg
            s["plan"] = cdg.muon_plan(rows, cols, batch=batch, dtype=case["dtype"], steps=STEPS,
                                      coefficients=(NS_A, NS_B, NS_C), eps=NS_EPS)
            s["workspace"] = torch.empty(s["plan"].workspace_bytes, device="cuda", dtype=torch.uint8)
    return s


# ---- plain forms: elementary operations in 32 bits, rounded once at the end


def _plain_logprobs(s):
    z = s["logits"].float() * s["scale"]
    m = z.max(1, keepdim=True).values
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    lp = z - lse
    zero = torch.zeros((), device="cuda")
    entropy = -torch.where(lp > -math.inf, torch.exp(lp) * lp, zero).sum(1)
    t = s["targets"]
    has = (t >= 0) & (t < s["vocab"])
    logp = torch.where(has, lp.gather(1, t.clamp(0, s["vocab"] - 1)[:, None])[:, 0], zero)
    out = dict(logp=logp, lse=lse[:, 0], entropy=entropy)
    if s["top"]:
        ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :s["top"]]
        out.update(top_ids=ids.int(), top_logp=lp.gather(1, ids))
    return out


def _plain_logprobs_grad(s):
    lp = s["logits"].float() * s["scale"] - s["lse"][:, None]
    p = torch.exp(lp)
    t = s["targets"]
    has = (t >= 0) & (t < s["vocab"])
    g = torch.where(has, s["g_logp"], torch.zeros_like(s["g_logp"]))[:, None]
    d = -g * p - s["g_entropy"][:, None] * p * (lp + s["entropy"][:, None])
    d.scatter_add_(1, t.clamp(0, s["vocab"] - 1)[:, None], g)
    return (d * s["scale"]).to(s["dlogits"].dtype)


def _plain_embed(s):
    t = s["tokens"]
    has = (t >= 0) & (t < s["vocab"])
    rows = s["table"][t.clamp(0, s["vocab"] - 1)].float() * s["scale"]
    return torch.where(has[:, None], rows, torch.zeros((), device="cuda")).to(s["out"].dtype)


def _plain_embed_grad(s):
    t = s["tokens"]
    has = (t >= 0) & (t < s["vocab"])
    d = torch.zeros(s["vocab"], s["dim"], device="cuda")
    d.index_add_(0, t[has], s["dout"][has].float())
    return (d * s["scale"]).to(s["dtable"].dtype)


def _plain_orthogonal(u):
    flip = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if flip else u
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(STEPS):
        a = x @ x.transpose(1, 2)
        b = NS_B * a + NS_C * (a @ a)
        x = NS_A * x + b @ x
    return x.transpose(1, 2).contiguous() if flip else x


def _plain_muon_step(s):
    g = s["G"].float()
    m = MOMENTUM * s["M"] + g
    o = _plain_orthogonal(g + MOMENTUM * m)
    return dict(W=s["W"] * (1.0 - LR * WEIGHT_DECAY) - LR * s["update_scale"] * o, M=m)


def _run_plain(s):
    op = s["op"]
    if op == "logprobs":
        return _plain_logprobs(s)
    if op == "logprobs_grad":
        return _plain_logprobs_grad(s)
    if op == "embed":
        return _plain_embed(s)
    if op == "embed_grad":
        return _plain_embed_grad(s)
    if op == "orthogonalize":
        return _plain_orthogonal(s["G"].float()).to(s["G"].dtype)
    return _plain_muon_step(s)


def _run_own(s):
    import implicit_gemm_dgrad_gb300 as cdg
    op, dtype = s["op"], s["dtype"]
    if op == "logprobs":
        cdg.token_logprobs(s["logits"], s["targets"], s["logp"], s["lse"], s["rows"], s["vocab"], dtype,
                           scale=s["scale"], entropy=s["entropy"], top=s["top"], top_ids=s.get("top_ids"),
                           top_logp=s.get("top_logp"))
        return {k: s[k] for k in ("logp", "lse", "entropy", "top_ids", "top_logp") if k in s}
    if op == "logprobs_grad":
        cdg.token_logprobs_grad(s["logits"], s["targets"], s["lse"], s["entropy"], s["g_logp"], s["g_entropy"],
                                s["dlogits"], s["rows"], s["vocab"], dtype, scale=s["scale"])
        return s["dlogits"]
    if op == "embed":
        cdg.embed(s["table"], s["tokens"], s["out"], s["count"], s["vocab"], s["dim"], dtype, scale=s["scale"])
        return s["out"]
    if op == "embed_grad":
        cdg.embed_grad(s["dout"], s["tokens"], s["dtable"], s["workspace"], s["count"], s["vocab"], s["dim"], dtype,
                       scale=s["scale"], out_f32=s["dtable"].dtype == torch.float32)
        return s["dtable"]
    if op == "orthogonalize":
        s["plan"].orthogonalize(s["G"], s["O"], s["workspace"])
        return s["O"]
    s["plan"].step(s["W"], s["G"], s["M"], s["W_out"], s["M_out"], s["workspace"], lr=LR, momentum=MOMENTUM,
                   weight_decay=WEIGHT_DECAY, update_scale=s["update_scale"], nesterov=True)
    return dict(W=s["W_out"], M=s["M_out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Bytes: every input read once and every output written once.  Flops of
    the orthogonalisation: X X^T and (X X^T)^2 are symmetric, so half of each."""
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * e + case["rows"] * (20 + 8 * case["top"]), "flops": 6 * n}
    if op == "logprobs_grad":
        n = case["rows"] * case["vocab"]
        return {"bytes": 2 * n * e + 24 * case["rows"], "flops": 6 * n}
    if op == "embed":
        n = case["count"] * case["dim"]
        return {"bytes": 2 * n * e + 8 * case["count"], "flops": n}
    if op == "embed_grad":
        n = case["count"] * case["dim"]
        out = 4 if case["out"] == "f32" else e
        return {"bytes": n * e + case["vocab"] * case["dim"] * out + 8 * case["count"], "flops": n}
    m, n = sorted((case["rows"], case["cols"]))
    flops = case["batch"] * STEPS * (3 * m * m * n + m * m * m)
    moved = (2 * e if op == "orthogonalize" else 16 + e) * case["batch"] * m * n
    return {"bytes": moved, "flops": flops}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        z = s["logits"].double() * case["scale"]
        lse = torch.logsumexp(z, dim=1)
        lp = z.sub_(lse[:, None])
        entropy = torch.special.entr(torch.exp(lp)).sum(1)
        logp = torch.zeros(case["rows"], device="cuda", dtype=torch.float64)
        at = torch.nonzero((s["targets"] >= 0) & (s["targets"] < case["vocab"]))[:, 0]
        logp[at] = lp[at, s["targets"][at]]
        out = dict(logp=logp, lse=lse, entropy=entropy)
        if case["top"]:
            ids = torch.argsort(-s["logits"].double(), dim=1, stable=True)[:, :case["top"]]
            out.update(top_ids=ids.int(), top_logp=torch.take_along_dim(lp, ids, 1))
        return out
    if op == "logprobs_grad":
        # d/dz_j of g log p_t + h H with z = scale * logits and the given lse and H
        lp = (s["logits"].double() * case["scale"]).sub_(s["lse"].double()[:, None])
        at = torch.nonzero((s["targets"] >= 0) & (s["targets"] < case["vocab"]))[:, 0]
        g = torch.zeros(case["rows"], device="cuda", dtype=torch.float64)
        g[at] = s["g_logp"].double()[at]
        weight = g[:, None] + s["g_entropy"].double()[:, None] * (lp + s["entropy"].double()[:, None])
        d = weight.mul_(lp.exp_()).neg_()
        d[at, s["targets"][at]] += g[at]
        return d.mul_(case["scale"])
    if op == "embed":
        at = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
        out = torch.zeros(case["count"], case["dim"], device="cuda", dtype=torch.float64)
        out[at] = s["table"][s["tokens"][at]].double() * math.sqrt(case["dim"])
        return out
    if op == "embed_grad":
        # sums over runs of equal tokens in sorted order, as differences of a running sum
        tokens, order = torch.sort(s["tokens"])
        first = int((tokens < 0).sum())
        tokens, order = tokens[first:], order[first:]
        out = torch.zeros(case["vocab"], case["dim"], device="cuda", dtype=torch.float64)
        if tokens.numel():
            run_sum = torch.cumsum(s["dout"][order].double(), 0)
            ids, counts = torch.unique_consecutive(tokens, return_counts=True)
            ends = run_sum[torch.cumsum(counts, 0) - 1]
            ends[1:] -= ends[:-1].clone()
            out[ids] = ends * math.sqrt(case["dim"])
        return out
    g = s["G"].double()
    m = None
    if op == "muon_step":
        m = MOMENTUM * s["M"].double() + g
        g = g + MOMENTUM * m
    # the iteration as a polynomial of the Gram matrix on the smaller side
    tall = g.shape[1] > g.shape[2]
    x = g / (torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True) + NS_EPS)
    eye = torch.eye(min(g.shape[1], g.shape[2]), device="cuda", dtype=torch.float64)
    for _ in range(STEPS):
        gram = x.mT @ x if tall else x @ x.mT
        p = NS_A * eye + (NS_B * eye + NS_C * gram) @ gram
        x = x @ p if tall else p @ x
    if op == "orthogonalize":
        return x
    return dict(W=s["W"].double() * (1.0 - LR * WEIGHT_DECAY) - LR * s["update_scale"] * x, M=m)
