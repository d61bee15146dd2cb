"""GPU test of the token operators and the weight update in a CUDA graph: one
step's calls captured together (their launches overlap each other's starts),
replayed on other inputs, give the bits that the calls give one by one."""
import pytest

import implicit_gemm_dgrad_gb300 as cdg

pytestmark = pytest.mark.gpu


class Step:
    """Lookup, log probabilities, their gradient, the table's gradient and two weight updates."""

    def __init__(self, count, vocab, dim, rows, cols):
        import torch
        self.count, self.vocab, self.dim = count, vocab, dim
        b16, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
        self.table, self.out = torch.empty(vocab, dim, **b16), torch.empty(count, dim, **b16)
        self.tokens = torch.empty(count, dtype=torch.int64, device="cuda")
        self.logits, self.d = torch.empty(count, vocab, **b16), torch.empty(count, vocab, **b16)
        self.rows = [torch.empty(count, **f32) for _ in range(5)]  # logp, lse, entropy, g, h
        self.ids, self.top = torch.empty(count, 3, dtype=torch.int32, device="cuda"), torch.empty(count, 3, **f32)
        self.dtable = torch.empty(vocab, dim, **f32)
        self.ws = torch.empty(cdg.embed_grad_workspace_bytes(count, vocab, dim), dtype=torch.uint8, device="cuda")
        self.plans = [cdg.muon_plan(rows, cols), cdg.muon_plan(min(rows, 96), cols)]
        self.mats = []
        for p in self.plans:
            shape = (p.shape["rows"], p.shape["cols"])
            self.mats.append(dict(W=torch.empty(shape, **f32), G=torch.empty(shape, **b16), M=torch.empty(shape, **f32),
                                  Wo=torch.empty(shape, **f32), Mo=torch.empty(shape, **f32),
                                  ws=torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")))

    def fill(self, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table.normal_(generator=g)
        self.tokens.copy_(torch.randint(-1, self.vocab, (self.count,), generator=g, device="cuda"))
        self.tokens[: self.count // 3] = seed % self.vocab
        self.logits.normal_(generator=g)
        for r in self.rows[3:]:
            r.normal_(generator=g)
        for m in self.mats:
            for k in "WGM":
                m[k].normal_(generator=g)

    def run(self):
        n, v, d = self.count, self.vocab, self.dim
        logp, lse, entropy, g, h = self.rows
        cdg.embed(self.table, self.tokens, self.out, n, v, d, scale=1.5)
        cdg.token_logprobs(self.logits, self.tokens, logp, lse, n, v, entropy=entropy, top=3, top_ids=self.ids, top_logp=self.top)
        cdg.token_logprobs_grad(self.logits, self.tokens, lse, entropy, g, h, self.d, n, v)
        cdg.embed_grad(self.out, self.tokens, self.dtable, self.ws, n, v, d, out_f32=True)
        for p, m in zip(self.plans, self.mats):
            p.step(m["W"], m["G"], m["M"], m["Wo"], m["Mo"], m["ws"], lr=0.1)

    def outputs(self):
        outs = [self.out, *self.rows[:3], self.ids, self.top, self.d, self.dtable]
        for m in self.mats:
            outs += [m["Wo"], m["Mo"]]
        return outs


@pytest.mark.parametrize("count,vocab,dim,rows,cols", [(200, 1000, 72, 130, 257), (5000, 3001, 256, 512, 640), (1, 70001, 8, 40, 24)])
def test_a_captured_step_replays(count, vocab, dim, rows, cols):
    import torch
    step = Step(count, vocab, dim, rows, cols)
    step.fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.run()
    for seed in range(1, 6):
        step.fill(seed)
        step.run()
        want = [t.clone() for t in step.outputs()]
        for t in step.outputs():
            t.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert all(p.device_status() == 0 for p in step.plans)
        for k, (a, b) in enumerate(zip(step.outputs(), want)):
            assert torch.equal(a, b), (seed, k)
