"""Train a small next-token model with this library alone.

    python examples/train_tokens.py [--steps 60] [--tokens 4096] [--vocab 512] [--dim 128]

The model maps a token to the logits of the next one:

    h = scale * E[token]            cdg.embed
    a = relu(h W1^T)                a 1x1 layer: its forward is a dgrad with the roles of the channels swapped
    z = a W2^T                      another

and a step is

    logp, lse, entropy              cdg.token_logprobs
    dz                              cdg.token_logprobs_grad (of the mean negative log probability, less a little entropy)
    da, gated by a > 0              dgrad of the output layer with the fused ReLU backward
    dW2, dW1                        cdg wgrad
    dh                              dgrad of the hidden layer
    dE                              cdg.embed_grad (sorted tokens)
    W1                              cdg.MuonPlan.step, W2 and E by plain SGD

Every product, sum and update of the step runs in the library's kernels but the
SGD updates, the ReLU of the forward pass and the casts of the weights, which are
torch's.  The data: a fixed random permutation of the vocabulary, which the
model learns (token t is followed by next[t]), with one position in 16 left
without a target.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_dgrad_gb300 as cdg  # noqa: E402


class Linear:
    """A 1x1 layer on rows x inputs: y = x W^T, with W [outputs][inputs] in fp32
    and its bf16 copies packed for the two dgrads (forward and backward)."""

    def __init__(self, rows, inputs, outputs, gated=False):
        self.rows, self.inputs, self.outputs = rows, inputs, outputs
        # dgrad computes dX[n, c] = sum over k of dY[n, k] W[k, c]: the forward
        # pass takes x for dY and W^T [inputs][outputs] for W
        self.fwd = cdg.plan(rows, 1, 1, outputs, inputs, 1, 1, dtype="bf16")
        self.bwd = cdg.plan(rows, 1, 1, inputs, outputs, 1, 1, dtype="bf16", relu=gated)
        self.wgrad = cdg.wgrad_plan(rows, 1, 1, inputs, outputs, 1, 1, dtype="bf16")
        b16 = dict(dtype=torch.bfloat16, device="cuda")
        self.W = torch.randn(outputs, inputs, device="cuda") * math.sqrt(1.0 / inputs)
        self.Wf, self.Wb = torch.empty(inputs * outputs, **b16), torch.empty(inputs * outputs, **b16)
        self.dW = torch.empty(outputs, inputs, **b16)
        self.ws = torch.empty(self.wgrad.workspace_bytes, dtype=torch.uint8, device="cuda")
        self.pack()

    def pack(self):
        w = self.W.bfloat16()
        self.fwd.prepack_weights(w.t().contiguous(), self.Wf)
        self.bwd.prepack_weights(w, self.Wb)

    def status(self):
        return max(p.device_status() for p in (self.fwd, self.bwd, self.wgrad))


def train(steps=60, tokens=4096, vocab=512, dim=128, seed=0, lr=0.005, log=None):
    """Returns the mean negative log probability before every step."""
    torch.manual_seed(seed)
    b16 = dict(dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    scale = math.sqrt(dim)
    E = (torch.randn(vocab, dim, device="cuda") / scale).bfloat16()
    hidden, out = Linear(tokens, dim, dim), Linear(tokens, dim, vocab, gated=True)
    M = torch.zeros(dim, dim, **f32)
    muon = cdg.muon_plan(dim, dim, dtype="bf16")
    muon_ws = torch.empty(muon.workspace_bytes, dtype=torch.uint8, device="cuda")
    following = torch.randperm(vocab, device="cuda")
    h, a, da, dh = (torch.empty(tokens, dim, **b16) for _ in range(4))
    z, dz = torch.empty(tokens, vocab, **b16), torch.empty(tokens, vocab, **b16)
    logp, lse, entropy = (torch.empty(tokens, **f32) for _ in range(3))
    dE = torch.empty(vocab, dim, **f32)
    embed_ws = torch.empty(cdg.embed_grad_workspace_bytes(tokens, vocab, dim), dtype=torch.uint8, device="cuda")
    losses = []
    for step in range(steps):
        token = torch.randint(0, vocab, (tokens,), device="cuda")
        target = following[token]
        target[::16] = -1
        count = int((target >= 0).sum())
        # forward
        cdg.embed(E, token, h, tokens, vocab, dim, "bf16", scale=scale)
        hidden.fwd.dgrad(h, hidden.Wf, a)
        a.relu_()
        out.fwd.dgrad(a, out.Wf, z)
        cdg.token_logprobs(z, target, logp, lse, tokens, vocab, "bf16", entropy=entropy)
        losses.append(float(-logp.sum() / count))
        if log and step % 10 == 0:
            log(f"step {step:4d}  loss {losses[-1]:.4f}  entropy {float(entropy.mean()):.4f}")
        # backward
        g = torch.full((tokens,), -1.0 / count, **f32)
        ge = torch.full((tokens,), -1e-4 / tokens, **f32)
        cdg.token_logprobs_grad(z, target, lse, entropy, g, ge, dz, tokens, vocab, "bf16")
        out.bwd.dgrad(dz, out.Wb, da, a)  # gated by a > 0
        out.wgrad.wgrad(dz, a, out.dW, out.ws)
        hidden.bwd.dgrad(da, hidden.Wb, dh)
        hidden.wgrad.wgrad(da, h, hidden.dW, hidden.ws)
        cdg.embed_grad(dh, token, dE, embed_ws, tokens, vocab, dim, "bf16", scale=scale, out_f32=True)
        # update
        muon.step(hidden.W, hidden.dW, M, hidden.W, M, muon_ws, lr=lr, momentum=0.9, weight_decay=0.01,
                  update_scale=0.2 * math.sqrt(dim))
        out.W -= 20 * lr * out.dW.float() * vocab
        E -= (lr * dE).bfloat16()
        hidden.pack()
        out.pack()
    status = max(hidden.status(), out.status(), muon.device_status())
    if status != cdg.OK:
        raise cdg.CdgError(status, "train")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="Train a small next-token model with this library alone.")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--dim", type=int, default=128)
    args = ap.parse_args()
    losses = train(args.steps, args.tokens, args.vocab, args.dim, log=print)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
