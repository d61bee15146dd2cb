"""The attention and the rotation of queries and keys in 64 bits, written from
their definitions, with the error bounds that the GPU tests hold results to.

Bounds count roundings: u = eps / 2 of the 16-bit type for every operand and
output rounded to it, 2^-24 for every fp32 operation, and half the smallest
subnormal where fp16 values underflow.
"""
import math

import torch

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}  # half the smallest subnormal
U32 = 2.0 ** -24
FLUSH = 2.0 ** -126  # the fp32 exponential answers 0 below this: a probability under it is off by itself
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def visible(n, kn, causal, window):
    r = torch.arange(n)[:, None] + (kn - n)
    j = torch.arange(kn)
    see = torch.ones(n, kn, dtype=torch.bool)
    if causal:
        see &= j <= r
    if window:
        see &= j > r - window
    return see


def forward(q, k, v, causal, window, scale, dtype):
    """q (n, D), k and v (m, D) of one head in 64 bits: o, lse, and their bounds."""
    n, m, dim = q.shape[0], k.shape[0], q.shape[1]
    see = visible(n, m, causal, window)
    s = torch.where(see, q @ k.T * scale, -math.inf)
    lse = torch.logsumexp(s, 1) if m else torch.full((n,), -math.inf, dtype=q.dtype)
    p = torch.where(see, torch.exp(s - lse[:, None]), 0.0)
    o = p @ v
    u = U[dtype]
    # a score: dim fp32 additions and the scaling; its exponential's argument is rounded, and 2^x is good to 2^-22
    e_s = (dim + 4) * U32 * scale * (q.abs() @ k.abs().T) if m else torch.zeros(n, m)
    top = torch.where(see, s.abs() + e_s, 0.0).amax(1) if m else torch.zeros(n)
    e_p = 2 * (e_s.amax(1) if m else torch.zeros(n)) + 8 * U32 * (top + 4) + (m + 16) * U32
    weight = p @ v.abs()
    # fp16: p about the running reference is at least 1 at the maximum, its small values underflow
    far = (TINY[dtype] + FLUSH) * (v.abs().sum(0) if m else torch.zeros(dim))
    tol_o = u * o.abs() + (u + e_p[:, None]) * (1 + u) * weight + (1 + u) * far + TINY[dtype]
    tol_lse = e_p + 8 * U32 * (lse.abs().nan_to_num(0, 0, 0) + 1)
    return o, lse, tol_o, tol_lse


def gradient(q, k, v, o, lse, do, causal, window, scale, dtype):
    """dq, dk, dv of one head for the given o and lse, and their bounds."""
    n, m, dim = q.shape[0], k.shape[0], q.shape[1]
    see = visible(n, m, causal, window)
    empty = torch.isinf(lse)
    ref = torch.where(empty, 0.0, lse)
    s = q @ k.T * scale
    p = torch.where(see & ~empty[:, None], torch.exp(s - ref[:, None]), 0.0)
    dp, total = do @ v.T, (do * o).sum(1, keepdim=True)
    ds = p * (dp - total)
    u, tiny = U[dtype], TINY[dtype]
    e_s = (dim + 4) * U32 * scale * (q.abs() @ k.abs().T)
    e_p = e_s + 8 * U32 * (s.abs() + ref.abs()[:, None] + 4)
    e_dp = (dim + 4) * U32 * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True))
    err_p = p * (u + e_p) * (1 + u) + tiny + FLUSH
    err_ds = (p * (e_p * (dp - total).abs() + e_dp) + (u + 4 * U32) * ds.abs()) * (1 + u) + tiny + FLUSH * (1 + (dp - total).abs())

    def out(value, err, grown):
        return (u + 4 * U32) * value.abs() + err + grown + tiny

    dq, dk, dv = ds @ k * scale, ds.T @ q * scale, p.T @ do
    return ((dq, dk, dv),
            (out(dq, scale * (err_ds @ k.abs()), scale * (m + 8) * U32 * (ds.abs() @ k.abs())),
             out(dk, scale * (err_ds.T @ q.abs()), scale * (n + 8) * U32 * (ds.abs().T @ q.abs())),
             out(dv, err_p.T @ do.abs(), (n + 8) * U32 * (p.T @ do.abs()))))


def rotate(x, positions, inv_freq, rot, interleaved, factor, norm, eps, w):
    """(tokens, heads, dim) in 64 bits."""
    if norm:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * (1.0 if w is None else w)
    half = rot // 2
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = factor * torch.cos(angle)[:, None], factor * torch.sin(angle)[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)
