"""A stack of ternary blocks from its training step to its served tokens.

Each block is one ternary projection between two norms:

    n = w_pre * h^;   y = n (T alpha)^T;   h <- res_scale h + gate * (w_post * y^)

Training runs the blocks on fake-quantized latent weights (straight-through
gradients), with `block_norm_ad` forward and backward around each projection
and `muon_step` on the latent weights.  Serving packs the weights once and runs
prompts through `adapter_gemm` and single tokens through `adapter_gemv`, each
request with an adapter of its own beside the shared packed weight.

    python examples/ternary_blocks.py [--dim 512] [--blocks 3] [--steps 30]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_quantization_sparse_amd as S  # noqa: E402

RES_SCALE = 0.9
BF16 = torch.bfloat16


class Blocks:
    """Latent weights, norm weights and gates of a stack, with momenta."""

    def __init__(self, dim, blocks, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.dim = dim
        self.w = [torch.randn(dim, dim, generator=g, device=device) * 0.02 for _ in range(blocks)]
        self.buf = [torch.zeros_like(w) for w in self.w]
        ones = torch.ones(dim, device=device)
        self.w_pre = [ones.clone() for _ in range(blocks + 1)]      # the last one ends the stack
        self.w_post = [ones.clone() for _ in range(blocks)]
        self.gate = [torch.full((dim,), 0.5, device=device, dtype=BF16) for _ in range(blocks)]

    def small(self):
        return [*self.w_pre, *self.w_post, *self.gate]


def forward(net, h, project, norm):
    """The stack on tokens ``h`` [M, D]: ``project(i, n)`` is block i's projection."""
    h, n = norm(h, net.w_pre[0])
    for i in range(len(net.w)):
        h, n = norm(h, net.w_pre[i + 1], y=project(i, n), w_post=net.w_post[i], gate=net.gate[i], res_scale=RES_SCALE)
    return n


def train_step(net, h, target, lr, small_lr):
    """One step on latent weights; returns the loss."""
    for t in (*net.w, *net.small()):
        t.requires_grad_(True)
    out = forward(net, h, lambda i, n: n @ S.fake_quant_ste(net.w[i]).to(BF16).t(), S.block_norm_ad)
    loss = (out.float() - target).pow(2).mean()
    grads = torch.autograd.grad(loss, [*net.w, *net.small()])
    with torch.no_grad():
        for t in (*net.w, *net.small()):
            t.requires_grad_(False)
        for i, g in enumerate(grads[:len(net.w)]):
            S.muon_step(net.w[i], g, net.buf[i], lr, weight_decay=0.01, out=(net.w[i], net.buf[i]))
        for t, g in zip(net.small(), grads[len(net.w):]):
            t -= small_lr * g
    return float(loss.detach())


def train(net, teacher, steps, tokens, lr=0.02, small_lr=0.05, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(tokens, net.dim, generator=g, device="cuda").to(BF16)
    target = forward(teacher, h, lambda i, n: n @ S.fake_quant(teacher.w[i])[0].to(BF16).t(), S.block_norm).float()
    return [train_step(net, h, target, lr, small_lr) for _ in range(steps)]


class Served:
    """The packed stack with one adapter set a block."""

    def __init__(self, net, requests, rank=16, seed=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.net = net
        self.packed = [S.quantize_pack(w) for w in net.w]
        d = net.dim
        self.adapters = [S.AdapterSet((torch.randn(requests, rank, d, generator=g, device="cuda") * d ** -0.5).to(BF16),
                                      (torch.randn(requests, d, rank, generator=g, device="cuda") * 0.05).to(BF16),
                                      torch.ones(requests, device="cuda")) for _ in net.w]

    def __call__(self, h, ids):
        """Tokens ``h`` [M, D] of requests ``ids`` [M] (-1: no adapter)."""
        run = S.adapter_gemv if h.shape[0] <= 16 else S.adapter_gemm
        return forward(self.net, h, lambda i, n: run(self.packed[i], n, self.adapters[i], ids), S.block_norm)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--dim", type=int, default=512)
    p.add_argument("--blocks", type=int, default=3)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--tokens", type=int, default=256)
    a = p.parse_args(argv)
    net, teacher = Blocks(a.dim, a.blocks, seed=0), Blocks(a.dim, a.blocks, seed=7)
    losses = train(net, teacher, a.steps, a.tokens)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Served(net, requests=3)
    h = torch.randn(a.tokens, a.dim, device="cuda").to(BF16)
    ids = torch.arange(a.tokens, device="cuda", dtype=torch.int32) * 4 // a.tokens - 1   # -1, 0, 1, 2 in runs
    prompt = served(h, ids)
    pick = torch.linspace(0, a.tokens - 1, 8, device="cuda").long()                      # one decode batch of 8
    decoded = served(h[pick], ids[pick].contiguous())
    diff = float((decoded.float() - prompt[pick].float()).norm() / prompt[pick].float().norm())
    print(f"{a.tokens} prompt tokens, 8 decoded ones: relative difference {diff:.1e}")
    return losses, diff


if __name__ == "__main__":
    main()
