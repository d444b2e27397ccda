"""Feed-forward blocks of ternary weights, distilled from a teacher's top
logits and served packed: a dense block, then one of experts.

    h += down f(gate n) * (up n)            n = norm(h), one weight or the top_k of several experts
    logits = head norm(h)

Training runs on fake-quantized latent weights (straight-through gradients)
with `distill_loss_ad` on the logits and `muon_step` on the latent weights.
Serving packs them: prompts go through `linear_gemm` (gate and up as one
weight, the residual in the epilogue of down), single tokens through
`linear_gemv`, and the experts through `moe_decode`, 16 tokens at a time.

    python examples/distilled_experts.py [--dim 256] [--vocab 1000] [--steps 10]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ternary_weight_quantization_sparse_amd as S  # noqa: E402

BF16 = torch.bfloat16
TOP_K, SLOTS, TEMPERATURE, KD_WEIGHT = 2, 8, 2.0, 0.7


class Model:
    """Latent weights; gate and up of a block are the halves of one weight."""

    def __init__(self, dim, hidden, experts, vocab, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=device) * 0.05

        self.dim, self.experts = dim, experts
        self.ternary = [weight(2 * hidden, dim), weight(dim, hidden)]                  # the dense block
        self.ternary += [weight(2 * hidden, dim) for _ in range(experts)] + [weight(dim, hidden) for _ in range(experts)]
        self.buf = [torch.zeros_like(w) for w in self.ternary]
        self.router, self.head = weight(experts, dim), weight(vocab, dim)
        self.norms = [torch.ones(dim, device=device) for _ in range(3)]

    def expert_weights(self):
        return self.ternary[2:2 + self.experts], self.ternary[2 + self.experts:]


def feed_forward(n, up, down):
    gate, value = (n @ S.fake_quant_ste(up).to(BF16).t()).chunk(2, -1)
    return (torch.nn.functional.silu(gate) * value) @ S.fake_quant_ste(down).to(BF16).t()


def train_logits(net, h):
    """Student logits of tokens ``h`` [T, D] on the fake-quantized weights."""
    h, n = S.block_norm_ad(h, net.norms[0])
    h = h + feed_forward(n, *net.ternary[:2])
    h, n = S.block_norm_ad(h, net.norms[1])
    score = (n.float() @ net.router.t()).softmax(-1)
    best = score.topk(TOP_K, -1)
    weight = torch.zeros_like(score).scatter(1, best.indices, best.values / best.values.sum(-1, keepdim=True))
    for e, (up, down) in enumerate(zip(*net.expert_weights())):
        h = h + weight[:, e:e + 1].to(BF16) * feed_forward(n, up, down)
    return S.block_norm_ad(h, net.norms[2])[1] @ net.head.to(BF16).t()


def teacher_of(logits):
    """What is kept of a teacher's logits: the largest, their ids, and the normaliser of all."""
    top, ids = logits.float().topk(SLOTS, -1)
    return top, ids, torch.logsumexp(logits.float() / TEMPERATURE, -1)


def loss_of(logits, teacher, labels):
    top, ids, lse = teacher
    return S.distill_loss_ad(logits, top, ids, temperature=TEMPERATURE, teacher_lse=lse, labels=labels,
                             kd_weight=KD_WEIGHT).mean()


def train_step(net, h, teacher, labels, lr):
    for w in net.ternary:
        w.requires_grad_(True)
    loss = loss_of(train_logits(net, h), teacher, labels)
    grads = torch.autograd.grad(loss, net.ternary)
    with torch.no_grad():
        for w in net.ternary:
            w.requires_grad_(False)
        for w, g, b in zip(net.ternary, grads, net.buf):
            S.muon_step(w, g, b, lr, out=(w, b))
    return float(loss.detach())


class Served:
    """The packed model."""

    def __init__(self, net):
        self.net = net
        self.up, self.down = (S.quantize_pack(w) for w in net.ternary[:2])
        ups, downs = net.expert_weights()
        self.ups, self.downs = S.quantize_pack_experts(torch.stack(ups)), S.quantize_pack_experts(torch.stack(downs))

    def __call__(self, h):
        net = self.net
        run = S.linear_gemv if h.shape[0] <= 16 else S.linear_gemm
        h, n = S.block_norm(h, net.norms[0])
        h = run(self.down, run(self.up, n, activation="silu", gated=True), residual=h)
        h, n = S.block_norm(h, net.norms[1])
        out = torch.empty_like(h)
        for t in range(0, h.shape[0], 16):
            S.moe_decode(n[t:t + 16], net.router, self.ups, self.downs, TOP_K, residual=h[t:t + 16], out=out[t:t + 16])
        return S.block_norm(out, net.norms[2])[1] @ net.head.to(BF16).t()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--dim", type=int, default=256)
    p.add_argument("--hidden", type=int, default=512)
    p.add_argument("--experts", type=int, default=6)
    p.add_argument("--vocab", type=int, default=1000)
    p.add_argument("--tokens", type=int, default=200)
    p.add_argument("--steps", type=int, default=10)
    a = p.parse_args(argv)
    net, teacher = (Model(a.dim, a.hidden, a.experts, a.vocab, seed) for seed in (0, 7))
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(a.tokens, a.dim, generator=g, device="cuda").to(BF16)
    with torch.no_grad():
        wanted = train_logits(teacher, h)
    labels = wanted.argmax(-1)
    losses = [train_step(net, h, teacher_of(wanted), labels, 0.02) for _ in range(a.steps)]
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Served(net)
    prompt = served(h)
    pick = torch.linspace(0, a.tokens - 1, 8, device="cuda").long()
    decoded = served(h[pick])
    diff = float((decoded.float() - prompt[pick].float()).norm() / prompt[pick].float().norm())
    print(f"{a.tokens} prompt tokens, 8 decoded ones: relative difference {diff:.1e}")
    return losses, diff, served, prompt


if __name__ == "__main__":
    main()
