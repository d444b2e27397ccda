"""The operators together, as the example uses them, and each inside a HIP
graph: one capture, several replays on new inputs with eager work between
them, each equal to the eager call bit for bit (every sum has a fixed order)."""

import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
S = pytest.importorskip("ternary_weight_quantization_sparse_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    S.load()


def example():
    spec = importlib.util.spec_from_file_location("distilled_experts", os.path.join(ROOT, "examples", "distilled_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    m = example()
    losses, diff, served, prompt = m.main(["--dim", "256", "--hidden", "256", "--steps", "3", "--tokens", "50"])
    assert all(l == l and abs(l) < 1e4 for l in losses) and prompt.shape == (50, 1000) and prompt.isfinite().all()
    # a token alone and inside its prompt: three roundings of the stream to bf16 apart at most, and a
    # norm; a choice of experts that differs for it would be far more
    assert diff < 2.0 ** -6


def test_example_gradient():
    """The gradient of the example's loss with respect to a latent weight, against the same model with the loss written
    in elementary operations (both run the model in bf16, the loss in fp32: its gradient is rounded to bf16 once)."""
    m = example()
    net, teacher = m.Model(128, 128, 3, 500, 0), m.Model(128, 128, 3, 500, 7)
    h = torch.randn(40, 128, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF16)
    with torch.no_grad():
        wanted = m.train_logits(teacher, h)
    top, ids, lse = m.teacher_of(wanted)
    labels = wanted.argmax(-1)
    for w in net.ternary:
        w.requires_grad_(True)
    logits = m.train_logits(net, h)
    got = torch.autograd.grad(m.loss_of(logits, (top, ids, lse), labels), logits, retain_graph=True)[0]

    z = logits.detach().double().requires_grad_(True)
    logq = (z / m.TEMPERATURE).log_softmax(-1)
    p = torch.exp(top.double() / m.TEMPERATURE - lse.double()[:, None])
    rest = 1 - p.sum(-1)
    mask = torch.zeros_like(z, dtype=torch.bool).scatter(1, ids, True)
    kd = (p * (p.log() - logq.gather(1, ids))).sum(-1)
    kd = kd + rest * (rest.log() - logq.masked_fill(mask, -float("inf")).logsumexp(-1))
    hard = -z.log_softmax(-1).gather(1, labels[:, None])[:, 0]
    loss = (m.KD_WEIGHT * m.TEMPERATURE ** 2 * kd + (1 - m.KD_WEIGHT) * hard).mean()
    want = torch.autograd.grad(loss, z)[0]
    # half a step of bf16, and 2^-18 of terms of at most w t + (1 - w) = 1.7 over 40 rows
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * 1.7 / 40).all()
    # and on to the weights: both gradients of the logits through the same graph, bf16 products of 40 tokens
    a = torch.autograd.grad(logits, net.ternary, got, retain_graph=True)
    b = torch.autograd.grad(logits, net.ternary, want.to(BF16))
    for x, y in zip(a, b):
        assert x.isfinite().all() and float((x - y).norm()) <= 2.0 ** -5 * float(y.norm()) + 1e-12


def test_served_equals_the_dense_model():
    """The packed model against the fake-quantized one on the same tokens: the dense path rounds its inner activations and
    its weights to bf16, so a relative difference of a few bf16 steps."""
    m = example()
    net = m.Model(256, 384, 5, 300, 0)
    h = torch.randn(33, 256, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(BF16)
    with torch.no_grad():
        dense = m.train_logits(net, h).float()
    served = m.Served(net)(h).float()
    assert float((served - dense).norm() / dense.norm()) < 2.0 ** -5


# ------------------------------------------------------------------- graphs
def rand(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def replays(call, inputs, fresh):
    """Captures call(*inputs); replays it on the inputs that fresh(i) makes."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*inputs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*inputs)
    for i in range(4):
        for t, new in zip(inputs, fresh(i)):
            t.copy_(new)
        want = [t.clone() for t in call(*inputs)]     # eager, on the same inputs
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


@pytest.mark.parametrize("tokens,n,k,gated", [(1, 512, 1024, False), (9, 300, 2048, True), (16, 16384, 512, True),
                                              (70, 384, 2048, True), (300, 1000, 512, False)])
def test_linear_in_a_graph(tokens, n, k, gated):
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    pw, b = S.quantize_pack(rand(gen, n, k) * 0.02), rand(gen, n)
    f = S.linear_gemv if tokens <= 16 else S.linear_gemm

    def fresh(i):
        return [rand(gen, tokens, k, dtype=BF16), rand(gen, tokens, n // 2 if gated else n, dtype=BF16)]
    replays(lambda x, r: [f(pw, x, bias=b, activation="gelu", gated=gated, residual=r)], fresh(0), fresh)


@pytest.mark.parametrize("tokens,n,k,gated", [(260, 2050, 8192, False), (2050, 4096, 1024, True)])
def test_long_prompt_in_a_graph(tokens, n, k, gated):
    """The kernel of many tiles, with K split and not."""
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    pw, b = S.quantize_pack(rand(gen, n, k) * 0.02), rand(gen, n)

    def fresh(i):
        return [rand(gen, tokens, k, dtype=BF16), rand(gen, tokens, n // 2 if gated else n, dtype=BF16)]
    replays(lambda x, r: [S.linear_gemm(pw, x, bias=b, activation="silu", gated=gated, residual=r)], fresh(0), fresh)


@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden", [(1, 8, 2, 512, 1024), (16, 40, 4, 2048, 512), (5, 200, 8, 256, 256)])
def test_experts_in_a_graph(tokens, experts, top_k, dim, hidden):
    """The experts in use change from replay to replay."""
    gen = torch.Generator(device=DEV).manual_seed(experts)
    up = S.quantize_pack_experts(rand(gen, experts, 2 * hidden, dim) * 0.05)
    down = S.quantize_pack_experts(rand(gen, experts, dim, hidden) * 0.05)
    router = rand(gen, experts, dim) * 0.05

    def fresh(i):
        return [rand(gen, tokens, dim, dtype=BF16), rand(gen, tokens, dim, dtype=BF16)]
    replays(lambda x, r: [S.moe_decode(x, router, up, down, top_k, residual=r)], fresh(0), fresh)


@pytest.mark.parametrize("rows,vocab,dtype,tail", [(1, 70000, BF16, True), (40, 3001, F32, False), (2100, 50000, BF16, True)])
def test_distillation_in_a_graph(rows, vocab, dtype, tail):
    gen = torch.Generator(device=DEV).manual_seed(vocab)

    def fresh(i):
        z = rand(gen, rows, vocab, dtype=dtype)
        u, ids = z.float().topk(16, 1)
        return [z, u + 0.1 * rand(gen, rows, 16), ids, torch.logsumexp(z.float() / 2, 1) + 0.5, rand(gen, rows)]

    def call(z, u, ids, lse, g):
        kw = dict(temperature=2.0, labels=ids[:, 3], kd_weight=0.6)
        loss, stats = S.distill_loss(z, u, ids, teacher_lse=lse if tail else None, with_stats=True, **kw)
        return [loss, stats, S.distill_loss_backward(g, z, ids, stats, **kw)]
    replays(call, fresh(0), fresh)


def test_captured_training_step_beside_an_eager_one():
    """The loss and its gradient captured while an eager graph of the same leaf lives, and both used."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    z = rand(gen, 32, 4000, dtype=BF16).requires_grad_(True)
    u, ids = z.detach().float().topk(8, 1)
    g = torch.full((32,), 1 / 32, device=DEV)
    eager = S.distill_loss_ad(z, u, ids, temperature=2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(S.distill_loss_ad(z, u, ids, temperature=2.0), z, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, stats = S.distill_loss(z.detach(), u, ids, temperature=2.0, with_stats=True)
        grad = S.distill_loss_backward(g, z.detach(), ids, stats, temperature=2.0)
    graph.replay()
    (want,) = torch.autograd.grad(eager, z, g)
    torch.cuda.synchronize()
    assert torch.equal(loss, eager.detach()) and torch.equal(grad, want)
