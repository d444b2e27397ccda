"""Outputs of the caller's are written through their addresses.  For autograd
they count as changed in place all the same: a graph that saved one refuses its
backward pass instead of giving wrong gradients."""

import pytest

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


def rand(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


def adapters(n, k):
    return S.AdapterSet(rand(2, 8, k, dtype=BF16), rand(2, n, 8, dtype=BF16), torch.ones(2, device=DEV))


def experts():
    return S.quantize_pack_experts(rand(4, 512, 256)), S.quantize_pack_experts(rand(4, 256, 256))


def distill(out):
    z = out if out.requires_grad is False else out.detach()
    ids, u = torch.zeros(4, 3, dtype=torch.int32, device=DEV), rand(4, 3)
    _, stats = S.distill_loss(z, u, ids, with_stats=True)
    S.distill_loss_backward(torch.ones(4, device=DEV), z, ids, stats, out=z)


CALLS = {
    "gemv": lambda pw, x, y: S.gemv(pw, x, out=y),
    "gemm": lambda pw, x, y: S.gemm(pw, x, out=y),
    "arenas_gemm": lambda pw, x, y: S.arenas_gemm(pw, rand(256, 256), 0.5, x, out=y),
    "gemv_batched": lambda pw, x, y: S.gemv_batched(pw.packed, pw.alpha, 256, 256, x, 1, pw.packed.numel(), pw.alpha.numel(), y=y),
    "adapter_gemv": lambda pw, x, y: S.adapter_gemv(pw, x, adapters(256, 256), torch.zeros(4, dtype=torch.int32, device=DEV), out=y),
    "adapter_gemm": lambda pw, x, y: S.adapter_gemm(pw, x, adapters(256, 256), torch.zeros(4, dtype=torch.int32, device=DEV), out=y),
    "orthogonalize": lambda pw, x, y: S.orthogonalize(x, out=y),
    "muon_step": lambda pw, x, y: S.muon_step(x, x, x, 0.1, out=(y, torch.empty_like(y))),
    "muon_step, momentum": lambda pw, x, y: S.muon_step(x, x, x, 0.1, out=(torch.empty_like(y), y)),
    "linear_gemv": lambda pw, x, y: S.linear_gemv(pw, x, residual=y, out=y),
    "linear_gemm": lambda pw, x, y: S.linear_gemm(pw, x, residual=y, out=y),
    "moe_decode": lambda pw, x, y: S.moe_decode(x, rand(4, 256, dtype=BF16), *experts(), 2, residual=y, out=y),
    "distill_loss_backward": lambda pw, x, y: distill(y),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [False, True])
def test_outputs_count_as_changed(name, stream):
    pw, x, y = S.quantize_pack(rand(256, 256)), rand(4, 256, dtype=BF16), rand(4, 256, dtype=BF16, seed=1)
    before, inputs = y._version, (x._version, pw.packed._version)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side if stream else None):
        CALLS[name](pw, x, y)
    torch.cuda.synchronize()
    assert y._version > before and (x._version, pw.packed._version) == inputs
    with torch.inference_mode():       # such tensors have no version
        CALLS[name](pw, x, torch.zeros_like(y))


def test_packed_outputs_count_as_changed():
    w = rand(64, 256)
    packed, alpha = torch.empty(64 * 40, dtype=torch.uint8, device=DEV), torch.empty(128, device=DEV)
    before = packed._version, alpha._version
    S.quantize_pack_noalloc(w, packed, alpha)
    assert packed._version > before[0] and alpha._version > before[1]
    planes, x = S.compare_repack(S.quantize_pack(w, "per_channel"), 0), rand(256, dtype=BF16)
    y = torch.empty(1, 64, dtype=BF16, device=DEV)
    before = y._version
    S.compare_gemv(0, planes, torch.ones(64, device=DEV), 64, 256, x, y=y, y_stride=64)
    assert y._version > before


def test_a_saved_tensor_that_was_written_over():
    """A capped head saves its tanh; the gradient in the place of the logits writes over it."""
    a = rand(4, 256, dtype=BF16).requires_grad_(True)
    z = torch.tanh(a)
    distill(z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    h = rand(4, 256, dtype=BF16).requires_grad_(True)
    stream = h * h                     # the residual stream; its square saves it
    square = stream * stream
    with torch.no_grad():
        S.linear_gemv(S.quantize_pack(rand(256, 256)), rand(4, 256, dtype=BF16), residual=stream, out=stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        square.sum().backward()
