"""The operators around the layer inside a HIP graph: one capture, several
replays on new inputs with eager work between them, each equal to the eager
call bit for bit (every sum has a fixed order)."""

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


@pytest.mark.parametrize("tokens,n,k,gran", [(1, 512, 1024, "per_group"), (9, 300, 2048, "per_channel"),
                                             (70, 384, 1024, "per_group"), (200, 256, 512, "per_tensor")])
def test_adapters(tokens, n, k, gran):
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    pw = S.quantize_pack(rand(gen, n, k) * 0.02, gran)
    ad = S.AdapterSet(rand(gen, 5, 16, k, dtype=BF16), rand(gen, 5, n, 16, dtype=BF16),
                      torch.ones(5, device=DEV), torch.tensor([16, 3, 0, 8, 11], dtype=torch.int32, device=DEV))
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm

    def fresh(i):
        return (rand(gen, tokens, k, dtype=BF16),
                torch.randint(-1, 6, (tokens,), generator=gen, device=DEV, dtype=torch.int32))
    replays(lambda x, ids: [f(pw, x, ad, ids)], list(fresh(0)), fresh)


@pytest.mark.parametrize("rows,dim,dtype", [(1, 2048, BF16), (257, 1001, F32)])
def test_norms(rows, dim, dtype):
    gen = torch.Generator(device=DEV).manual_seed(dim)
    w1, w2, gate = 1 + 0.1 * rand(gen, dim), 1 + 0.1 * rand(gen, dim), rand(gen, dim, dtype=dtype)

    def fresh(i):
        return [rand(gen, rows, dim, dtype=dtype) for _ in range(4)]

    def call(h, y, dh, dn):
        args = dict(y=y, w_post=w2, gate=gate, res_scale=0.8)
        return [*S.block_norm(h, w1, **args), *S.block_norm_backward(dh, dn, h, w1, **args)]
    replays(call, fresh(0), fresh)


@pytest.mark.parametrize("count,n,k,dtype", [(1, 100, 300, F32), (2, 512, 1024, BF16), (1, 1100, 1100, F32)])
def test_updates(count, n, k, dtype):
    gen = torch.Generator(device=DEV).manual_seed(n)

    def fresh(i):
        return [rand(gen, count, n, k, dtype=dtype) for _ in range(3)]

    def call(w, grad, buf):
        return [*S.muon_step(w, grad, buf, 0.02, weight_decay=0.1), S.orthogonalize(grad)]
    replays(call, fresh(0), fresh)
