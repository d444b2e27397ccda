"""The packed product with bias, activation and residual against its definition
in 64 bits (the packed weight as the library unpacks it, which other tests
hold to the oracle bit for bit).

Tolerances.  A sum of K products in fp32 by steps of 32 and groups of 128 and
more is off by at most (K / 32 + K / 128 + 64) 2^-23 of the sum of magnitudes;
the activations pass that on by their slopes (at most 1.13, 2 |z| for the
square) and are off by 2^-17 of themselves (an exponential's argument of up to
32 has steps of 2^-19); products and the residual add 2^-22; the result is
rounded once, by half a step."""

import math

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("ternary_weight_quantization_sparse_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
INF = float("inf")
ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    S.load()


def rand(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def act_tol(z, dz, name):
    slope = 2 * z.abs() + dz if name == "relu2" else 1.0 if name in ("none", "relu") else 1.13
    return slope * dz + (0 if name in ("none", "relu") else 2.0 ** -17 * act(z, name).abs())


def oracle(dense, x, bias, name, gated, residual, res_scale):
    """(value, tolerance before the last rounding) in 64 bits."""
    w, xd = dense.double(), x.double()
    k = x.shape[1]
    z = xd @ w.t().contiguous()
    dz = (k / 32 + k / 128 + 64) * 2.0 ** -23 * (xd.abs() @ w.abs().t().contiguous())
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2.0 ** -23 * z.abs()
    if gated:
        half = z.shape[1] // 2
        f, df, u, du = act(z[:, :half], name), act_tol(z[:, :half], dz[:, :half], name), z[:, half:], dz[:, half:]
        y, dy = f * u, df * u.abs() + (f.abs() + df) * du + 2.0 ** -23 * (f * u).abs()
    else:
        y, dy = act(z, name), act_tol(z, dz, name)
    if residual is not None:
        y = y + res_scale * residual.double()
        dy = dy + 2.0 ** -22 * (y.abs() + (res_scale * residual.double()).abs())
    return y, dy


def close(got, want, tol):
    bound = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol) + 1e-37
    err = (got.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


def make(tokens, n, k, grain="per_group", group=128, bias="float32", residual=True, gated=False, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed + 7 * tokens + n + k)
    pw = S.quantize_pack(rand(gen, n, k, std=0.04), grain, group)
    b = None if bias is None else rand(gen, n, std=0.5, dtype=getattr(torch, bias))
    x = rand(gen, tokens, k, dtype=BF16)
    res = rand(gen, tokens, n // 2 if gated else n, std=2.0, dtype=BF16) if residual else None
    return pw, x, b, res


def check(pw, x, bias, name, gated, residual, res_scale=0.8, f=None, **kw):
    f = f or (S.linear_gemv if x.shape[0] <= 16 else S.linear_gemm)
    res_scale = res_scale if residual is not None else 1.0
    y = f(pw, x, bias=bias, activation=name, gated=gated, residual=residual, res_scale=res_scale, **kw)
    want, tol = oracle(S.unpack(pw, "float32"), x, bias, name, gated, residual, res_scale)
    close(y, want, tol)
    return y


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ACTS)
def test_activations(name, gated):
    for tokens in (3, 70):
        pw, x, b, res = make(tokens, 272, 512, gated=gated)
        check(pw, x, b, name, gated, res)


@pytest.mark.parametrize("grain,group", [("per_group", 128), ("per_group", 512), ("per_channel", 128), ("per_tensor", 128)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens,n,k", [(1, 16, 128), (1, 2, 1024), (2, 1002, 512), (4, 4096, 2048), (5, 130, 8192),
                                        (16, 514, 3584), (9, 34, 6656), (17, 62, 1024), (64, 128, 512), (129, 1002, 2048),
                                        (300, 2050, 512), (1000, 4098, 1024)])
def test_sizes(tokens, n, k, grain, group, gated):
    if k % group:
        group = 128
    pw, x, b, res = make(tokens, n, k, grain, group, gated=gated)
    check(pw, x, b, "silu", gated, res)


@pytest.mark.parametrize("tokens,n,k", [(1, 1, 128), (7, 1001, 1024), (20, 77, 512), (200, 1001, 1024), (700, 2049, 512)])
@pytest.mark.parametrize("bias", [None, "bfloat16"])
def test_odd_widths(tokens, n, k, bias):
    for residual in (False, True):
        pw, x, b, res = make(tokens, n, k, bias=bias, residual=residual)
        check(pw, x, b, "gelu", False, res)


def test_wide_tiles():
    """Enough 256-row tiles for the wide kernel, ragged on both sides, and row scales."""
    for grain in ("per_group", "per_channel"):
        pw, x, b, res = make(1030, 8200, 256, grain, gated=True)
        check(pw, x, b, "silu", True, res)
        pw, x, b, res = make(1030, 8190, 256, grain)
        check(pw, x, b, "relu2", False, res)


@pytest.mark.parametrize("k", [512, 1024, 2048, 4096, 8192, 12416])
@pytest.mark.parametrize("gated", [False, True])
def test_decode_tiles(k, gated):
    """64 weight rows a workgroup and 16, at every count of superblocks a wave, ragged."""
    for tokens, n in ((5, 16390), (16, 70), (1, 1030)):
        pw, x, b, res = make(tokens, n, k, bias="bfloat16", gated=gated)
        check(pw, x, b, "silu", gated, res)


def test_prompts_in_several_launches():
    """Rows past one launch's address range (3968 of them at K = 2^18)."""
    n, k, tokens = 32, 1 << 18, 4100
    pw, x, b, res = make(tokens, n, k, "per_channel", gated=True)
    y = S.linear_gemm(pw, x, bias=b, activation="silu", gated=True, residual=res, res_scale=0.8)
    dense = S.unpack(pw, "float32")
    rows = [0, 63, 3967, 3968, 4031, 4032, 4099]
    want, tol = oracle(dense, x[rows], b, "silu", True, res[rows], 0.8)
    close(y[rows], want, tol)


@pytest.mark.parametrize("grain", ["per_group", "per_channel", "per_tensor"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens,n,k", [(517, 4098, 2048), (260, 2050, 8192), (2050, 2050, 1024), (2050, 16386, 512)])
def test_prompts_of_many_tiles(tokens, n, k, grain, gated):
    """Splits of K, narrow and wide tiles of the long prompts' kernel."""
    pw, x, b, res = make(tokens, n, k, grain, gated=gated)
    check(pw, x, b, "silu", gated, res)


@pytest.mark.parametrize("grain", ["per_group", "per_channel", "per_tensor"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens,n,k", [(1024, 8190, 640), (1000, 8002, 640), (2048, 8190, 4096)])
def test_prompts_of_wide_tiles(tokens, n, k, grain, gated):
    """Wide tiles in one full round and in two."""
    pw, x, b, res = make(tokens, n, k, grain, gated=gated)
    check(pw, x, b, "gelu", gated, res)


@pytest.mark.parametrize("tokens,n,k", [(1024, 2048, 2048), (1024, 2050, 2048), (17, 64, 128), (31, 66, 8192), (255, 1002, 384),
                                        (4096, 128, 2048)])
def test_prompts_of_few_tiles(tokens, n, k):
    """Up to the last size of the short workgroups' kernel and past it, with four waves and with eight."""
    for gated in (False, True):
        pw, x, b, res = make(tokens, n, k, gated=gated)
        check(pw, x, b, "gelu_tanh", gated, res)
        pw, x, _, _ = make(tokens, n, k, "per_channel", bias=None, residual=False, gated=gated)
        check(pw, x, None, "relu2", gated, None)


def test_no_epilogue_is_the_product():
    for tokens in (1, 16, 400):
        pw, x, _, _ = make(tokens, 512, 1024, bias=None, residual=False)
        y = (S.linear_gemv if tokens <= 16 else S.linear_gemm)(pw, x)
        plain = (S.gemv if tokens <= 16 else S.gemm)(pw, x)
        if tokens > 16:
            assert torch.equal(y, plain)     # the same kernel's sums
        want, tol = oracle(S.unpack(pw, "float32"), x, None, "none", False, None, 1.0)
        close(y, want, tol)


def test_float32_output():
    pw, x, b, res = make(6, 300, 1024)
    y = check(pw, x, b, "silu", False, res, y_dtype="float32")
    assert y.dtype == F32
    x1 = x[0]                                # a single token without its batch axis
    y1 = S.linear_gemv(pw, x1, bias=b, residual=res[0])
    assert y1.shape == (1, 300) and torch.equal(y1, S.linear_gemv(pw, x[:1], bias=b, residual=res[:1]))


@pytest.mark.parametrize("tokens", [5, 90, 400])
def test_residual_updated_in_place(tokens):
    pw, x, b, res = make(tokens, 1024, 512, gated=True)
    want = check(pw, x, b, "silu", True, res)
    f = S.linear_gemv if tokens <= 16 else S.linear_gemm
    y = f(pw, x, bias=b, activation="silu", gated=True, residual=res, res_scale=0.8, out=res)
    assert y is res and torch.equal(res, want)


def test_strided_operands():
    pw, x, b, res = make(8, 256, 512)
    wide, rwide = torch.zeros(8, 1024, dtype=BF16, device=DEV), torch.zeros(8, 2, 256, dtype=BF16, device=DEV)
    wide[:, ::2], rwide[:, 1] = x, res
    bwide = torch.stack([b, b], 1)
    y = S.linear_gemv(pw, wide[:, ::2], bias=bwide[:, 0], residual=rwide[:, 1])
    assert torch.equal(y, S.linear_gemv(pw, x, bias=b, residual=res))


def test_rows_behind_the_output_are_left_alone():
    for tokens in (3, 77):
        pw, x, b, res = make(tokens, 100, 256)
        store = torch.full((tokens + 2, 100), 7.0, dtype=BF16, device=DEV)
        f = S.linear_gemv if tokens <= 16 else S.linear_gemm
        f(pw, x, bias=b, residual=res, out=store[:tokens])
        assert (store[tokens:] == 7).all() and torch.equal(store[:tokens], f(pw, x, bias=b, residual=res))


@pytest.mark.parametrize("tokens", [4, 40])
def test_tokens_do_not_meet(tokens):
    """Not a number and infinities in one token, and in its residual, stay in its row; large sums keep their sign."""
    pw, x, b, res = make(tokens, 200, 512, gated=True)
    clean = check(pw, x, b, "silu", True, res)
    x[1, 3], res[2, 5] = float("nan"), float("inf")
    f = S.linear_gemv if tokens <= 16 else S.linear_gemm
    y = f(pw, x, bias=b, activation="silu", gated=True, residual=res, res_scale=0.8)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[2, 5] = False, False
    assert torch.equal(y[keep], clean[keep]) and y[2, 5] == float("inf")
    big = torch.full_like(x, 1e30)
    for name in ACTS[1:]:
        z = f(pw, big, activation="none")
        y = f(pw, big, activation=name)
        # far from zero an activation is the identity (squared: past the type's range) or zero
        assert torch.equal(y[z > 0], z[z > 0] if name != "relu2" else z[z > 0] * INF) and (y[z < 0] == 0).all(), name


def test_repeats_and_streams():
    pw, x, b, res = make(16, 1024, 2048, gated=True)
    first = S.linear_gemv(pw, x, bias=b, activation="gelu", gated=True, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = S.linear_gemv(pw, x, bias=b, activation="gelu", gated=True, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(y, first)


def test_rows_past_32_bits():
    n, k, tokens = 65536 + 130, 256, 33000       # 2.17 * 10^9 outputs
    pw, x, b, _ = make(tokens, n, k, bias="bfloat16", residual=False)
    y = S.linear_gemm(pw, x, bias=b, activation="relu")
    dense = S.unpack(pw, "float32")
    for r in (0, 16384, 32767, 32999):
        want, tol = oracle(dense, x[r:r + 1], b, "relu", False, None, 1.0)
        close(y[r:r + 1], want, tol)


def test_refusals():
    pw, x, b, res = make(4, 64, 256)
    for bad in (dict(activation="tanh"), dict(bias=b[:-1]), dict(bias=b.double()), dict(residual=res.float()),
                dict(residual=res[:3]), dict(res_scale=0.5), dict(out=res.float()), dict(out=x[:, :64]),
                dict(bias=b.cpu()), dict(residual=res.cpu()), dict(residual=res, out=res.flatten()[:4 * 64].view(4, 64)[:, :32])):
        with pytest.raises(ValueError):
            S.linear_gemv(pw, x, **bad)
    for bad in (x.float(), x[:, :128], x[None], x.cpu(), x[:0], torch.zeros(17, 256, dtype=BF16, device=DEV)):
        with pytest.raises(ValueError):
            S.linear_gemv(pw, bad)
    odd = make(4, 63, 256)[0]
    with pytest.raises(ValueError, match="even"):
        S.linear_gemv(odd, x, gated=True)
    short = S.PackedWeight(pw.packed[:-1], pw.alpha, 64, 256)
    with pytest.raises(ValueError, match="packed"):
        S.linear_gemm(short, x)
    with pytest.raises(ValueError, match="alpha"):
        S.linear_gemm(S.PackedWeight(pw.packed, pw.alpha[:-1], 64, 256), x)


@pytest.mark.parametrize("grain", ["per_group", "per_channel", "per_tensor"])
@pytest.mark.parametrize("n,k", [(40, 128), (40, 640), (40, 1152), (20000, 640)])
def test_a_scale_that_is_infinite_stays_so(n, k, grain):
    """Waves without a superblock of their own add nothing.  The sums of a superblock are far from zero: x is one
    there, and each row's weights have one sign."""
    gen = torch.Generator(device=DEV).manual_seed(n + k)
    sign = torch.where(torch.arange(n, device=DEV) % 3 == 0, -1.0, 1.0)[:, None]
    pw = S.quantize_pack(rand(gen, n, k).abs() * sign, grain, 128)
    pw.alpha.fill_(INF)
    y = S.linear_gemv(pw, torch.ones(2, k, dtype=BF16, device=DEV))
    assert torch.equal(y, (sign[:, 0] * INF).to(BF16).expand(2, -1))


@pytest.mark.parametrize("grain", ["per_group", "per_channel"])
@pytest.mark.parametrize("tokens", [3, 60])
def test_a_gate_and_its_values_packed_together(tokens, grain):
    """What `quantize_pack_fused` makes of the two, gated and as the stacked product."""
    gen = torch.Generator(device=DEV).manual_seed(11)
    gate, values = rand(gen, 200, 512, std=0.04), rand(gen, 200, 512, std=0.04)
    fw = S.quantize_pack_fused([gate, values], grain)
    x, b = rand(gen, tokens, 512, dtype=BF16), rand(gen, 400, std=0.5)
    f = S.linear_gemv if tokens <= 16 else S.linear_gemm
    for gated in (True, False):
        y = f(fw, x, bias=b, activation="silu", gated=gated)
        want, tol = oracle(S.unpack(fw.pw, "float32"), x, b, "silu", gated, None, 1.0)
        close(y, want, tol)
        assert torch.equal(y, f(fw.pw, x, bias=b, activation="silu", gated=gated))
    for members in ([gate, values[:128]], [gate[:128], values], [gate], [gate, values, gate, values]):
        with pytest.raises(ValueError, match="two members"):
            f(S.quantize_pack_fused(members, grain), x, activation="silu", gated=True)
