"""Adapters beside a packed projection on the GPU against 64-bit products.

Tolerance.  The fp32 sums of K (or rank) terms lose at most sqrt(K) half-ulps
in all likelihood, 2^-17 of the sum of absolute terms for K up to 8192; the
prefill's a x enter as two bf16 terms, 2^-16 of the low-rank sum.  A bf16 y adds
half an ulp (2^-8 of its value at most)."""

import numpy as np
import pytest

import oracle as O

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


def make(n, k, gran, tokens, count, rank, seed=0, group=128):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + n + 3 * k + 7 * tokens)
    w = torch.randn(n, k, generator=g, device=DEV) * 0.02
    pw = S.quantize_pack(w, gran, group)
    wq = S.unpack(pw, "float32").double()
    x = torch.randn(tokens, k, generator=g, device=DEV).to(BF16)
    a = (torch.randn(count, rank, k, generator=g, device=DEV) * k ** -0.5).to(BF16)
    b = (torch.randn(count, n, rank, generator=g, device=DEV) * 0.2).to(BF16)
    scale = torch.rand(count, generator=g, device=DEV) + 0.5
    ids = torch.randint(-1, count, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    return pw, wq, x, S.AdapterSet(a, b, scale), ids


def reference(wq, x, ad, ids):
    xd = x.double()
    y, size, low = xd @ wq.t(), xd.abs() @ wq.abs().t(), 0
    low = torch.zeros_like(y)
    for m, c in enumerate(ids.tolist()):
        if 0 <= c < ad.a.shape[0]:
            r = ad.a.shape[1] if ad.rank is None else max(0, min(int(ad.rank[c]), ad.a.shape[1]))
            a, b, s = ad.a[c, :r].double(), ad.b[c, :, :r].double(), float(ad.scale[c])
            v = a @ xd[m]
            y[m] += s * (b @ v)
            size[m] += s * (b.abs() @ (a.abs() @ xd[m].abs()))
            low[m] = s * (b.abs() @ v.abs())
    return y, size * 2.0 ** -17 + low * 2.0 ** -15


def check(got, want, tol, dtype):
    assert got.dtype == dtype
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all()) and bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("batch", [1, 2, 5, 16])
@pytest.mark.parametrize("n,k", [(64, 256), (517, 128), (2048, 2048), (300, 8192), (4100, 384)])
@pytest.mark.parametrize("gran", ["per_group", "per_channel", "per_tensor"])
def test_decode(batch, n, k, gran):
    pw, wq, x, ad, ids = make(n, k, gran, batch, 3, 16)
    if batch == 1:
        ids[0] = 2
    want, tol = reference(wq, x, ad, ids)
    check(S.adapter_gemv(pw, x, ad, ids), want, tol, BF16)
    check(S.adapter_gemv(pw, x, ad, ids, "float32"), want, tol, F32)


@pytest.mark.parametrize("rank", [8, 24, 40, 64, 136, 256])
def test_ranks(rank):
    for tokens in (1, 7, 70):
        pw, wq, x, ad, ids = make(200, 512, "per_group", tokens, 5, rank)
        ad.rank = torch.tensor([0, 1, rank - 3, rank, rank + 9], dtype=torch.int32, device=DEV)
        ids.copy_(torch.arange(tokens, device=DEV) % 6 - 1 if tokens > 1 else torch.tensor([2], device=DEV))
        want, tol = reference(wq, x, ad, ids)
        f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
        check(f(pw, x, ad, ids), want, tol, BF16)


@pytest.mark.parametrize("m", [1, 15, 16, 17, 63, 64, 65, 200, 517])
@pytest.mark.parametrize("n,k,gran,group", [(256, 512, "per_group", 128), (130, 1024, "per_channel", 128),
                                            (77, 128, "per_tensor", 128), (2048, 2048, "per_group", 128),
                                            (384, 2048, "per_group", 256), (2048, 2048, "per_channel", 128)])
def test_prefill(m, n, k, gran, group):
    pw, wq, x, ad, ids = make(n, k, gran, m, 4, 16, group=group)
    ids = ids.sort().values
    want, tol = reference(wq, x, ad, ids)
    check(S.adapter_gemm(pw, x, ad, ids), want, tol, BF16)


@pytest.mark.parametrize("gran", ["per_group", "per_channel", "per_tensor"])
def test_prefill_wide_tiles(gran):
    pw, wq, x, ad, ids = make(16384, 256, gran, 600, 6, 32)
    want, tol = reference(wq, x, ad, ids)
    check(S.adapter_gemm(pw, x, ad, ids), want, tol, BF16)


def test_prefill_past_the_copy_range():
    """More activations than one launch addresses (2^31 bytes): the next
    launch's tokens keep their ids and low-rank products."""
    tokens, k = 131100, 8192
    pw, wq, _, ad, _ = make(64, k, "per_group", 1, 5, 16)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(tokens, k, generator=g, device=DEV, dtype=BF16)
    ids = (torch.arange(tokens, device=DEV) // 7 % 6).to(torch.int32)
    y = S.adapter_gemm(pw, x, ad, ids)
    at = torch.cat([torch.arange(0, 10), torch.arange(130930, 130960), torch.arange(131060, 131100)]).to(DEV)
    want, tol = reference(wq, x[at], ad, ids[at])
    check(y[at], want, tol, BF16)


@pytest.mark.parametrize("tokens", [1, 5, 16, 40])
def test_adapters_past_32_bit_offsets(tokens):
    """2.2e9 elements of b: the last adapters are found."""
    pw, wq, x, _, _ = make(16384, 256, "per_group", tokens, 1, 8)
    g = torch.Generator(device=DEV).manual_seed(9)
    b = torch.randn(2100, 16384, 64, generator=g, device=DEV, dtype=BF16)
    a = torch.randn(2100, 64, 256, generator=g, device=DEV, dtype=BF16) * 0.1
    ad = S.AdapterSet(a, b, torch.rand(2100, generator=g, device=DEV))
    ids = (2099 - torch.arange(tokens, device=DEV) // 3).to(torch.int32)
    want, tol = reference(wq, x, ad, ids)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    check(f(pw, x, ad, ids), want, tol, BF16)


@pytest.mark.parametrize("tokens", [3, 16, 33, 300])
def test_ids(tokens):
    """No adapter, ids out of range, every token its own, one for all; ids in any order."""
    pw, wq, x, ad, _ = make(192, 640, "per_group", tokens, 40, 24)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    t = torch.arange(tokens, device=DEV)
    for ids in (torch.full((tokens,), -1), torch.full((tokens,), 40), torch.full((tokens,), 39), (t * 7) % 40,
                torch.where(t % 2 == 0, -(2 ** 31), 2 ** 31 - 1), 39 - t % 40):
        ids = ids.to(DEV, torch.int32)
        want, tol = reference(wq, x, ad, ids)
        check(f(pw, x, ad, ids), want, tol, BF16)


def test_tokens_without_adapter_get_the_projection():
    for tokens in (1, 9, 64, 333):
        pw, _, x, ad, ids = make(512, 1024, "per_group", tokens, 3, 16)
        ids.fill_(-1)
        if tokens <= 16:
            assert torch.equal(S.adapter_gemv(pw, x, ad, ids, "float32"), S.gemv(pw, x, "float32"))
        else:
            assert torch.equal(S.adapter_gemm(pw, x, ad, ids), S.gemm(pw, x))


@pytest.mark.parametrize("tokens", [5, 16, 48, 130])
def test_bad_values_stay_with_their_tokens(tokens):
    """Infinities and NaN in one adapter, in its unused rows, and in one token."""
    pw, wq, x, ad, ids = make(320, 512, "per_group", tokens, 4, 16)
    ids.copy_(torch.arange(tokens, device=DEV) % 4)
    ad.rank = torch.tensor([16, 9, 16, 12], dtype=torch.int32, device=DEV)
    want, tol = reference(wq, x, ad, ids)
    ad.a[1, 9:], ad.b[1, :, 9:] = float("nan"), float("inf")      # beyond the rank
    ad.b[2, 5, 3], ad.a[2, 1, 7] = float("inf"), float("nan")     # adapter 2 itself
    x[3, 9] = float("nan")                                        # a token of adapter 3
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    got = f(pw, x, ad, ids)
    good = (ids != 2) & (torch.arange(tokens, device=DEV) != 3)
    check(got[good], want[good], tol[good], BF16)
    assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[2]).all())


@pytest.mark.parametrize("tokens", [4, 16, 40, 150])
def test_an_infinite_scale_keeps_its_signs(tokens):
    """One adapter of rank 1 and infinite scale: its tokens' outputs are the signed infinities of b."""
    pw, _, x, ad, ids = make(256, 512, "per_group", tokens, 3, 8)
    ids.fill_(1)
    ad.rank = torch.tensor([8, 1, 8], dtype=torch.int32, device=DEV)
    ad.scale[1] = float("inf")
    want = torch.sign(x.double() @ ad.a[1, 0].double())[:, None] * ad.b[1, :, 0].double() * float("inf")
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    assert torch.equal(f(pw, x, ad, ids).double(), want)


def test_one_token_alike_in_both_forms():
    pw, wq, x, ad, ids = make(256, 256, "per_channel", 1, 2, 8)
    ids[0] = 1
    want, tol = reference(wq, x, ad, ids)
    check(S.adapter_gemm(pw, x, ad, ids), want, tol, BF16)
    check(S.adapter_gemv(pw, x[0], ad, ids), want, tol, BF16)


def test_out_and_stream():
    pw, wq, x, ad, ids = make(512, 512, "per_group", 100, 3, 16)
    want, tol = reference(wq, x, ad, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty(100, 512, dtype=BF16, device=DEV)
    assert S.adapter_gemm(pw, x, ad, ids, stream=s, out=out) is out
    y = S.adapter_gemv(pw, x[:8], ad, ids[:8], stream=s)
    torch.cuda.synchronize()
    check(out, want, tol, BF16)
    check(y, want[:8], tol[:8], BF16)


def test_against_the_oracle():
    """The base product of the oracle's own quantization, and the adapters' by numpy."""
    rng = np.random.default_rng(5)
    w = rng.standard_normal((64, 256)).astype(np.float32) * 0.02
    pw = S.quantize_pack(torch.from_numpy(w).to(DEV))
    _, alpha = O.quantize_pack(w, "per_group", 128)
    wq = torch.from_numpy(O.dequant(O.ternary(w), alpha, "per_group", 128)).to(DEV).double()
    _, _, x, ad, ids = make(64, 256, "per_group", 20, 3, 8)
    want, tol = reference(wq, x, ad, ids)
    check(S.adapter_gemm(pw, x, ad, ids), want, tol, BF16)
    check(S.adapter_gemv(pw, x[:11], ad, ids[:11]), want[:11], tol[:11], BF16)


def test_refusals():
    pw, _, x, ad, ids = make(64, 256, "per_group", 4, 2, 16)
    bad = [
        (x, S.AdapterSet(ad.a[:, :12], ad.b, ad.scale), ids), (x, S.AdapterSet(ad.a, ad.b[:1], ad.scale), ids),
        (x, S.AdapterSet(ad.a.float(), ad.b, ad.scale), ids), (x, S.AdapterSet(ad.a, ad.b, ad.scale[:1]), ids),
        (x, S.AdapterSet(ad.a, ad.b, ad.scale, ids[:1]), ids), (x, ad, ids[:3]), (x, ad, ids.long()),
        (x, ad, ids.cpu()), (x.float(), ad, ids), (x[:, :128], ad, ids),
        (x, S.AdapterSet(ad.a, ad.b.transpose(1, 2).contiguous().transpose(1, 2), ad.scale), ids),
    ]
    for args in bad:
        for f in (S.adapter_gemv, S.adapter_gemm):
            with pytest.raises(ValueError):
                f(pw, *args)
    with pytest.raises(ValueError):
        S.adapter_gemv(pw, x.repeat(5, 1), ad, ids.repeat(5))
    with pytest.raises(ValueError):
        S.adapter_gemm(pw, x[:0], ad, ids[:0])


@pytest.mark.parametrize("n", [1048064, 1048065, 1 << 20])
@pytest.mark.parametrize("gran", ["per_group", "per_channel"])
def test_one_token_on_the_widest_weights(n, gran):
    """From N = 1048065 a single call takes workgroups of 512 rows, with adapters as without."""
    pw, wq, x, ad, ids = make(n, 128, gran, 1, 2, 8)
    for c in (-1, 1):
        ids[0] = c
        want, tol = reference(wq, x, ad, ids)
        check(S.adapter_gemv(pw, x, ad, ids), want, tol, BF16)
        check(S.adapter_gemv(pw, x, ad, ids, "float32"), want, tol, F32)


def same_as_defined(got, want, tol):
    """Infinities and NaN where the 64-bit product has them, the rest within bounds."""
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf].double(), want[inf])
    check(got[fine], want[fine], tol[fine], BF16)


@pytest.mark.parametrize("tokens", [3, 16, 40, 150])
@pytest.mark.parametrize("n,gran", [(256, "per_group"), (256, "per_tensor"), (16384, "per_channel")])
def test_infinities_in_b_keep_their_signs(tokens, n, gran):
    """b times its token's a x: signed infinities, whether a x is a bf16 number or not, and NaN where it is zero."""
    pw, wq, x, ad, ids = make(n, 256, gran, tokens, 3, 16)
    ids.copy_(torch.arange(tokens, device=DEV) // 2 % 3)
    ad.scale.fill_(1.0)
    ad.a[0, 0], ad.a[0, 1] = 0, 0
    ad.a[0, 0, 5] = 1.0                        # a x is the token's value itself: no second term
    ad.a[0, 1, 5], ad.a[0, 1, 6] = 1.0, 2 ** -9   # and one that has a second term of either sign
    x[1, 5] = 0
    inf = float("inf")
    ad.b[0, 7, 0], ad.b[0, 60, 1], ad.b[0, 61, 1] = inf, inf, -inf
    ad.b[1, 100, 15] = -inf
    ad.b[2, 9, 2] = float("nan")
    want, tol = reference(wq, x, ad, ids)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    same_as_defined(f(pw, x, ad, ids), want, tol)


@pytest.mark.parametrize("tokens", [3, 40, 150])
def test_low_rank_sums_past_the_largest_bf16(tokens):
    """a x between the largest bf16 and the largest fp32 number: finite, as b x it is."""
    pw, wq, x, ad, ids = make(256, 256, "per_group", tokens, 2, 8)
    ids.fill_(1)
    ad.a[1] = 0
    ad.a[1, 0, 0] = 1.0
    x[:, 0] = torch.where(torch.arange(tokens, device=DEV) % 2 == 0, 1.0, -1.0).to(BF16)
    ad.scale[1] = 3.399e38
    ad.b[1, :, 0] = (ad.b[1, :, 0].double() * 2.0 ** -120).to(BF16)
    want, tol = reference(wq, x, ad, ids)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    same_as_defined(f(pw, x, ad, ids), want, tol)


@pytest.mark.parametrize("tokens", [3, 40, 150])
def test_infinities_in_both_factors(tokens):
    """b and a x infinite at once: their product's sign."""
    pw, wq, x, ad, ids = make(256, 256, "per_group", tokens, 2, 8)
    ids.fill_(1)
    ad.rank = torch.tensor([8, 1], dtype=torch.int32, device=DEV)
    ad.scale[1] = float("inf")
    ad.b[1, 9, 0], ad.b[1, 77, 0] = float("inf"), -float("inf")
    want, tol = reference(wq, x, ad, ids)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    same_as_defined(f(pw, x, ad, ids), want, tol)


@pytest.mark.parametrize("tokens", [3, 40, 700])
@pytest.mark.parametrize("n", [200, 16384])
def test_cancelling_low_rank_sums(tokens, n):
    """Two terms that leave 2^-14 of themselves: a x of fp32's 24 bits (three half-ulps of each term), y rounded
    once.  16 bits of a x would be off by up to 2^-18 of each."""
    pw, wq, x, ad, ids = make(n, 128, "per_group", tokens, 3, 8)
    pw.alpha.mul_(2.0 ** -40)
    ids.copy_(torch.arange(tokens, device=DEV) % 3)
    for t in (x, ad.a, ad.b):
        t.zero_()
    x[:, 0], x[:, 1] = 1.0, -(1 - 2.0 ** -7)
    ad.a[:, 0, 0], ad.a[:, 1, 1] = 1.0, 1.0
    ad.b[:, :, 0], ad.b[:, :, 1] = 1.0, 1 + 2.0 ** -7
    ad.scale.copy_(torch.tensor([1.2345678, 0.7654321, 1.9996643], device=DEV))
    want, _ = reference(wq * 2.0 ** -40, x, ad, ids)
    size = 2.0 * ad.scale[ids.long()].double()[:, None].expand_as(want)
    f = S.adapter_gemv if tokens <= 16 else S.adapter_gemm
    check(f(pw, x, ad, ids), want, 3 * 2.0 ** -24 * size, BF16)
