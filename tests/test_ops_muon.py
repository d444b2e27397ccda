"""Orthogonalised updates on the GPU against the same steps in 64 bits.

Tolerance.  Every factor carries 22 bits and every sum is fp32: a product is
off by about 2^-21 of its norm, a step has three with weights up to |a| + |b| +
|c| ~ 10, and five steps add up: 5 * 3 * 10 * 2^-21 ~ 7e-5 of the result for a
spectrum that rises together.  Directions far below the largest one rise by up
to 3.44 a step more than the rest: 1e-3 for low-rank and spiked ones.  A bf16
result adds 2^-9."""

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


def rand(*shape, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * std


def steps64(u, steps=5, coeffs=S.NEWTON_SCHULZ, eps=1e-7):
    a, b, c = coeffs
    out = []
    for x in (u if u.dim() == 3 else u[None]).double():
        x = x / (x.norm() + eps)
        for _ in range(steps):
            if x.shape[0] <= x.shape[1]:
                m = x @ x.t()
                x = a * x + (b * m + c * (m @ m)) @ x
            else:
                m = x.t() @ x
                x = a * x + x @ (b * m + c * (m @ m))
        out.append(x)
    return torch.stack(out).reshape(u.shape)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("n,k", [(1, 1), (1, 7), (9, 1), (3, 5), (33, 100), (64, 64), (65, 129), (200, 64), (256, 512),
                                 (257, 300), (300, 2049), (512, 2048), (1000, 1000), (2048, 640)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shapes(n, k, dtype):
    g = rand(n, k, seed=n + k).to(dtype)
    got = S.orthogonalize(g)
    assert got.dtype == dtype and got.shape == g.shape
    assert off(got, steps64(g)) < (1e-4 if dtype == F32 else 1e-4 + 2.0 ** -8)


@pytest.mark.parametrize("n,k", [(1300, 1300), (600, 5500), (5500, 600), (1420, 1600), (1090, 4100), (4100, 1090)])
def test_large_tiles_on_ragged_sides(n, k):
    """Sides that no tile divides, padded to 128 and 256; whole steps and steps in groups."""
    g = rand(n, k, seed=n)
    want = steps64(g)
    assert off(S.orthogonalize(g), want) < 1e-4
    w, _ = S.muon_step(torch.zeros_like(g), g, torch.zeros_like(g), 1.0, momentum=0.0, scale=1.0)
    assert off(-w, want) < 1e-4


def spectra(n, k):
    yield rand(n, 8, seed=1) @ rand(8, k, seed=2) + 0.01 * rand(n, k, seed=3)
    yield 0.02 * rand(n, k, seed=4) + rand(n, 1, seed=5) @ rand(1, k, seed=6)
    u, _, v = torch.linalg.svd(rand(n, k, seed=7), full_matrices=False)
    yield (u * torch.logspace(0, -6, u.shape[1], device=DEV)) @ v


@pytest.mark.parametrize("n,k", [(96, 96), (128, 400), (500, 260)])
def test_spectra(n, k):
    for g in spectra(n, k):
        assert off(S.orthogonalize(g), steps64(g)) < 1e-3


def test_singular_values_come_near_one():
    g = rand(256, 700, seed=9)
    s = torch.linalg.svdvals(S.orthogonalize(g).double())
    assert float(s.min()) > 0.6 and float(s.max()) < 1.3


@pytest.mark.parametrize("count", [1, 2, 5])
@pytest.mark.parametrize("n,k", [(48, 200), (300, 130)])
def test_batches(count, n, k):
    g = rand(count, n, k, seed=count)
    got = S.orthogonalize(g)
    assert off(got, steps64(g)) < 1e-4
    for i in range(count):
        assert torch.equal(got[i], S.orthogonalize(g[i]))


@pytest.mark.parametrize("steps", [1, 2, 7])
@pytest.mark.parametrize("coeffs", [None, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)])
def test_steps_and_coefficients(steps, coeffs):
    g = rand(100, 180, seed=steps)
    got = S.orthogonalize(g, steps=steps, coeffs=coeffs)
    assert off(got, steps64(g, steps, coeffs or S.NEWTON_SCHULZ)) < 2e-5 * max(5, steps)


@pytest.mark.parametrize("std", [1e-25, 1e-6, 1e6, 1e25])
def test_scale_of_the_gradient(std):
    g = rand(70, 90, seed=3)
    eps = 1e-7 * min(std, 1.0)
    assert off(S.orthogonalize(g * std, eps=eps), steps64(g * std, eps=eps)) < 1e-4


def test_zero_and_bad_matrices_stay_alone():
    g = rand(4, 65, 80, seed=8)
    clean = S.orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    got = S.orthogonalize(g)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])
    assert not got[1].any() and bool(torch.isnan(got[2]).any())


@pytest.mark.parametrize("n,k", [(96, 256), (260, 96)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(n, k, dtype, nesterov):
    w, g, b = (rand(2, n, k, seed=i, std=s).to(dtype) for i, s in enumerate((0.02, 1e-3, 1e-2)))
    w2, b2 = S.muon_step(w, g, b, 0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1)
    bd = 0.9 * b.double() + g.double()
    u = g.double() + 0.9 * bd if nesterov else bd
    scale = max(1.0, n / k) ** 0.5
    o = steps64(u)
    want = w.double() * (1 - 0.02 * 0.1) - 0.02 * scale * o
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -22
    assert off(b2, bd) < half
    err = (w2.double() - want).norm()
    assert float(err) < 1e-4 * float((0.02 * scale * o).norm()) + half * float(want.norm())


def test_step_scale_and_in_place():
    w, g, b = (rand(64, 96, seed=i) for i in range(3))
    want = S.muon_step(w, g, b, 0.1, scale=0.3)
    w1, b1 = w.clone(), b.clone()
    got = S.muon_step(w1, g, b1, 0.1, scale=0.3, out=(w1, b1))
    assert got[0] is w1 and got[1] is b1
    assert torch.equal(w1, want[0]) and torch.equal(b1, want[1])
    o = S.orthogonalize(g + 0.95 * (0.95 * b + g))
    assert off(want[0], w.double() - 0.03 * o.double()) < 1e-5


def test_strided_unaligned_and_streams():
    base = rand(70 * 81 + 1, seed=4)
    g = base[1:].reshape(70, 81)
    want = S.orthogonalize(g.clone())
    assert torch.equal(S.orthogonalize(g), want)
    assert torch.equal(S.orthogonalize(g.t().contiguous().t()), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = S.orthogonalize(g, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_even_rows_at_any_element(dtype, shift):
    """Rows of a multiple of 8 elements that begin at any element, read there as aligned ones are."""
    base = rand(72 * 80 + shift, seed=shift).to(dtype)
    g = base[shift:].reshape(72, 80)
    w, b = g + 1, g * 2
    assert torch.equal(S.orthogonalize(g), S.orthogonalize(g.clone()))
    assert all(torch.equal(x, y) for x, y in zip(S.muon_step(w, g, b, 0.1), S.muon_step(w, g.clone(), b, 0.1)))


@pytest.mark.parametrize("n,k", [(16384, 16384), (16384, 8)])
def test_longest_sides(n, k):
    """One step at the largest side (1 GB a matrix): some rows against 64 bits."""
    g = rand(n, k, seed=13)
    got = S.orthogonalize(g, steps=1)
    a, b, c = S.NEWTON_SCHULZ
    x = g.double() / (g.double().norm() + 1e-7)
    at = torch.tensor([0, 1, 4097, 9000, 16382, 16383], device=DEV)
    if n <= k:
        m = x @ x.t()
        rows = b * m[at] + c * (m[at] @ m)
        want = a * x[at] + rows @ x
    else:
        m = x.t() @ x
        want = a * x[at] + x[at] @ (b * m + c * (m @ m))
    assert off(got[at], want) < 2e-5


def test_transpose_agrees():
    g = rand(150, 333, seed=11)
    assert off(S.orthogonalize(g.t().contiguous()).t(), S.orthogonalize(g).double()) < 1e-4


def test_refusals():
    w = rand(8, 8)
    for bad in (w[0], w.half(), w.cpu(), w[:0]):
        with pytest.raises(ValueError):
            S.orthogonalize(bad)
    with pytest.raises(ValueError):
        S.orthogonalize(w, steps=0)
    with pytest.raises(ValueError):
        S.orthogonalize(w, out=w[:4])
    with pytest.raises(ValueError):
        S.muon_step(w, w[:4], w, 0.1)
    with pytest.raises(ValueError):
        S.muon_step(w, w.bfloat16(), w, 0.1)
    with pytest.raises(ValueError):
        S.muon_step(w, w, w, float("nan"))


@pytest.mark.parametrize("coeffs,steps", [((2.82, 0.0, 0.0), 2), ((3.3, -0.4, 0.0), 1), ((1.0, 7.9, 0.0), 1),
                                          ((4.2, -5.2, 1.6), 5), ((3.9, -5.2, 1.8), 5), ((-3.4445, 4.775, -2.0315), 3)])
@pytest.mark.parametrize("n,k", [(1, 1), (40, 60), (520, 1200)])
def test_coefficients_at_the_edge(coeffs, steps, n, k):
    """Coefficients that just keep what the steps hold in range, single and (updates of 520 x 1200) grouped: 15
    products of |a| + |b| + |c| ~ 11, 2.5 times as much where steps are grouped."""
    g = torch.ones(1, 1, device=DEV) if n == 1 else rand(n, k, seed=5)
    want = steps64(g, steps, coeffs)
    assert off(S.orthogonalize(g, steps=steps, coeffs=coeffs), want) < 1e-4
    w, _ = S.muon_step(torch.zeros_like(g), g, torch.zeros_like(g), 1.0, momentum=0.0, scale=1.0, steps=steps, coeffs=coeffs)
    assert off(-w, want) < 2.5e-4


def test_coefficients_out_of_range_are_refused():
    g = rand(8, 8)
    for coeffs, steps in (((3.3, -0.4, 0.0), 2), ((8.3, -23.6, 17.3), 5), ((2.83, 0.0, 0.0), 3)):
        with pytest.raises(ValueError):
            S.orthogonalize(g, steps=steps, coeffs=coeffs)
        with pytest.raises(ValueError):
            S.muon_step(g, g, g, 0.1, steps=steps, coeffs=coeffs)


@pytest.mark.parametrize("count,n,k", [(131, 1, 16384), (1030, 256, 200), (4100, 100, 128), (65535, 8, 8), (18, 2048, 2040)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_batches_of_several_launches(count, n, k, dtype):
    """More matrices than are taken at a time (2^26 elements): those around the cuts and some others against 64 bits."""
    g = rand(count, n, k, seed=count)
    g *= torch.logspace(-3, 3, count, device=DEV)[:, None, None]
    g = g.to(dtype)
    up = lambda x: -(-x // 32) * 32  # noqa: E731
    per = (1 << 26) // (up(n) * up(k))
    at = torch.tensor(sorted({0, 1, per - 1, per, per + 1, count // 2, count - 2, count - 1} & set(range(count))), device=DEV)
    want = steps64(g[at])
    got = S.orthogonalize(g)
    half = 2.0 ** -8 if dtype == BF16 else 0.0
    for i in range(len(at)):
        assert off(got[at[i]], want[i]) < 1e-4 + half, int(at[i])
    if dtype == F32:
        w, b = S.muon_step(torch.zeros_like(g), g, g, 1.0, momentum=0.5, nesterov=False, scale=1.0)
        for i in range(len(at)):
            assert off(-w[at[i]], want[i]) < 2.5e-4, int(at[i])
        assert torch.equal(b, 1.5 * g)


def steps32(u, steps=5, coeffs=S.NEWTON_SCHULZ, eps=1e-7):
    """The same steps in plain fp32 products."""
    a, b, c = coeffs
    x = u.float() if u.shape[0] <= u.shape[1] else u.float().t().contiguous()
    x = x / (x.norm() + eps)
    for _ in range(steps):
        m = x @ x.t().contiguous()
        x = a * x + (b * m + c * (m @ m)) @ x
    return x if u.shape[0] <= u.shape[1] else x.t()


def update(g, **kw):
    """orthogonalize(g) as an update of zero weights shows it (steps in groups where the shape takes them)."""
    w, _ = S.muon_step(torch.zeros_like(g), g, torch.zeros_like(g), 1.0, momentum=0.0, scale=1.0, **kw)
    return -w


@pytest.mark.parametrize("n,k", [(200, 700), (600, 1400), (1400, 600), (520, 6100), (1100, 2300), (2300, 1100), (1300, 1300)])
def test_spectra_in_every_form(n, k):
    """Low-rank, spiked and flat spectra on every tile, single and grouped: single steps are as near to 64 bits as
    plain fp32 products, grouped ones within twice that."""
    r = min(n, k) // 8
    cases = [rand(n, k, seed=n), rand(n, r, seed=1) @ rand(r, k, seed=2) * r ** -0.5 + 0.3 * rand(n, k, seed=3),
             rand(n, 8, seed=1) @ rand(8, k, seed=2) + 0.01 * rand(n, k, seed=3),
             0.02 * rand(n, k, seed=4) + rand(n, 1, seed=5) @ rand(1, k, seed=6)]
    for i, g in enumerate(cases):
        want = steps64(g)
        plain = off(steps32(g), want)
        assert off(S.orthogonalize(g), want) < plain, i
        assert off(update(g), want) < 2 * plain, i


@pytest.mark.parametrize("count", [2, 3])
@pytest.mark.parametrize("n,k", [(600, 1400), (1400, 600), (1300, 1300), (1100, 2300)])
def test_batches_on_large_tiles_and_groups(count, n, k):
    """Every matrix of a batch, each of another size of values, by itself against 64 bits."""
    g = torch.stack([rand(n, k, seed=10 + i) * 100.0 ** (1 - i) for i in range(count)])
    want = steps64(g)
    one, grouped = S.orthogonalize(g), update(g)
    for i in range(count):
        assert off(one[i], want[i]) < 1e-5 and off(grouped[i], want[i]) < 2e-5, i


def test_bf16_results_are_rounded_once_and_repeat():
    """2 x 512 x 2048 in bf16, on memory full of NaN: the same bits each time, and those of the 64-bit result's
    rounding but for one element in 500 (an error of 5e-6 of the result lies that often across a rounding)."""
    g = torch.stack([rand(512, 2048, seed=21), 1e-3 * rand(512, 2048, seed=22)]).to(BF16)
    first = S.orthogonalize(g)
    want = steps64(g)
    assert float((first != want.to(BF16)).float().mean()) < 2e-3
    for _ in range(10):
        junk = [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(30)]
        del junk
        assert torch.equal(S.orthogonalize(g), first)


@pytest.mark.parametrize("std", [1e-38, 1e-36, 1e-34, 5e37])
@pytest.mark.parametrize("n,k", [(70, 90), (90, 70), (600, 1400)])
def test_norms_at_the_ends_of_fp32(n, k, std):
    """Without eps the result does not see the gradient's scale (1e-38: most values are subnormal)."""
    g = rand(n, k, seed=6) * std
    want = steps64(g, eps=0.0)
    assert off(S.orthogonalize(g, eps=0.0), want) < 1e-4
    assert off(update(g, eps=0.0), want) < 1e-4


def test_outputs_on_inputs():
    """An output may be an input; the momentum's may not be the weights' (they are read after it is written)."""
    w, g, b = (rand(64, 96, seed=i) for i in range(3))
    want = S.muon_step(w, g, b, 0.1)
    for i in range(3):
        t = [w.clone(), g.clone(), b.clone()]
        got = S.muon_step(*t, 0.1, out=(t[i], torch.empty_like(b)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for out in ((w, w), (g, w), (b, b)):
        with pytest.raises(ValueError):
            S.muon_step(w, g, b, 0.1, out=out)
    flat = torch.zeros(2 * w.numel(), device=DEV)
    with pytest.raises(ValueError):
        S.orthogonalize(flat[:w.numel()].reshape(w.shape), out=flat[4:4 + w.numel()].reshape(w.shape))
