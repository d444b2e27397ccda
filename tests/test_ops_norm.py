"""Block norms on the GPU against the formulas in 64 bits.

Tolerances.  Sums are fp32 with at most 64 terms in a row (a thread's channels,
then a tree), so a sum's error is below 2^-18 of the sum of its absolute terms;
every output is at most a few such factors and sums, so it is bounded by
2^-16 of the same expression in absolute values.  A bf16 output adds half an
ulp, 2^-8 of the value at most."""

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("ternary_weight_quantization_sparse_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
REL = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    S.load()


def inputs(rows, dim, dtype, wdtype, gate, seqs=1, seed=0, shift=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1000 * rows + dim)

    def rand(*shape, std=1.0, dt=dtype):
        n = 1
        for s in shape:
            n *= s
        flat = torch.randn(n + shift, generator=g, device=DEV) * std
        return flat.to(dt)[shift:].reshape(shape)

    shape = {None: None, "channel": (dim,), "token": (rows, 1), "rows": (seqs, dim)}[gate]
    return dict(h=rand(rows, dim, std=2.0), w_pre=1 + rand(dim, std=0.2, dt=wdtype), y=rand(rows, dim),
                w_post=1 + rand(dim, std=0.2, dt=wdtype), gate=None if shape is None else rand(*shape)), \
        (rand(rows, dim), rand(rows, dim))


def spread(gate, rows, dim):
    """The gate over [rows, dim], and the sum of such a field back to its shape."""
    if gate is None:
        return torch.ones((), dtype=torch.float64, device=DEV), None
    g = gate.double()
    if gate.dim() == 2 and gate.shape == (rows, 1) and dim > 1:
        return g, lambda f: f.sum(1, keepdim=True)
    if gate.dim() == 1:
        return g, lambda f: f.sum(0)
    return g.repeat_interleave(rows // gate.shape[0], 0), lambda f: f.reshape(gate.shape[0], -1, dim).sum(1)


def reference(a, dh, dn, scale, eps, absolute=False):
    """Outputs and gradients in 64 bits; with ``absolute`` every term's magnitude
    added up instead, which bounds the rounding errors."""
    sg = (lambda t: t.abs()) if absolute else (lambda t: t)
    minus = 1.0 if absolute else -1.0
    d = {k: None if v is None else sg(v.double()) for k, v in a.items()}
    exact = {k: None if v is None else v.double() for k, v in a.items()}
    rows, dim = a["h"].shape
    g, back = spread(d["gate"] if a["gate"] is None else sg(a["gate"].double()), rows, dim)
    ge, _ = spread(a["gate"], rows, dim)
    one = torch.ones((), dtype=torch.float64, device=DEV)
    if a["y"] is None:
        h2, h2e = d["h"], exact["h"]
    else:
        r_y = one if a["w_post"] is None else (exact["y"].pow(2).mean(1, keepdim=True) + eps).rsqrt()
        wq, wqe = (one, one) if a["w_post"] is None else (d["w_post"], exact["w_post"])
        p = wq * (d["y"] * r_y)
        h2 = abs(scale) * d["h"] + g * p if absolute else scale * d["h"] + g * p
        h2e = scale * exact["h"] + ge * (wqe * exact["y"] * r_y)
    out = {"h": h2}
    t = sg(dh.double()) if dh is not None else torch.zeros_like(h2)
    if a["w_pre"] is not None:
        r_h = (h2e.pow(2).mean(1, keepdim=True) + eps).rsqrt()
        hh = h2 * r_h
        out["n"] = d["w_pre"] * hh
        dnd = sg(dn.double()) if dn is not None else torch.zeros_like(h2)
        u = d["w_pre"] * dnd
        t = t + r_h * (u + minus * hh * (u * hh).mean(1, keepdim=True))
        out["dw_pre"] = (dnd * hh).sum(0)
    out["dh"] = (abs(scale) if absolute else scale) * t if a["y"] is not None else t
    if a["y"] is not None:
        q = g * t
        if back is not None:
            out["dgate"] = back(t * p)
        v = q * wq
        if a["w_post"] is not None:
            yh = d["y"] * r_y
            out["dw_post"] = (q * yh).sum(0)
            out["dy"] = r_y * (v + minus * yh * (v * yh).mean(1, keepdim=True))
        else:
            out["dy"] = v
    return out


def close(name, got, want, size):
    got = got.double()
    tol = REL * size.reshape(got.shape) + 1e-30
    if name[1] == BF16:
        tol = tol + 2.0 ** -8 * (want.reshape(got.shape).abs() + tol)
    bad = (got - want.reshape(got.shape)).abs() > tol
    assert not bool(bad.any()) and bool(torch.isfinite(got).all()), \
        (name, int(bad.sum()), float(((got - want.reshape(got.shape)).abs() / tol).max()))


def check(a, dh, dn, scale=0.75, eps=1e-5, stream=None):
    kw = dict(a, res_scale=scale if a["y"] is not None else 1.0, eps=eps)
    h = kw.pop("h")
    want = reference(a, dh, dn, scale, eps)
    size = reference(a, dh, dn, scale, eps, absolute=True)
    h2, n = S.block_norm(h, stream=stream, **kw)
    got = dict(zip(("dh", "dw_pre", "dy", "dw_post", "dgate"),
                   S.block_norm_backward(dh, dn, h, stream=stream, **kw)))
    torch.cuda.synchronize()
    got["h"], got["n"] = h2, n
    for k, v in got.items():
        assert (v is None) == (k not in want), k
        if v is not None:
            close((k, v.dtype), v, want[k], size[k])


DIMS = [1, 7, 64, 100, 512, 513, 1001, 1024, 2048, 2500, 4096, 5000, 8192, 8200, 9001]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
def test_widths(dim, dtype, wdtype):
    a, (dh, dn) = inputs(9, dim, dtype, wdtype, "channel")
    check(a, dh, dn)


@pytest.mark.parametrize("rows,seqs", [(1, 1), (2, 2), (3, 1), (6, 3), (600, 600), (600, 300), (1500, 3), (1023, 341),
                                       (2100, 7), (4099, 1)])
@pytest.mark.parametrize("gate", [None, "channel", "token", "rows"])
@pytest.mark.parametrize("dim,dtype", [(256, BF16), (2048, BF16), (129, F32)])
def test_rows_and_gates(rows, seqs, gate, dim, dtype):
    a, (dh, dn) = inputs(rows, dim, dtype, F32, gate, seqs)
    check(a, dh, dn)


@pytest.mark.parametrize("dim", [512, 2048, 9000])
@pytest.mark.parametrize("gate,seqs", [("token", 1), ("rows", 2), ("rows", 12), ("rows", 6)])
def test_long_rows_and_gates(dim, gate, seqs):
    a, (dh, dn) = inputs(12, dim, BF16, F32, gate, seqs)
    check(a, dh, dn)


@pytest.mark.parametrize("drop", [("w_pre",), ("w_post",), ("gate",), ("w_post", "w_pre"), ("w_post", "gate"),
                                  ("y", "w_post", "gate"), ("w_pre", "gate")])
@pytest.mark.parametrize("dim", [40, 2048, 8448])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_absent_parts(drop, dim, dtype):
    a, (dh, dn) = inputs(515, dim, dtype, F32, "channel")
    for k in drop:
        a[k] = None
    check(a, dh, dn)


@pytest.mark.parametrize("which", ["dh", "dn"])
def test_one_incoming_gradient(which):
    a, (dh, dn) = inputs(70, 1024, BF16, F32, "channel")
    check(a, dh if which == "dh" else None, dn if which == "dn" else None)


@pytest.mark.parametrize("dim", [64, 96, 2048])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_unaligned_rows(dim, dtype):
    a, (dh, dn) = inputs(33, dim, dtype, F32, "rows", 11, shift=1)
    assert a["h"].data_ptr() % 16 != 0
    check(a, dh, dn)


def test_strided_inputs_and_leading_shape():
    a, (dh, dn) = inputs(64, 256, F32, F32, "channel")
    t = {k: None if v is None else (v.t().contiguous().t() if v.dim() == 2 else v) for k, v in a.items()}
    check(t, dh.t().contiguous().t(), dn)
    h, n = S.block_norm(a["h"].reshape(4, 16, 256), a["w_pre"], a["y"].reshape(4, 16, 256), a["w_post"], a["gate"])
    h1, n1 = S.block_norm(a["h"], a["w_pre"], a["y"], a["w_post"], a["gate"])
    assert h.shape == (4, 16, 256) and torch.equal(h.reshape(64, 256), h1) and torch.equal(n.reshape(64, 256), n1)


def test_no_rows():
    h = torch.zeros(0, 128, device=DEV, dtype=BF16)
    w = torch.ones(128, device=DEV)
    h2, n = S.block_norm(h, w, h, w)
    assert h2.shape == n.shape == (0, 128)
    dh, dw_pre, dy, dw_post, dgate = S.block_norm_backward(h, h, h, w, h, w, torch.ones(128, device=DEV, dtype=BF16))
    assert dh.shape == dy.shape == (0, 128) and not dw_pre.any() and not dw_post.any() and not dgate.any()


@pytest.mark.parametrize("dim", [96, 2048, 8200])
def test_a_bad_row_stays_alone(dim):
    """An infinity, a NaN and a row of zeros: every other row keeps its bits."""
    a, (dh, dn) = inputs(20, dim, F32, F32, "rows", 20)
    kw = {k: v for k, v in a.items() if k != "h"}
    clean = S.block_norm(a["h"], **kw) + S.block_norm_backward(dh, dn, a["h"], **kw)[::2]
    h, y = a["h"].clone(), a["y"].clone()
    h[3, 5], y[7, 1], h[11], y[11] = float("inf"), float("nan"), 0, 0
    kw["y"] = y
    got = S.block_norm(h, **kw) + S.block_norm_backward(dh, dn, h, **kw)[::2]
    ok = torch.tensor([i not in (3, 7, 11) for i in range(20)], device=DEV)
    for g, c in zip(got, clean):
        if g.shape == (20, dim):
            assert torch.equal(g[ok], c[ok])
    assert torch.isfinite(got[0][11]).all() and not got[1][11].any()


def test_large_and_small_values():
    for std in (1e-12, 1e12):
        a, (dh, dn) = inputs(8, 512, F32, F32, None)
        a["h"], a["y"] = a["h"] * std, a["y"] * std
        check(a, dh, dn, eps=0.0)


@pytest.mark.parametrize("power", [-45, 45])
@pytest.mark.parametrize("dim", [100, 512, 2048, 9001])
def test_gradients_scale_back(dim, power):
    """Norms do not see a power of two: rows 2^45 times as large or small have gradients as much
    smaller or larger, to the bit (every product is exact but for its rounding)."""
    a, (_, dn) = inputs(8, dim, F32, F32, None)
    by = 2.0 ** power
    want = S.block_norm_backward(None, dn, a["h"], a["w_pre"], eps=0.0)
    got = S.block_norm_backward(None, dn, a["h"] * by, a["w_pre"], eps=0.0)
    assert torch.equal(got[0] * by, want[0]) and torch.equal(got[1], want[1])
    want = S.block_norm_backward(dn, None, a["h"], y=a["y"], w_post=a["w_post"], eps=0.0)
    got = S.block_norm_backward(dn, None, a["h"], y=a["y"] * by, w_post=a["w_post"], eps=0.0)
    assert torch.equal(got[2] * by, want[2]) and torch.equal(got[3], want[3])


def test_another_stream():
    a, (dh, dn) = inputs(300, 2048, BF16, F32, "channel")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(a, dh, dn, stream=s)


def test_rows_past_32_bit_offsets():
    """2.3e9 elements: the last rows are what the same rows by themselves are."""
    dim, w = 2048, torch.rand(2048, device=DEV) + 0.5
    h = torch.randn(1100003, dim, device=DEV, dtype=BF16)
    end = h[-9:].clone()
    out = S.block_norm(h, w, y=h, w_post=w, res_scale=0.5)
    for got, want in zip(out, S.block_norm(end, w, y=end, w_post=w, res_scale=0.5)):
        assert torch.equal(got[-9:], want)
    del out
    grads = S.block_norm_backward(h, h, h, w, y=h, w_post=w)
    want = S.block_norm_backward(end, end, end, w, y=end, w_post=w)
    assert torch.equal(grads[0][-9:], want[0]) and torch.equal(grads[2][-9:], want[2])


def test_repeats_bit_for_bit():
    a, (dh, dn) = inputs(3000, 1024, BF16, F32, "rows", 3)
    kw = {k: v for k, v in a.items() if k != "h"}
    first = S.block_norm_backward(dh, dn, a["h"], **kw)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, S.block_norm_backward(dh, dn, a["h"], **kw)))


@pytest.mark.parametrize("gate,seqs", [("channel", 1), ("token", 1), ("rows", 4), ("rows", 16)])
def test_gradients_against_differences(gate, seqs):
    """The directional derivative of sum(c1 h' + c2 n) by central differences of
    the fp32 forward: truncation ~ e^2, rounding ~ 2^-23 sqrt(size) / e of the
    terms; with e = 2^-6 both stay below 1e-3 of the derivative's scale."""
    a, (c1, c2) = inputs(16, 384, F32, F32, gate, seqs)
    names = [k for k in a if a[k] is not None]
    d = {k: torch.randn(a[k].shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)) for i, k in
         enumerate(names)}

    def value(e):
        x = {k: (a[k].double() + e * d[k].double()).float() if a[k] is not None else None for k in a}
        h, n = S.block_norm(res_scale=0.9, **x)
        return float((c1.double() * h.double()).sum() + (c2.double() * n.double()).sum())

    e = 2.0 ** -6
    # Richardson: the e^2 term of the central difference removed
    diff = (8 * (value(e / 2) - value(-e / 2)) - (value(e) - value(-e))) / (6 * e)
    leaves = {k: a[k].clone().requires_grad_(True) for k in names}
    h, n = S.block_norm_ad(res_scale=0.9, **{k: leaves.get(k) for k in a})
    grads = torch.autograd.grad((h, n), [leaves[k] for k in names], (c1, c2))
    parts = [float((g.double() * d[k].double()).sum()) for k, g in zip(names, grads)]
    scale = sum(float((g.double() * d[k].double()).pow(2).sum()) ** 0.5 for k, g in zip(names, grads))
    assert abs(sum(parts) - diff) < 1e-3 * scale, (sum(parts), diff, scale)


def test_autograd_partial_graphs():
    a, (c1, c2) = inputs(12, 256, F32, F32, "channel")
    kw = {k: v for k, v in a.items() if k not in ("h", "y")}
    want = S.block_norm_backward(c1, None, a["h"], y=a["y"], **kw)
    h, y = a["h"].clone().requires_grad_(True), a["y"].clone().requires_grad_(True)
    h2, _ = S.block_norm_ad(h, y=y, **kw)
    gh, gy = torch.autograd.grad(h2, (h, y), c1)
    assert torch.equal(gh, want[0]) and torch.equal(gy, want[2])
    h0, n0 = S.block_norm_ad(h, a["w_pre"])
    (g,) = torch.autograd.grad((h0 * 2 + n0).sum(), h)
    ones = torch.ones_like(a["h"])
    ref = S.block_norm_backward(2 * ones, ones, a["h"], a["w_pre"])[0]
    assert torch.equal(g, ref)


def test_second_derivatives_are_refused():
    """The gradients have no gradient of their own: asking for one raises."""
    h = torch.randn(3, 64, device=DEV, requires_grad=True)
    _, n = S.block_norm_ad(h, torch.ones(64, device=DEV))
    (g,) = torch.autograd.grad(n.sum(), h, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad((g + h).sum(), h)


def test_refusals():
    h, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    for kw in (dict(), dict(w_pre=w[:32]), dict(w_pre=w, w_post=w), dict(w_pre=w, res_scale=0.5),
               dict(w_pre=w, y=h[:2]), dict(w_pre=w, y=h.bfloat16()), dict(w_pre=w, y=h, gate=w.bfloat16()),
               dict(w_pre=w, y=h, gate=torch.zeros(3, 64, device=DEV)), dict(w_pre=w.bfloat16(), y=h, w_post=w),
               dict(w_pre=w, eps=-1.0), dict(w_pre=w.cpu()), dict(w_pre=w.half())):
        with pytest.raises(ValueError):
            S.block_norm(h, **kw)
    with pytest.raises(ValueError):
        S.block_norm(h.half(), w)
    with pytest.raises(ValueError):
        S.block_norm_backward(h[:2], None, h, w)


@pytest.mark.parametrize("rows,dim,gate", [((1 << 26) + 8, 8, "token"), ((1 << 26) + 8, 8, "rows"), ((1 << 24) + 3, 129, None)])
def test_rows_of_more_than_one_launch(rows, dim, gate):
    """More rows than the 2^32 threads of a launch hold: every row is what it is in a call of its own part."""
    g = torch.Generator(device=DEV).manual_seed(2)
    h = torch.randn(rows, dim, generator=g, device=DEV, dtype=BF16)
    w = torch.rand(dim, generator=g, device=DEV) + 0.5
    gates = {None: None, "token": torch.randn(rows, 1, generator=g, device=DEV, dtype=BF16),
             "rows": torch.randn(rows // 8, dim, generator=g, device=DEV, dtype=BF16)}[gate]

    def call(part):
        if gate is None:
            return S.block_norm(h[part], w)[1:]
        per = 8 if gate == "rows" else 1
        return S.block_norm(h[part], w, y=h[part], w_post=w, gate=gates[part.start // per:part.stop // per])

    out = call(slice(0, rows))
    step = 1 << 22
    for at in range(0, rows, step):
        part = slice(at, min(at + step, rows))
        assert all(torch.equal(a[part], b) for a, b in zip(out, call(part))), at


@pytest.mark.parametrize("dim", [100, 2048, 9001])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_an_unused_norm_takes_no_part(dim, eps):
    """No gradient from n: the others are those of a call without its norm, whatever h' holds, and dw_pre is zero."""
    a, (dh, _) = inputs(12, dim, F32, F32, "channel")
    a["h"][3, 5], a["h"][4], a["y"][4] = float("inf"), 0, 0
    kw = {k: v for k, v in a.items() if k not in ("h", "w_pre")}
    got = S.block_norm_backward(dh, None, a["h"], a["w_pre"], eps=eps, **kw)
    want = S.block_norm_backward(dh, None, a["h"], eps=eps, **kw)
    assert torch.equal(got[0], want[0]) and bool(torch.isfinite(got[0]).all()) and torch.equal(got[0], dh)
    for i in (2, 3, 4):
        assert torch.equal(got[i].nan_to_num(7.0), want[i].nan_to_num(7.0))
    assert got[1].shape == (dim,) and not got[1].any()
    alone = S.block_norm_backward(dh, None, a["h"], a["w_pre"], eps=eps)
    assert torch.equal(alone[0], dh) and not alone[1].any()
