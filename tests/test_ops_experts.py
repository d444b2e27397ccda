"""The mixture-of-experts layer of packed experts against its definition in 64
bits (the packed experts as the library unpacks them).

Tolerances, as in the product's tests: fp32 sums of K products by steps of 32
and of 128 are off by (K / 32 + K / 128 + 64) 2^-23 of the sum of magnitudes; an
activation by 2^-17 of itself, its argument's error times its slope; h, two
bf16 terms, by 2^-17; a weight of the router by twice its logits' error and
2^-18; y by one rounding."""

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("ternary_weight_quantization_sparse_amd")

from test_ops_linear import act, act_tol, close  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    S.load()


def rand(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


class Layer:
    def __init__(self, experts, dim, hidden, shared=0, grain="per_group", group=128, gated=True, router=BF16, seed=0):
        gen = self.gen = torch.Generator(device=DEV).manual_seed(seed + experts + 3 * dim + hidden)
        total = experts + shared
        self.experts, self.shared, self.dim, self.hidden, self.gated = experts, shared, dim, hidden, gated
        self.up = S.quantize_pack_experts(rand(gen, total, (2 if gated else 1) * hidden, dim, std=0.04), grain, group)
        self.down = S.quantize_pack_experts(rand(gen, total, dim, hidden, std=0.04), grain, group)
        self.router = self.steps(rand(gen, experts, dim, std=1.5 * dim ** -0.5), 512, 0.5).to(router)

    def dense(self, packed, e):
        return S.unpack(S.PackedWeight(packed.packed[e].clone(), packed.alpha[e].clone(), packed.n, packed.k, packed.granularity,
                                       packed.group_size), "float32").double()

    @staticmethod
    def steps(t, per_one, most):
        return ((t * per_one).round() / per_one).clamp(-most, most)

    def tokens(self, m):
        return self.steps(rand(self.gen, m, self.dim), 8, 8).to(BF16), rand(self.gen, m, self.dim, std=0.3, dtype=BF16)

    def oracle(self, x, top_k, scoring, normalize, bias, scale, activation, residual, margin=True):
        """(y, tolerance) in 64 bits."""
        xd, r = x.double(), self.router.double()
        logits = xd @ r.t().contiguous()
        if margin:
            assert (xd.abs() @ r.abs().t().contiguous()).max() * 2 ** 12 < 2 ** 24
        score = logits.softmax(1) if scoring == "softmax" else logits.sigmoid()
        key = logits if bias is None else score + bias.double()     # scores rise with their logits, also where they round to 1
        y = torch.zeros_like(xd) if residual is None else residual.double()
        dy = 2.0 ** -22 * y.abs()
        for t in range(len(x)):
            on = [e for e in range(self.experts) if float(key[t, e]) != -INF]
            rank = sorted(on, key=lambda e: (-float(key[t, e]), e))
            chosen = rank[:top_k]
            if bias is not None and margin and len(rank) > len(chosen) and chosen:   # scores are rounded
                gap = float(key[t, chosen[-1]] - key[t, rank[len(chosen)]])
                assert gap == 0 or gap > 2.0 ** -20, "a draw too near"
            w = score[t, chosen]
            if normalize and len(chosen):
                w = w / w.sum()
            pairs = [(e, float(v) * scale, 2.0 ** -18) for e, v in zip(chosen, w)]
            pairs += [(self.experts + s, 1.0, 0.0) for s in range(self.shared)]
            for e, v, dv in pairs:
                up, down = self.dense(self.up, e), self.dense(self.down, e)
                z, dz = up.mv(xd[t]), (self.dim / 32 + self.dim / 128 + 64) * 2.0 ** -23 * up.abs().mv(xd[t].abs())
                if self.gated:
                    f, u = act(z[:self.hidden], activation), z[self.hidden:]
                    df = act_tol(z[:self.hidden], dz[:self.hidden], activation)
                    h, dh = f * u, df * u.abs() + (f.abs() + df) * dz[self.hidden:]
                else:
                    h, dh = act(z, activation), act_tol(z, dz, activation)
                dh = dh + 2.0 ** -16 * h.abs()
                size = down.abs().mv(h.abs())
                y[t] += v * down.mv(h)
                chain = (len(pairs) * self.hidden / 32 + self.hidden / 128 + 64) * 2.0 ** -23
                dy[t] += abs(v) * ((1 + dv) * down.abs().mv(dh) + (dv + chain) * size)
        return y, dy

    def check(self, m, top_k, scoring="softmax", normalize=True, bias=None, scale=1.0, activation="silu", residual=True,
              x=None, margin=True, **kw):
        x, res = (x, None) if x is not None else self.tokens(m)
        res = res if residual else None
        y = S.moe_decode(x, self.router, self.up, self.down, top_k, shared=self.shared, scoring=scoring,
                         normalize=normalize, bias=bias, scale=scale, activation=activation, residual=res, **kw)
        want, tol = self.oracle(x, top_k, scoring, normalize, bias, scale, activation, res, margin)
        close(y, want, tol)
        return x, res, y


@pytest.mark.parametrize("tokens", [1, 2, 5, 16])
@pytest.mark.parametrize("experts,top_k,shared", [(1, 1, 0), (4, 4, 1), (8, 2, 0), (30, 3, 2), (64, 8, 0), (65, 1, 0),
                                                  (128, 16, 1), (200, 6, 0), (512, 4, 4)])
def test_experts(tokens, experts, top_k, shared):
    Layer(experts, 256, 128, shared).check(tokens, top_k)


@pytest.mark.parametrize("dim,hidden", [(128, 128), (128, 1024), (1152, 384), (2048, 512), (384, 3200)])
@pytest.mark.parametrize("tokens", [1, 7])
@pytest.mark.parametrize("grain,group", [("per_group", 128), ("per_group", 384), ("per_channel", 128), ("per_tensor", 128)])
def test_sizes(dim, hidden, tokens, grain, group):
    group = 128 if dim % group or hidden % group else group
    Layer(5, dim, hidden, 1, grain, group).check(tokens, 2)


@pytest.mark.parametrize("dim", [512, 1024, 2048, 4096, 8192, 8320])
@pytest.mark.parametrize("gated", [False, True])
def test_wide_tiles(dim, gated):
    """64 weight rows a workgroup (4 tokens may use 32 experts), at every count of superblocks a wave."""
    Layer(36, dim, 512, gated=gated).check(4, 8)


@pytest.mark.parametrize("router", [BF16, F32])
@pytest.mark.parametrize("experts,tokens,top_k,hidden", [(8, 16, 2, 4096), (16, 11, 2, 2048), (27, 16, 3, 1024), (60, 7, 8, 512),
                                                         (16, 3, 2, 1024), (32, 5, 4, 256), (64, 2, 8, 128)])
def test_routing_by_itself_and_in_the_first_products(router, experts, tokens, top_k, hidden):
    """A router that one workgroup reads, with few and with many workgroups of first products."""
    Layer(experts, 128, hidden, router=router).check(tokens, top_k)
    Layer(experts, 128, hidden, 1, gated=False, router=router).check(tokens, top_k, "sigmoid", bias=torch.zeros(experts, device=DEV),
                                                                     margin=False)


@pytest.mark.parametrize("hidden", [1024, 1920, 2048, 2176])
def test_items_of_the_second_products(hidden):
    """One to five superblocks a wave in one range, and ranges (4 experts a token)."""
    for tokens in (1, 2):
        Layer(12, 256, hidden).check(tokens, 4)


def test_long_hidden():
    Layer(3, 256, 8320, 1).check(2, 2)
    Layer(3, 8320, 8320).check(1, 1)


def test_a_router_row_that_is_not_a_number():
    layer = Layer(9, 256, 128, 1)
    x, res = layer.tokens(3)
    layer.router[4, 7] = float("nan")
    for normalize in (True, False):
        y = S.moe_decode(x, layer.router, layer.up, layer.down, 2, shared=1, normalize=normalize, residual=res)
        assert y.isnan().all()                   # no softmax without it
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 2, shared=1, scoring="sigmoid", residual=res)
    layer.router[4, 7] = 0                       # a sigmoid for each: the others are chosen before it
    off = torch.zeros(9, device=DEV)
    off[4] = -INF
    want, tol = layer.oracle(x, 2, "sigmoid", True, off, 1.0, "silu", res, margin=False)
    close(y, want, tol)


@pytest.mark.parametrize("activation", ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(activation, gated):
    Layer(6, 256, 256, gated=gated).check(3, 2, activation=activation)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("router", [BF16, F32])
def test_routing(scoring, normalize, biased, router):
    layer = Layer(70, 384, 128, 1, router=router)
    bias = rand(layer.gen, 70, std=0.05) if biased else None
    layer.check(9, 4, scoring, normalize, bias, scale=2.5, y_dtype="float32")
    layer.check(1, 4, scoring, normalize, bias, scale=2.5, residual=False)


@pytest.mark.parametrize("router", [BF16, F32])
def test_router_of_full_precision(router):
    """Logits of any rounding, where every expert is taken.  They are off by (D / 32 + 64) 2^-23 of the sum of
    magnitudes (about 20), below 2^-12, and the weights by at most twice that of themselves; each expert's part of y is
    below y's own largest, six of which are added."""
    layer = Layer(6, 1024, 128, router=router)
    layer.router = rand(layer.gen, 6, 1024, std=0.03, dtype=router)
    x = rand(layer.gen, 5, 1024, dtype=BF16)
    size = (x.double().abs() @ layer.router.double().abs().t().contiguous()).max()
    assert (1024 / 32 + 64) * 2.0 ** -23 * size < 2.0 ** -12
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 6, y_dtype="float32")
    want, tol = layer.oracle(x, 6, "softmax", True, None, 1.0, "silu", None, margin=False)
    close(y, want, tol + 6 * 2.0 ** -11 * want.abs().max())


def test_equal_logits_take_the_lower_index():
    layer = Layer(12, 256, 128)
    layer.router[3], layer.router[7], layer.router[11] = layer.router[1], layer.router[1], layer.router[1]
    for m in (1, 9):
        for top_k in (1, 2, 3, 6):
            layer.check(m, top_k)
    layer.router.zero_()                       # every expert the same, for every token
    layer.check(5, 4, margin=False)
    layer.check(1, 4, bias=torch.zeros(12, device=DEV), margin=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [1, 6])
def test_experts_that_are_off(scoring, tokens):
    layer = Layer(10, 256, 128, 1)
    bias = torch.zeros(10, device=DEV)
    bias[[0, 2, 3, 5, 6, 8, 9]] = -INF
    layer.check(tokens, 2, scoring, bias=bias)
    layer.check(tokens, 5, scoring, bias=bias)                          # three are left
    layer.check(tokens, 5, scoring, normalize=False, bias=bias)
    x, res, y = layer.check(tokens, 3, scoring, bias=torch.full((10,), -INF, device=DEV))   # the shared one alone
    bare = Layer(10, 256, 128, 0)
    x, res = bare.tokens(tokens)
    y = S.moe_decode(x, bare.router, bare.up, bare.down, 3, scoring=scoring, bias=torch.full((10,), -INF, device=DEV),
                     residual=res)
    assert torch.equal(y, res)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_weights_of_far_logits(scoring):
    """Logits of hundreds: weights by their logarithms lose none to another's size."""
    layer = Layer(9, 256, 128, router=F32)
    layer.router *= 32
    layer.check(4, 3, scoring)
    layer.router[:] = -layer.router.abs()
    x = torch.ones(3, 256, dtype=BF16, device=DEV) * torch.tensor([[0.5], [0.25], [0.125]], device=DEV).to(BF16)
    layer.check(3, 2, scoring, x=x)      # (logits of -300 to -50)


def test_tokens_do_not_meet():
    layer = Layer(16, 512, 256, 1)
    x, res, clean = layer.check(8, 3)
    x[2, 9], x[5] = float("nan"), INF
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 3, shared=1, residual=res)
    others = [0, 1, 3, 4, 6, 7]
    assert y[2].isnan().all() and y[5].isnan().any()
    want, tol = layer.oracle(x[others], 3, "softmax", True, None, 1.0, "silu", res[others])
    close(y[others], want, tol)


@pytest.mark.parametrize("value", [INF, float("nan")])
@pytest.mark.parametrize("hidden", [256, 1024])
def test_an_expert_that_is_not_finite_reaches_its_own_tokens_alone(value, hidden):
    """Another expert's scales change nothing of a token's sums, so the others' results stay the same bit for bit."""
    layer = Layer(8, 256, hidden)
    x, res, clean = layer.check(9, 2)
    logits = x.double() @ layer.router.double().t().contiguous()
    chosen = torch.zeros_like(logits).scatter_(1, logits.topk(2, 1).indices, 1)
    e = int(chosen.sum(0).sub(4.5).abs().argmin())          # some take it, some do not
    takes = chosen[:, e] > 0
    assert takes.any() and not takes.all()
    for planes in (layer.up, layer.down):
        kept = planes.alpha[e].clone()
        planes.alpha[e] = value
        y = S.moe_decode(x, layer.router, layer.up, layer.down, 2, residual=res)
        planes.alpha[e] = kept
        assert torch.equal(y[~takes], clean[~takes]) and not y[takes].isfinite().any()


def test_one_expert_for_all_and_all_experts():
    layer = Layer(64, 256, 128)
    x, res = layer.tokens(16)
    layer.check(16, 2, x=x[:1].expand(16, -1).contiguous(), residual=False)
    small = Layer(4, 256, 128)
    small.check(16, 4)


def test_in_place():
    layer = Layer(8, 512, 256)
    x, res, want = layer.check(5, 2)
    args = (layer.router, layer.up, layer.down, 2)
    other = res.clone()
    assert S.moe_decode(x, *args, residual=other, out=other) is other and torch.equal(other, want)
    assert torch.equal(S.moe_decode(x.clone(), *args, residual=res), want)
    own = x.clone()
    assert torch.equal(S.moe_decode(own, *args, residual=own, out=own), S.moe_decode(x, *args, residual=x))


def test_repeats_and_streams():
    layer = Layer(32, 1024, 512)
    x, res, want = layer.check(16, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = [S.moe_decode(x, layer.router, layer.up, layer.down, 4, residual=res, stream=s) for s in (None, side, None)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


def test_experts_past_32_bits():
    """Planes of 2.4 * 10^9 bytes and more: the last experts lie past them."""
    dim, hidden, experts = 4096, 4096, 460
    layer = Layer(2, dim, hidden)
    def grow(p):
        packed = torch.zeros(experts, p.packed.shape[1], dtype=torch.uint8, device=DEV)
        alpha = torch.zeros(experts, p.alpha.shape[1], device=DEV)
        packed[:2], alpha[:2], packed[-2:], alpha[-2:] = p.packed, p.alpha, p.packed, p.alpha
        return S.PackedExperts(packed, alpha, experts, p.n, p.k)
    up, down = grow(layer.up), grow(layer.down)
    assert up.packed.numel() > 1 << 31
    router = torch.zeros(experts, dim, dtype=BF16, device=DEV)
    router[-2:] = layer.router
    x, res = layer.tokens(3)
    bias = torch.full((experts,), -INF, device=DEV)
    bias[-2:] = 0
    y = S.moe_decode(x, router, up, down, 2, bias=bias, residual=res)
    want, tol = layer.oracle(x, 2, "softmax", True, bias[-2:], 1.0, "silu", res)     # (another order of the same sums)
    close(y, want, tol)


def test_refusals():
    layer = Layer(4, 256, 384)
    x, res = layer.tokens(3)
    args = dict(x=x, router=layer.router, up=layer.up, down=layer.down, top_k=2)
    short = S.PackedExperts(layer.up.packed[:3], layer.up.alpha, 4, 768, 256)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x[0]), dict(x=x[:0]), dict(x=x.cpu()), dict(top_k=5), dict(top_k=0),
                dict(shared=1), dict(shared=4), dict(router=layer.router[:3]), dict(router=layer.router.double()),
                dict(scoring="max"), dict(activation="tanh"), dict(bias=torch.zeros(3, device=DEV)), dict(bias=torch.zeros(4)),
                dict(residual=res.float()), dict(residual=res[:2]), dict(out=res.float()), dict(out=res[:2]), dict(up=layer.down),
                dict(up=short), dict(down=layer.up), dict(y_dtype="float16"), dict(x=x[:1].expand(17, -1))):
        with pytest.raises(ValueError):
            S.moe_decode(**{**args, **bad})
    assert S.moe_decode(**args).shape == (3, 256)


def exact_layer(total, n, k, active, gen, grain="per_channel"):
    """Packed weights whose rows have the scale 1, and of each weight only ``active`` rows: sums of integers."""
    p = S.quantize_pack_experts(rand(gen, total, n, k), grain)
    p.alpha.zero_()
    for e in range(total):
        p.alpha[e, torch.randperm(n, generator=gen, device=DEV)[:active]] = 1
    return p


@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden", [(1, 1, 1, 128, 128), (1, 6, 1, 256, 1152), (7, 4, 1, 128, 8192),
                                                             (16, 70, 1, 128, 512)])
@pytest.mark.parametrize("gated", [False, True])
def test_hidden_values_keep_24_bits(tokens, experts, top_k, dim, hidden, gated):
    """Integers of up to 20 and more bits that no sum rounds (their magnitudes add up to less than 2^24), so fp32 results
    are exact: h held in 16 bits would be off by whole units."""
    layer = Layer(experts, dim, hidden, gated=gated)
    gen = layer.gen
    layer.up = exact_layer(experts, (2 if gated else 1) * hidden, dim, hidden if gated else 32, gen)
    layer.down = exact_layer(experts, dim, hidden, dim, gen)
    if gated:       # 24 hidden values of which both factors count
        layer.up.alpha.zero_()
        for e in range(experts):
            at = torch.randperm(hidden, generator=gen, device=DEV)[:24]
            layer.up.alpha[e, at], layer.up.alpha[e, hidden + at] = 1, 1
    top = 8 if gated else 17
    power = torch.randint(0, top, (tokens, dim), generator=gen, device=DEV)
    power[:, 64:] = 0       # (64 of the channels large, whatever dim is)
    sign = torch.randint(0, 2, (tokens, dim), generator=gen, device=DEV) * 2.0 - 1
    x = (sign * torch.exp2(power.float())).to(BF16)
    y = S.moe_decode(x, layer.router, layer.up, layer.down, top_k, activation="none", y_dtype="float32")
    chosen = (x.double() @ layer.router.double().t().contiguous()).argmax(1)
    bits = 0
    for t in range(tokens):
        up, down = layer.dense(layer.up, int(chosen[t])), layer.dense(layer.down, int(chosen[t]))
        z = up.mv(x[t].double())
        h = z[:hidden] * z[hidden:] if gated else z
        assert h.abs().sum() < 2 ** 24 and up.abs().mv(x[t].double().abs()).max() < 2 ** 24
        bits = max(bits, float((h.abs() / torch.exp2(torch.floor(torch.log2(h.abs().clamp(min=1)) - 16)) % 1).max()))
        assert torch.equal(y[t].double(), down.mv(h))
    assert bits > 0       # some have more than 17


def test_hidden_values_beyond_bfloat16():
    """A finite h past the largest bf16 (3.39e38) stays finite."""
    layer = Layer(2, 128, 128, gated=False)
    for e in range(2):
        layer.up.alpha[e], layer.down.alpha[e] = 1, 2.0 ** -100
    t = layer.dense(layer.up, 0)[5].sign()
    x = torch.zeros(1, 128, dtype=BF16, device=DEV)
    at = t.nonzero()[:2, 0]
    x[0, at] = (t[at] * torch.tensor([255 * 2.0 ** -7, 255 * 2.0 ** -15], device=DEV)).to(BF16)
    layer.router[:] = 0       # equal logits: the first one
    layer.up.alpha[0, 5] = 2.0 ** 127
    h = layer.dense(layer.up, 0).mv(x[0].double())
    assert torch.finfo(BF16).max * (1 + 2.0 ** -9) < h[5] < torch.finfo(F32).max
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 1, activation="none", y_dtype="float32")
    want = layer.dense(layer.down, 0).mv(h)
    # a sum of which one term is of the order of 2^27 and the others are below it: by steps of fp32
    assert ((y[0].double() - want).abs() <= 2.0 ** -22 * 2.0 ** 28).all() and y.isfinite().all()


def test_experts_that_do_not_stand_back_to_back():
    """Planes or scales with room after each expert are refused; more experts than are counted, and one flat tensor of
    them, are read as they stand."""
    layer = Layer(4, 256, 384)
    x, res, want = layer.check(3, 2)
    run = lambda up, down: S.moe_decode(x, layer.router, up, down, 2, residual=res)     # noqa: E731
    new = lambda p, packed, alpha: S.PackedExperts(packed, alpha, 4, p.n, p.k)           # noqa: E731
    pad = torch.nn.functional.pad
    for which in ("up", "down"):
        p, both = getattr(layer, which), {"up": layer.up, "down": layer.down}
        for name, bad in (("packed", new(p, pad(p.packed, (0, 16)), p.alpha)), ("alpha", new(p, p.packed, pad(p.alpha, (0, 4)))),
                          ("packed", new(p, pad(p.packed, (0, 16)).view(4, 4, -1), p.alpha))):
            with pytest.raises(ValueError, match=f"{which}: {name}"):
                run(**{**both, which: bad})
        for good in (new(p, pad(p.packed, (0, 0, 0, 1)), pad(p.alpha, (0, 0, 0, 2))), new(p, p.packed.flatten(), p.alpha.flatten()),
                     new(p, pad(p.packed.flatten(), (0, 16)), p.alpha.view(4, -1, 128))):
            assert torch.equal(run(**{**both, which: good}), want)


@pytest.mark.parametrize("experts,dim", [(6, 256), (70, 512)])
@pytest.mark.parametrize("normalize", [False, True])
def test_a_float32_router_at_the_ends_of_its_range(experts, dim, normalize):
    """Infinite entries of the router give the logits that they give by definition, and finite ones past the largest bf16
    stay finite."""
    layer = Layer(experts, dim, 128, router=F32)
    x, res = layer.tokens(4)
    x[:, 3:6] = torch.tensor([2.0, -0.5, 2.0 ** -127], device=DEV).to(BF16)
    layer.router[1, 3], layer.router[2, 4], layer.router[4, 3] = INF, INF, -INF       # logits inf, -inf, -inf
    layer.router[3, 5] = torch.finfo(F32).max                                          # adds 2
    layer.router[5, 5] = -torch.finfo(F32).max
    logits = x.double() @ layer.router.double().t().contiguous()
    assert (logits[:, 1] == INF).all() and (logits[:, 2] == -INF).all() and logits[:, [0, 3, 5]].isfinite().all()
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 4, scoring="sigmoid", normalize=normalize, residual=res)
    want, tol = layer.oracle(x, 4, "sigmoid", normalize, None, 1.0, "silu", res, margin=False)
    close(y, want, tol)
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 4, residual=res)
    assert y.isnan().all()                     # no softmax of an infinite logit
    layer.router[1, 3] = 0
    layer.check(4, 4, x=x, residual=False, margin=False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("experts,dim,hidden,tokens,top_k", [
    (8, 2048, 8192, 1, 2), (8, 2048, 8192, 1, 1), (8, 1024, 4096, 2, 2), (4, 512, 8192, 2, 1),      # wide, 4 and 8 waves
    (4, 4096, 512, 1, 2), (4, 4096, 8192, 1, 2), (2, 4096, 384, 3, 1),                             # 16 waves, narrow and wide
    (2, 8192, 384, 1, 2), (2, 8192, 8192, 1, 1), (1, 8320, 256, 2, 1), (1, 8320, 8192, 1, 1)])
def test_routing_in_the_first_products_at_every_count_of_waves(experts, dim, hidden, tokens, top_k, gated):
    """At most 64 KB of router and tokens and 512 workgroups of first products: each of them makes the routing for
    itself, and the waves share the channels of its tiles."""
    used = min(experts, tokens * top_k)
    rows = hidden * (2 if gated else 1)
    tile = (32 if gated else 64) if rows // 64 * used >= 256 else 16
    assert (experts + tokens) * 2 * dim <= 65536 and hidden // tile * used <= 512
    Layer(experts, dim, hidden, gated=gated).check(tokens, top_k)


@pytest.mark.parametrize("experts,dim,tokens", [(6, 256, 3), (70, 256, 3), (40, 2048, 16)])
def test_no_softmax_for_outputs_of_scale_zero_either(experts, dim, tokens):
    """Without a softmax a token's weights are not numbers, nor is their product with a row of zeros."""
    layer = Layer(experts, dim, 128)
    x, res = layer.tokens(tokens)
    for e in range(experts):
        layer.down.alpha[e].view(-1, dim)[:, ::3] = 0
    x[:, 0] = 1                              # of token 1 the logit of expert 2 is not a number
    x[1, 0] = 0
    layer.router[2, 0] = INF
    y = S.moe_decode(x, layer.router, layer.up, layer.down, 2, scoring="softmax", residual=res)
    assert y.isnan().all()
    x[:, 0], x[1, 0] = 0, 1
    layer.router[2, 0] = 0
    layer.router[2, 1] = float("nan")
    assert S.moe_decode(x, layer.router, layer.up, layer.down, 2, residual=res).isnan().all()
