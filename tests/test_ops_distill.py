"""Distillation from a teacher's top logits against its definition in 64 bits,
and its gradient against the formula's and against differences.

Tolerances.  An exponential of the kernels is off by 2^-22 of itself for near
elements and, for an exponent (base 2) of up to 128 in fp32, by at most 2^-18;
sums of a row, weighted by the exponentials, by 2^-21.  A loss is then off by
2^-21 of each logarithm's weight (w t^2 for p and for the rest, 1 - w for the
label), twice for the two sums, and by half a step of fp32; a gradient's
element by 2^-18 of the terms that it is made of, and half a step of its type.
"""

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("ternary_weight_quantization_sparse_amd")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    S.load()


def make(rows, vocab, slots, dtype, tail, labels, seed=0, std=2.5, tau=2.0, wide=False, pad=0, offset=0):
    """Inputs: logits (rows ``pad`` elements further apart, ``offset`` into their memory), teacher, ids, lse, labels."""
    gen = torch.Generator(device=DEV).manual_seed(seed + 13 * rows + vocab)
    store = torch.empty(offset + rows * (vocab + pad), device=DEV, dtype=dtype)
    store.copy_(torch.randn(store.shape, generator=gen, device=DEV) * std)
    z = store[offset:].view(rows, vocab + pad)[:, :vocab]
    teacher = 0.8 * z.float() + torch.randn(rows, vocab, generator=gen, device=DEV)
    u, ids = teacher.topk(min(slots, vocab), 1)
    if slots > vocab:
        u = torch.cat([u, torch.zeros(rows, slots - vocab, device=DEV)], 1)
        ids = torch.cat([ids, torch.full((rows, slots - vocab), -1, device=DEV)], 1)
    u = u.to(dtype)
    lse = torch.logsumexp(teacher / tau, 1) + 0.02 if tail else None
    y = torch.randint(0, vocab, (rows,), generator=gen, device=DEV)
    y[::3] = ids[::3, 0]
    y[1::5] = -100
    return z, u, (ids if wide else ids.to(torch.int32)), lse, ((y if wide else y.to(torch.int32)) if labels else None)


def oracle(z, u, ids, lse, y, tau, w, g):
    """(loss, tolerance, gradient, its terms' sizes) on the host in 64 bits, row by row."""
    z, u, ids = z.detach().cpu().double(), u.cpu().double(), ids.cpu().long()
    rows, vocab = z.shape
    loss, tol = torch.zeros(rows, dtype=F64), torch.zeros(rows, dtype=F64)
    grad, size = torch.zeros(rows, vocab, dtype=F64), torch.zeros(rows, vocab, dtype=F64)
    for r in range(rows):
        used = [(int(i), float(v)) for i, v in zip(ids[r], u[r]) if 0 <= i < vocab]
        at = torch.tensor([i for i, _ in used], dtype=torch.long)
        top = torch.tensor([v for _, v in used], dtype=F64) / tau
        rest = 0.0
        if lse is not None:
            p = torch.exp(top - float(lse[r]))
            rest = max(0.0, 1 - float(p.sum()))
        elif len(used) and top.max() > -float("inf"):
            p = torch.softmax(top, 0)
        else:
            p, at = torch.zeros(0, dtype=F64), at[:0]
        logq = torch.log_softmax(z[r] / tau, 0)
        q = logq.exp()
        outside = torch.ones(vocab, dtype=torch.bool)
        outside[at] = False
        if not outside.any():
            rest = 0.0
        live = p > 0
        kd = (p[live] * (p[live].log() - logq[at[live]])).sum()
        G = (p.sum() + rest) * q
        G2 = G.clone()
        G.index_add_(0, at, -p)
        G2.index_add_(0, at, p)
        if rest > 0:
            # (from the logits: at 1e30 a log of q has steps of 1e14, in which the tail's own differences are lost)
            away = (z[r] / tau).masked_fill(~outside, -float("inf"))
            logr = torch.logsumexp(away, 0) - torch.logsumexp(z[r] / tau, 0)
            kd = kd + rest * (torch.log(torch.tensor(rest, dtype=F64)) - logr)
            tail = rest * torch.softmax(away, 0)
            G, G2 = G - tail, G2 + tail
        if w != 0 and (len(at) or rest > 0):
            loss[r] += w * tau ** 2 * kd
            grad[r] += w * tau * G
            size[r] += w * tau * G2
        tol[r] += abs(w) * tau ** 2 * float(p.sum() + rest) * 2.0 ** -20
        if y is not None and 0 <= int(y[r]) < vocab and w != 1:
            soft = torch.softmax(z[r], 0)
            hot = torch.zeros(vocab, dtype=F64)
            hot[int(y[r])] = 1
            loss[r] += (1 - w) * -torch.log_softmax(z[r], 0)[int(y[r])]
            grad[r] += (1 - w) * (soft - hot)
            size[r] += abs(1 - w) * (soft + hot)
            tol[r] += abs(1 - w) * 2.0 ** -20
    tol += 2.0 ** -24 * loss.abs()
    g = g.cpu().double()[:, None]
    return loss, tol, grad * g, size * g.abs()


def check(z, u, ids, lse, y, tau=2.0, w=0.7, g=None, **kw):
    rows = z.shape[0]
    if g is None:
        g = torch.linspace(0.3, 1.0, rows, device=DEV)
    loss, stats = S.distill_loss(z, u, ids, tau, lse, y, w, with_stats=True)
    grad = S.distill_loss_backward(g, z, ids, stats, tau, y, w, **kw)
    want, tol, dwant, size = oracle(z, u, ids, lse, y, tau, w, g)
    assert ((loss.cpu().double() - want).abs() <= tol).all(), ((loss.cpu().double() - want).abs() / tol).max()
    dtol = 2.0 ** -18 * size + torch.finfo(z.dtype).eps / 2 * dwant.abs() + 1e-36
    err = (grad.cpu().double() - dwant).abs()
    assert grad.dtype == z.dtype and grad.shape == z.shape
    assert (err <= dtol).all(), (err / dtol).max()
    return loss, grad


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("labels", [False, True])
@pytest.mark.parametrize("rows,vocab,slots", [(1, 1, 1), (2, 2, 1), (5, 7, 3), (3, 8, 8), (4, 100, 120), (1, 4099, 64),
                                              (3, 16385, 1), (2, 50001, 20), (70, 1003, 33)])
def test_sizes(rows, vocab, slots, dtype, tail, labels):
    check(*make(rows, vocab, slots, dtype, tail, labels), w=0.7 if labels else 1.0)


@pytest.mark.parametrize("tau,w", [(1.0, 0.5), (1.0, 1.0), (0.5, 0.0), (3.7, 0.25), (20.0, 1.5)])
@pytest.mark.parametrize("tail", [False, True])
def test_temperatures_and_weights(tau, w, tail):
    check(*make(6, 3001, 12, F32, tail, True, tau=tau), tau=tau, w=w)
    check(*make(6, 3001, 12, BF16, tail, True, tau=tau), tau=tau, w=w)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(3, 0), (0, 1), (5, 7), (8, 8)])
def test_rows_at_any_element(dtype, pad, offset):
    check(*make(9, 2050, 10, dtype, True, True, pad=pad, offset=offset))


def test_wide_indexes_and_ids_outside():
    z, u, ids, lse, y = make(7, 5000, 16, BF16, True, True, wide=True)
    ids[0, 3], ids[1, 0], ids[2, :], y[3], y[4] = 5000, -1, 1 << 40, 1 << 33, (1 << 32) + 5
    u[0, 3], u[1, 0], u[2, 4] = float("nan"), float("inf"), float("nan")     # of empty slots: never looked at
    check(z, u, ids, lse, y)
    check(z, u, ids, None, y)


@pytest.mark.parametrize("tail", [False, True])
def test_an_id_in_several_slots(tail):
    z, u, ids, lse, y = make(5, 3000, 70, F32, tail, True)
    ids[:, 5], ids[:, 69], ids[0, 1], y[1] = ids[:, 2], ids[:, 2], ids[0, 0], ids[1, 2]
    check(z, u, ids, lse + 1 if tail else None, y)


def test_ids_are_the_whole_vocabulary():
    z, u, ids, lse, y = make(4, 40, 40, F32, True, False)
    check(z, u, ids, lse, None)              # nothing outside: no tail, though p leaves something of 1
    check(z, u, ids, lse, None, w=1.0)


def test_rows_without_teacher_or_label():
    z, u, ids, lse, y = make(6, 900, 4, F32, False, True)
    ids[1], y[1] = -1, -1
    u[2] = float("-inf")
    y[2] = -1
    loss, grad = check(z, u, ids, None, y)
    assert loss[1] == 0 and loss[2] == 0 and not grad[1].any() and not grad[2].any()
    ids[:] = -1
    z2, _, _, lse2, _ = make(6, 900, 4, F32, True, False)
    loss, grad = check(z2, u, ids, lse2, None, w=1.0)      # the tail is everything: nothing to learn
    assert loss.abs().max() <= 2.0 ** -20 and grad.abs().max() <= 2.0 ** -18


@pytest.mark.parametrize("fill", [float("-inf"), "lowest"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_vocabulary(fill, dtype):
    fill = torch.finfo(dtype).min if fill == "lowest" else fill
    z, u, ids, lse, y = make(5, 3000, 8, dtype, False, True)
    mask = torch.rand(z.shape, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV) < 0.6
    mask[0, 7] = False                       # (a row of nothing but -infinity has no softmax)
    mask.scatter_(1, ids.long(), False)
    mask[torch.arange(5, device=DEV), y.clamp(min=0).long()] = False
    z.masked_fill_(mask, fill)
    mask0 = torch.ones(3000, dtype=torch.bool, device=DEV)      # a row of which only one element is left
    mask0[7] = False
    z[0].masked_fill_(mask0, fill)
    ids[0], y[0] = -1, 7
    loss, grad = check(z, u, ids, None, y)
    assert torch.isfinite(loss).all() and torch.isfinite(grad.float()).all()
    assert not grad[mask & (ids[:, :1] >= 0)].any()
    # the teacher's mass on what the student cannot say
    z[1, ids[1, 0].long()] = float("-inf")
    loss, stats = S.distill_loss(z, u, ids, with_stats=True)
    assert loss[1] == float("inf") and torch.isfinite(loss[[0, 2, 3, 4]]).all()


@pytest.mark.parametrize("gap", [50.0, 300.0, 1e4, 1e30])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_tail_far_below_the_ids(gap, tau, dtype):
    """The student's mass outside the ids is what fp32 exponentials below the largest logit cannot hold."""
    z, u, ids, lse, y = make(5, 2000, 6, dtype, True, True, tau=tau)
    far = torch.ones_like(z, dtype=torch.bool).scatter(1, ids.long(), False)
    z[far] -= gap
    y[0], y[2] = int(far[0].nonzero()[0]), ids[2, 1]
    loss, grad = check(z, u, ids, lse, y, tau=tau)
    assert (loss > gap / 1e3).all() and grad.isfinite().all()
    z[3, far[3]] = float("-inf")                 # what the student cannot say at all
    assert S.distill_loss(z, u, ids, tau, lse)[3] == float("inf")


def test_ids_far_below_the_tail():
    z, u, ids, lse, y = make(4, 2000, 6, F32, True, True)
    z.scatter_add_(1, ids.long(), torch.full(ids.shape, -500.0, device=DEV))
    check(z, u, ids, lse, y)
    check(z, u, ids, None, y)


def test_a_term_of_weight_zero_is_left_out():
    z, u, ids, lse, y = make(4, 900, 6, F32, True, True)
    want = check(z, u, ids, lse, y, w=0.0)
    u[1, 2], lse[2], u[3] = float("nan"), float("nan"), float("inf")
    for tail in (lse, None):
        loss, stats = S.distill_loss(z, u, ids, 2.0, tail, y, 0.0, with_stats=True)
        grad = S.distill_loss_backward(torch.linspace(0.3, 1.0, 4, device=DEV), z, ids, stats, 2.0, y, 0.0)
        assert torch.allclose(loss, want[0], rtol=2.0 ** -20) and torch.allclose(grad, want[1], rtol=2.0 ** -17, atol=1e-9)


def test_not_a_number_stays_in_its_row():
    z, u, ids, lse, y = make(6, 2000, 8, BF16, True, True)
    clean, dclean = check(z, u, ids, lse, y)
    z[1, 5], u[2, 0], lse[3], z[4] = float("nan"), float("nan"), float("nan"), float("inf")
    g = torch.linspace(0.3, 1.0, 6, device=DEV)
    loss, stats = S.distill_loss(z, u, ids, 2.0, lse, y, 0.7, with_stats=True)
    grad = S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7)
    assert loss[1:5].isnan().all() and torch.equal(loss[[0, 5]], clean[[0, 5]])
    assert torch.equal(grad[[0, 5]], dclean[[0, 5]]) and grad[[1, 4]].isnan().any(1).all()
    # rows that no gradient comes to (padding) get zeros
    g[1:5] = 0
    grad = S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7)
    assert not grad[1:5].any() and torch.equal(grad[[0, 5]], dclean[[0, 5]])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 5)])
def test_gradient_in_place_of_the_logits(dtype, pad, offset):
    z, u, ids, lse, y = make(4, 40001, 40, dtype, True, True, pad=pad, offset=offset)
    g = torch.tensor([1.0, 0.0, -2.0, 0.5], device=DEV)
    loss, stats = S.distill_loss(z, u, ids, 2.0, lse, y, 0.7, with_stats=True)
    want = S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7)
    got = S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7, out=z)
    assert got is z and torch.equal(z, want)


def test_padding_of_a_strided_output_is_left_alone():
    z, u, ids, lse, y = make(4, 1001, 6, BF16, False, True)
    g = torch.ones(4, device=DEV)
    _, stats = S.distill_loss(z, u, ids, 2.0, None, y, 0.7, with_stats=True)
    store = torch.full((4, 1024), 7.0, dtype=BF16, device=DEV)
    S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7, out=store[:, 3:1004])
    assert torch.equal(store[:, 3:1004], S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7))
    assert (store[:, :3] == 7).all() and (store[:, 1004:] == 7).all()


def test_gradient_against_differences():
    z, u, ids, lse, y = make(2, 60, 5, F32, True, True, tau=1.5)
    g = torch.tensor([0.7, -1.3], device=DEV)
    loss, stats = S.distill_loss(z, u, ids, 1.5, lse, y, 0.6, with_stats=True)
    grad = S.distill_loss_backward(g, z, ids, stats, 1.5, y, 0.6).cpu().double()
    zd = z.cpu().double()
    h = 1e-5

    def value(zz):
        return (oracle(zz, u, ids, lse, y, 1.5, 0.6, g)[0] * g.cpu().double()).sum()

    for r, i in [(0, int(ids[0, 0])), (0, int(ids[0, 4])), (1, int(y[1].clamp(min=0))), (0, 11), (1, 59), (0, int(y[0]))]:
        up, down = zd.clone(), zd.clone()
        up[r, i] += h
        down[r, i] -= h
        # h^2 of the third derivative (below 10), the loss's 2^-52 over h, and the kernel's own 2^-18
        assert abs(float(value(up) - value(down)) / (2 * h) - float(grad[r, i])) <= 1e-8 + 2.0 ** -18 * 4


def test_autograd():
    z, u, ids, lse, y = make(12, 3000, 9, BF16, True, True)
    z = z.reshape(3, 4, 3000).clone().requires_grad_(True)
    u, ids, lse, y = u.reshape(3, 4, 9), ids.reshape(3, 4, 9), lse.reshape(3, 4), y.reshape(3, 4)
    loss = S.distill_loss_ad(z, u, ids, temperature=2.0, teacher_lse=lse, labels=y, kd_weight=0.7)
    assert loss.shape == (3, 4)
    (grad,) = torch.autograd.grad(loss.sum() / 12, z, retain_graph=True)
    want = oracle(z.detach().reshape(12, -1), u.reshape(12, 9), ids.reshape(12, 9), lse.reshape(-1), y.reshape(-1), 2.0, 0.7,
                  torch.full((12,), 1 / 12))
    err = (grad.reshape(12, -1).cpu().double() - want[2]).abs()
    assert (err <= 2.0 ** -18 * want[3] + 2.0 ** -9 * 2 * want[2].abs() + 1e-36).all()
    (again,) = torch.autograd.grad(loss.mean(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(again.float().sum(), z)
    with pytest.raises(ValueError, match="constant"):
        S.distill_loss_ad(z, u.float().requires_grad_(True), ids)


def test_one_row_without_its_axis():
    z, u, ids, lse, y = make(1, 700, 5, F32, True, True)
    loss, stats = S.distill_loss(z[0], u[0], ids[0], 2.0, lse[0], y[0], 0.7, with_stats=True)
    grad = S.distill_loss_backward(torch.ones((), device=DEV), z[0], ids[0], stats, 2.0, y[0], 0.7)
    want, stats = S.distill_loss(z, u, ids, 2.0, lse, y, 0.7, with_stats=True)
    assert loss.shape == () and loss == want[0] and grad.shape == (700,)
    assert torch.equal(grad, S.distill_loss_backward(torch.ones(1, device=DEV), z, ids, stats, 2.0, y, 0.7)[0])


def test_more_rows_than_one_launch():
    rows = (1 << 22) + 7
    gen = torch.Generator(device=DEV).manual_seed(0)
    z = torch.randn(rows, 3, generator=gen, device=DEV)
    ids = torch.randint(0, 3, (rows, 1), generator=gen, device=DEV)
    u = torch.zeros(rows, 1, device=DEV)
    loss, stats = S.distill_loss(z, u, ids, with_stats=True)
    grad = S.distill_loss_backward(torch.ones(rows, device=DEV), z, ids, stats)
    q = z.double().softmax(1)                    # one slot has all of the teacher: cross entropy
    want = -q.gather(1, ids).log()[:, 0]
    assert ((loss.double() - want).abs() <= 2.0 ** -20 + 2.0 ** -24 * want).all()
    hot = torch.zeros_like(q).scatter(1, ids, 1.0)
    assert ((grad.double() - (q - hot)).abs() <= 2.0 ** -18 * (q + hot)).all()


def test_refusals():
    z, u, ids, lse, y = make(4, 300, 6, BF16, True, True)
    g = torch.ones(4, device=DEV)
    loss, stats = S.distill_loss(z, u, ids, 2.0, lse, y, with_stats=True)
    for args, kw in [((z.half(), u, ids), {}), ((z, u.half(), ids), {}), ((z, u[:3], ids), {}), ((z, u, ids.float()), {}),
                     ((z, u, ids[:, :3]), {}), ((z, u, ids[0]), {}), ((z, u.cpu(), ids), {}), ((z, u, ids.cpu()), {}),
                     ((z, u, ids), dict(temperature=0.0)), ((z, u, ids), dict(teacher_lse=lse.double())),
                     ((z, u, ids), dict(teacher_lse=lse[:2])), ((z, u, ids), dict(labels=y.float())),
                     ((z, u, ids), dict(labels=y[:2])), ((z, u, ids), dict(kd_weight=float("nan"))),
                     ((z, u[:, :0], ids[:, :0]), {}), ((z[:, :0], u, ids), {})]:
        with pytest.raises(ValueError):
            S.distill_loss(*args, **kw)
    for args, kw in [((g.double(), z, ids, stats), {}), ((g[:2], z, ids, stats), {}), ((g, z, ids, stats[:, :5]), {}),
                     ((g, z, ids, stats[:2]), {}), ((g, z, ids, stats.double()), {}), ((g, z, ids, stats.cpu()), {}),
                     ((g, z, ids, stats), dict(out=z.float())), ((g, z, ids, stats), dict(out=z[:2])),
                     ((g, z, ids, stats), dict(out=z.t().contiguous().t())), ((g.cpu(), z, ids, stats), {})]:
        with pytest.raises(ValueError):
            S.distill_loss_backward(*args, temperature=2.0, labels=y, **kw)
    store = torch.zeros(4 * 300 + 8, dtype=BF16, device=DEV)     # over the logits, but not in their place
    with pytest.raises(ValueError):
        S.distill_loss_backward(g, store[:1200].view(4, 300), ids, stats, 2.0, out=store[8:].view(4, 300))


def test_no_rows():
    z = torch.zeros(0, 100, device=DEV, requires_grad=True)
    loss = S.distill_loss_ad(z, torch.zeros(0, 4, device=DEV), torch.zeros(0, 4, dtype=torch.int32, device=DEV))
    assert loss.shape == (0,)
    loss.sum().backward()
    assert z.grad.shape == (0, 100)


def test_repeats_bit_for_bit_and_on_a_stream():
    z, u, ids, lse, y = make(33, 70001, 50, BF16, True, True)
    g = torch.rand(33, device=DEV)
    first = S.distill_loss(z, u, ids, 2.0, lse, y, 0.7, with_stats=True)
    grad = S.distill_loss_backward(g, z, ids, first[1], 2.0, y, 0.7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        loss, stats = S.distill_loss(z, u, ids, 2.0, lse, y, 0.7, with_stats=True, stream=stream)
        again = S.distill_loss_backward(g, z, ids, stats, 2.0, y, 0.7, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(loss, first[0]) and torch.equal(stats, first[1]) and torch.equal(again, grad)


def test_offsets_past_32_bits():
    rows, vocab = 5, (1 << 29) + 3          # 2.1 * 10^9 elements and more from row 4 on
    z = torch.zeros(rows, vocab, dtype=BF16, device=DEV)
    z[4, vocab - 1] = 20.0
    z[4, 5] = 21.0
    ids = torch.tensor([[vocab - 1, 5]], dtype=torch.int32, device=DEV).expand(rows, 2).contiguous()
    u = torch.tensor([[1.0, 2.0]], device=DEV).expand(rows, 2).contiguous()
    loss, stats = S.distill_loss(z, u, ids, with_stats=True)
    p = torch.softmax(torch.tensor([1.0, 2.0], dtype=F64), 0)
    s = torch.tensor([20.0, 21.0], dtype=F64)
    total = torch.logsumexp(torch.cat([s, torch.log(torch.tensor([vocab - 2.0], dtype=F64))]), 0)
    want = (p * (p.log() - (s - total))).sum()
    assert abs(float(loss[4]) - float(want)) <= 2.0 ** -20 + 2.0 ** -24 * float(want)
    grad = S.distill_loss_backward(torch.ones(rows, device=DEV), z, ids, stats, out=z)
    q = torch.exp(s - total)
    assert torch.allclose(grad[4, [vocab - 1, 5]].cpu().double(), q - p, rtol=2.0 ** -8, atol=2.0 ** -18)
    assert abs(float(grad[4, 12345]) - float(torch.exp(-total))) <= 2.0 ** -8 * float(torch.exp(-total))


@pytest.mark.parametrize("rows,vocab,dtype", [(2050, 128000, BF16), (2050, 64003, F32), (2100, 1 << 18, BF16)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_confident_rows_in_long_ranges(rows, vocab, dtype, tail, tau):
    """One range a row, so hundreds of elements a thread: one logit far above a flat rest, whose many small exponentials
    are the loss.  At the row's start, in a thread's middle, in its last groups and at the row's end."""
    z, u, ids, lse, y = make(rows, vocab, 6, dtype, tail, True, std=0.05, tau=tau)
    some = list(range(0, rows, rows // 15))[:16]
    for i, r in enumerate(some):
        at = (0, vocab // 2, vocab - 2100, vocab - 1)[i % 4]
        z[r, at] = (16.0, 18.0, 20.0, 36.0)[i // 4]
        y[r] = at
        if i % 8 < 4:          # the teacher agrees, or says other things
            ids[r, 0], u[r, 0] = at, 12.0
    args = (z, u, ids, tau, lse, y, 0.4)
    loss, stats = S.distill_loss(*args, with_stats=True)
    g = torch.linspace(0.3, 1.0, rows, device=DEV)
    grad = S.distill_loss_backward(g, z, ids, stats, tau, y, 0.4)
    part = [t if t is None else t[some] for t in (z, u, ids, lse, y)]
    want, tol, dwant, size = oracle(*part, tau, 0.4, g[some])
    err = (loss[some].cpu().double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    dtol = 2.0 ** -18 * size + torch.finfo(dtype).eps / 2 * dwant.abs() + 1e-36
    err = (grad[some].cpu().double() - dwant).abs()
    assert (err <= dtol).all(), (err / dtol).max()
    # hard labels alone, whose loss is nothing but the rest's sum
    loss = S.distill_loss(z, u, ids, tau, None, y, 0.0)
    want, tol, _, _ = oracle(*part[:3], None, part[4], tau, 0.0, g[some])
    err = (loss[some].cpu().double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()


def test_label_exponentials_of_far_elements():
    """The label's softmax is as exact far below the largest logit as near it: log2(e) rounded to one fp32 term (1.3e-8 of
    itself too small) would make elements 16 to 20 below 2.1e-7 of themselves larger than ones 0 to 4 below, on the
    average.  What remains: roundings of an exponent (below 32, so 2^-20 ln 2, by chance: divided by the root of 20000
    elements 5e-9), and the exponential's own last place and the row's factor, which are the same near and far."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    z = torch.rand(1, 40000, generator=gen, device=DEV) * 4
    z[0, 20000:] -= 16
    z[0, 0] = 4
    ids = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    y = torch.tensor([[1]], device=DEV).reshape(1)
    loss, stats = S.distill_loss(z, torch.zeros(1, 1, device=DEV), ids, 2.0, None, y, 0.0, with_stats=True)
    grad = S.distill_loss_backward(torch.ones(1, device=DEV), z, ids, stats, 2.0, y, 0.0)
    q = z.cpu().double().softmax(1)      # (on the host: the device's softmax in 64 bits is off by 2e-7 the same way)
    off = (grad.cpu().double() / q - 1)[0]
    assert abs(float(off[20000:].mean() - off[2:20000].mean())) <= 2.0 ** -23
