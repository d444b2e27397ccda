"""Distillation, the product with an epilogue and the mixture of experts
(include/sherry_ops.h) without a GPU: workspace sizes and every refusal before
any launch.  Each rejected call has one invalid argument and addresses that are
never read."""

import pytest

S = pytest.importorskip("ternary_weight_quantization_sparse_amd")
torch = pytest.importorskip("torch")
L = S._lib

P, MIS2, MIS4 = 0x10000, 0x10001, 0x10002
NONE = (1 << 64) - 1


@pytest.fixture(scope="module")
def lib():
    return L.load()


def distill(lib, rows=4, vocab=100, z=P, stride=100, dt=L.F32, u=P, ut=L.F32, ids=P, wide=0, slots=8, tau=2.0, lse=P,
            y=P, ywide=0, w=0.5, loss=P, stats=P, ws=P, wsb=1 << 30):
    return lib.sherry_distill_loss(rows, vocab, z, stride, dt, u, ut, ids, wide, slots, tau, lse, y, ywide, w, loss, stats,
                                   ws, wsb, None)


def distill_bwd(lib, rows=4, vocab=100, g=P, z=P, stride=100, dt=L.F32, ids=P, wide=0, slots=8, tau=2.0, y=P, ywide=0,
                w=0.5, stats=P, dz=1 << 40, dstride=100):
    return lib.sherry_distill_loss_backward(rows, vocab, g, z, stride, dt, ids, wide, slots, tau, y, ywide, w, stats, dz,
                                            dstride, None)


DISTILL_BAD = [
    (dict(rows=0), L.ERR_ARG), (dict(rows=1 << 31), L.ERR_ARG), (dict(vocab=0), L.ERR_ARG),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), L.ERR_ARG), (dict(stride=99), L.ERR_ARG), (dict(stride=1 << 60), L.ERR_ARG),
    (dict(slots=0), L.ERR_ARG), (dict(slots=1025), L.ERR_ARG), (dict(tau=0.0), L.ERR_ARG), (dict(tau=-1.0), L.ERR_ARG),
    (dict(tau=float("nan")), L.ERR_ARG), (dict(tau=1e4), L.ERR_ARG), (dict(w=float("inf")), L.ERR_ARG),
    (dict(dt=L.I8), L.ERR_DTYPE), (dict(z=None), L.ERR_NULL), (dict(ids=None), L.ERR_NULL), (dict(z=MIS4), L.ERR_ALIGN),
    (dict(z=MIS2, dt=L.BF16), L.ERR_ALIGN), (dict(ids=MIS4), L.ERR_ALIGN), (dict(ids=P + 4, wide=1), L.ERR_ALIGN),
    (dict(y=MIS4), L.ERR_ALIGN), (dict(y=P + 4, ywide=1), L.ERR_ALIGN)]


@pytest.mark.parametrize("kw,code", DISTILL_BAD + [
    (dict(ut=L.I8), L.ERR_DTYPE), (dict(u=None), L.ERR_NULL), (dict(loss=None), L.ERR_NULL), (dict(u=MIS4), L.ERR_ALIGN),
    (dict(lse=MIS4), L.ERR_ALIGN), (dict(stats=MIS4), L.ERR_ALIGN), (dict(ws=None), L.ERR_WORKSPACE),
    (dict(wsb=8), L.ERR_WORKSPACE), (dict(ws=P + 8), L.ERR_ALIGN)])
def test_distill_rejects(lib, kw, code):
    assert distill(lib, **kw) == code


@pytest.mark.parametrize("kw,code", DISTILL_BAD + [
    (dict(g=None), L.ERR_NULL), (dict(stats=None), L.ERR_NULL), (dict(dz=None), L.ERR_NULL), (dict(dstride=99), L.ERR_ARG),
    (dict(dz=(1 << 40) + 2), L.ERR_ALIGN), (dict(g=MIS4), L.ERR_ALIGN),
    # over the logits, but not in their place
    (dict(dz=P + 4), L.ERR_ARG), (dict(dz=P, dstride=104), L.ERR_ARG), (dict(dz=P - 4 * 399), L.ERR_ARG)])
def test_distill_backward_rejects(lib, kw, code):
    assert distill_bwd(lib, **kw) == code


def test_distill_bytes(lib):
    f = lib.sherry_distill_workspace_bytes
    assert f(0, 4, L.F32) == NONE and f(4, 0, L.F32) == NONE and f(4, 4, L.I8) == NONE
    for rows in (1, 100, 5000, 1 << 20):       # a record for each of about 2048 ranges, or one a row
        assert 24 <= f(rows, 128000, L.BF16) <= 24 * (rows + 2048 + 32)
    assert f(1, 1 << 30, L.F32) <= 24 * 4200


def test_distill_binding_rejects():
    z, u, ids = torch.zeros(4, 64), torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        S.distill_loss(z, u, ids)
    with pytest.raises(ValueError, match="CUDA"):
        S.distill_loss_ad(z.requires_grad_(True), u, ids)
    with pytest.raises(ValueError, match="CUDA"):
        S.distill_loss_backward(torch.ones(4), z.detach(), ids, torch.zeros(4, 7))


Y = 1 << 40


def linear(lib, decode, n=64, k=256, gran=L.PER_GROUP, g=128, packed=P, alpha=P, x=P, m=4, y=Y, yd=L.BF16, bias=P,
           bd=L.F32, act=3, gated=0, res=P, rs=0.5, ws=P, wsb=1 << 40):
    if decode:
        return lib.sherry_linear_gemv(n, k, gran, g, packed, alpha, x, m, y, yd, bias, bd, act, gated, res, rs, None)
    return lib.sherry_linear_gemm(n, k, gran, g, packed, alpha, x, m, y, bias, bd, act, gated, res, rs, ws, wsb, None)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(m=0), L.ERR_BATCH), (dict(m=-1), L.ERR_BATCH), (dict(n=0), L.ERR_SHAPE), (dict(k=200), L.ERR_SHAPE),
    (dict(gran=9), L.ERR_SHAPE), (dict(g=100), L.ERR_SHAPE), (dict(g=0), L.ERR_SHAPE), (dict(act=6), L.ERR_ARG),
    (dict(act=-1), L.ERR_ARG), (dict(n=63, gated=1), L.ERR_ARG), (dict(rs=float("inf")), L.ERR_ARG),
    (dict(res=None), L.ERR_ARG), (dict(bd=L.I8), L.ERR_DTYPE), (dict(packed=None), L.ERR_NULL),
    (dict(alpha=None), L.ERR_NULL), (dict(x=None), L.ERR_NULL), (dict(y=None), L.ERR_NULL), (dict(packed=P + 8), L.ERR_ALIGN),
    (dict(x=P + 8), L.ERR_ALIGN), (dict(bias=MIS4), L.ERR_ALIGN), (dict(bias=MIS2, bd=L.BF16), L.ERR_ALIGN),
    (dict(res=MIS2), L.ERR_ALIGN), (dict(y=Y + 1), L.ERR_ALIGN),
    (dict(y=P), L.ERR_ARG), (dict(y=P + 4 * 256 * 2 - 16), L.ERR_ARG),          # over x
    (dict(res=Y + 16), L.ERR_ARG), (dict(res=Y - 64), L.ERR_ARG)])              # over the residual, but not in its place
def test_linear_rejects(lib, decode, kw, code):
    assert linear(lib, decode, **kw) == code


def test_linear_limits(lib):
    assert linear(lib, True, m=17) == L.ERR_BATCH
    assert linear(lib, True, yd=L.I8) == L.ERR_DTYPE
    assert linear(lib, True, yd=L.F32, y=Y, res=Y) == L.ERR_ARG      # two types cannot share a place
    # 40 tokens split K, so need a workspace
    assert linear(lib, False, n=128, k=2048, m=40, ws=None) == L.ERR_WORKSPACE
    assert linear(lib, False, n=128, k=2048, m=40, wsb=64) == L.ERR_WORKSPACE
    assert linear(lib, False, n=128, k=2048, m=40, ws=P + 8) == L.ERR_ALIGN
    assert linear(lib, False, k=1 << 22) == L.ERR_UNSUPPORTED
    assert linear(lib, False, m=128 * 65536 + 1) == L.ERR_BATCH
    assert linear(lib, False, res=P + 4) == L.ERR_ALIGN


def moe(lib, m=4, d=256, f=128, x=P, router=P, rd=L.BF16, e=8, sh=0, k=2, score=0, norm=1, bias=P, scale=1.0, act=3, gated=1,
        up=P, ua=P, ug=L.PER_GROUP, ugs=128, down=P, da=P, dg=L.PER_GROUP, dgs=128, res=P, y=Y, yd=L.BF16, ws=P, wsb=1 << 40):
    return lib.sherry_moe_decode(m, d, f, x, router, rd, e, sh, k, score, norm, bias, scale, act, gated, up, ua, ug, ugs, down,
                                 da, dg, dgs, res, y, yd, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), L.ERR_BATCH), (dict(m=17), L.ERR_BATCH), (dict(d=0), L.ERR_ARG), (dict(d=200), L.ERR_ARG),
    (dict(d=65536 + 128), L.ERR_ARG), (dict(f=64), L.ERR_ARG), (dict(f=-128), L.ERR_ARG), (dict(e=0), L.ERR_ARG),
    (dict(e=513), L.ERR_ARG), (dict(sh=-1), L.ERR_ARG), (dict(sh=5), L.ERR_ARG), (dict(k=0), L.ERR_ARG), (dict(k=9), L.ERR_ARG),
    (dict(e=40, k=17), L.ERR_ARG), (dict(score=2), L.ERR_ARG), (dict(act=6), L.ERR_ARG), (dict(scale=float("nan")), L.ERR_ARG),
    (dict(ug=7), L.ERR_SHAPE), (dict(dgs=384), L.ERR_SHAPE), (dict(rd=L.I8), L.ERR_DTYPE), (dict(yd=L.I8), L.ERR_DTYPE),
    (dict(x=None), L.ERR_NULL), (dict(router=None), L.ERR_NULL), (dict(up=None), L.ERR_NULL), (dict(ua=None), L.ERR_NULL),
    (dict(down=None), L.ERR_NULL), (dict(da=None), L.ERR_NULL), (dict(y=None), L.ERR_NULL), (dict(x=P + 8), L.ERR_ALIGN),
    (dict(router=P + 8), L.ERR_ALIGN), (dict(up=P + 8), L.ERR_ALIGN), (dict(da=P + 8), L.ERR_ALIGN), (dict(bias=MIS4), L.ERR_ALIGN),
    (dict(res=MIS2), L.ERR_ALIGN), (dict(y=Y + 1), L.ERR_ALIGN), (dict(res=Y + 64), L.ERR_ARG), (dict(res=Y, yd=L.F32), L.ERR_ARG),
    (dict(ws=None), L.ERR_WORKSPACE), (dict(wsb=64), L.ERR_WORKSPACE), (dict(ws=P + 8), L.ERR_ALIGN)])
def test_moe_rejects(lib, kw, code):
    assert moe(lib, **kw) == code


def test_moe_bytes(lib):
    f = lib.sherry_moe_workspace_bytes
    assert f(17, 256, 128, 8, 0, 2) == NONE and f(1, 256, 128, 8, 0, 9) == NONE and f(1, 100, 128, 8, 0, 2) == NONE
    for m, e, sh, k, hidden in [(1, 8, 0, 2, 128), (16, 512, 4, 16, 4096), (7, 60, 1, 4, 1536)]:
        least = 4 * m * e + 4 * m * (k + sh) * hidden          # logits, and two bf16 terms of h
        assert least <= f(m, 256, hidden, e, sh, k) <= 2 * least + (1 << 20) + 512 * 4 * m * 64   # and partials of 512 blocks


def test_linear_and_moe_binding_reject():
    pw = S.PackedWeight(torch.zeros(64 * 256 * 5 // 32, dtype=torch.uint8), torch.zeros(128), 64, 256)
    x = torch.zeros(1, 256, dtype=torch.bfloat16)
    for f in (S.linear_gemv, S.linear_gemm):
        with pytest.raises(ValueError, match="CUDA"):
            f(pw, x)
    up = S.PackedExperts(torch.zeros(4, 256 * 256 * 5 // 32, dtype=torch.uint8), torch.zeros(4, 512), 4, 256, 256)
    down = S.PackedExperts(torch.zeros(4, 256 * 128 * 5 // 32, dtype=torch.uint8), torch.zeros(4, 256), 4, 256, 128)
    with pytest.raises(ValueError, match="CUDA"):
        S.moe_decode(x, torch.zeros(4, 256), up, down, 2)
    with pytest.raises(ValueError, match=r"\[E, N, K\]"):
        S.quantize_pack_experts(torch.zeros(4, 256))


def test_gated_products_of_members_that_are_no_pair():
    pw = S.PackedWeight(torch.zeros(96 * 256 * 5 // 32, dtype=torch.uint8), torch.zeros(192), 96, 256)
    x = torch.zeros(1, 256, dtype=torch.bfloat16)
    for f in (S.linear_gemv, S.linear_gemm):
        for sizes in ((64, 32), (96,), (32, 32, 32)):
            with pytest.raises(ValueError, match="two members"):
                f(S.FusedWeight(pw, sizes), x, gated=True)
        with pytest.raises(ValueError, match="CUDA"):
            f(S.FusedWeight(pw, (48, 48)), x, gated=True)
