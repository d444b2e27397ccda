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
