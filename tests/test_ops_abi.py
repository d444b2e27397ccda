"""The operators around the packed layer (include/sherry_ops.h) without a GPU:
exported symbols, workspace sizes, and every refusal before any launch.  Each
rejected call has one invalid argument and addresses that are never read."""

import os
import re

import pytest

from conftest import ROOT

S = pytest.importorskip("ternary_weight_quantization_sparse_amd")
torch = pytest.importorskip("torch")
L = S._lib

P, MIS2, MIS4 = 0x10000, 0x10001, 0x10002
NONE = (1 << 64) - 1


@pytest.fixture(scope="module")
def lib():
    return L.load()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "sherry_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    assert set(re.findall(r"\b(sherry_[a-z_]+)\s*\(", src)) == set(L.OPS_SYMBOLS)
    assert all(hasattr(lib, name) for name in L.OPS_SYMBOLS)
    assert lib.sherry_status_string(L.ERR_ARG).decode().startswith("SHERRY_ERR_ARG")


def norm(lib, rows=4, dim=64, h=P, y=P, dt=L.F32, wpost=P, wpre=P, wdt=L.F32, gate=P, kind=L.GATE_CHANNEL, per=1,
         scale=0.5, eps=1e-6, ho=P, no=P):
    return lib.sherry_block_norm(rows, dim, h, y, dt, wpost, wpre, wdt, gate, kind, per, scale, eps, ho, no, None)


NORM_BAD = [
    (dict(rows=0), L.ERR_ARG), (dict(rows=1 << 31), L.ERR_ARG), (dict(dim=0), L.ERR_ARG),
    (dict(dim=(1 << 24) + 1), L.ERR_ARG), (dict(kind=4), L.ERR_ARG), (dict(kind=-1), L.ERR_ARG),
    (dict(kind=L.GATE_ROWS, per=3), L.ERR_ARG), (dict(kind=L.GATE_ROWS, per=0), L.ERR_ARG),
    (dict(dt=L.I8), L.ERR_DTYPE), (dict(wdt=L.I8), L.ERR_DTYPE), (dict(h=None), L.ERR_NULL),
    (dict(gate=None), L.ERR_NULL), (dict(y=None, wpost=None, gate=None, kind=L.GATE_NONE), L.ERR_ARG),
    (dict(y=None, scale=1.0, gate=None, kind=L.GATE_NONE), L.ERR_ARG),
    (dict(y=None, wpost=None, wpre=None, gate=None, kind=L.GATE_NONE, scale=1.0), L.ERR_NULL),
    (dict(eps=-1.0), L.ERR_ARG), (dict(eps=float("nan")), L.ERR_ARG), (dict(scale=float("inf")), L.ERR_ARG),
    (dict(h=MIS4), L.ERR_ALIGN), (dict(y=MIS2, dt=L.BF16), L.ERR_ALIGN), (dict(wpost=MIS4), L.ERR_ALIGN),
]


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(ho=None), L.ERR_NULL), (dict(no=None), L.ERR_NULL), (dict(no=MIS4), L.ERR_ALIGN)])
def test_block_norm_rejects(lib, kw, code):
    assert norm(lib, **kw) == code


def norm_bwd(lib, rows=4, dim=64, h=P, y=P, dho=P, dno=P, dt=L.F32, wpost=P, wpre=P, wdt=L.F32, gate=P,
             kind=L.GATE_CHANNEL, per=1, scale=0.5, eps=1e-6, dh=P, dy=P, dwpost=P, dwpre=P, dgate=P, ws=P,
             wsb=1 << 30):
    return lib.sherry_block_norm_backward(rows, dim, h, y, dho, dno, dt, wpost, wpre, wdt, gate, kind, per, scale, eps,
                                          dh, dy, dwpost, dwpre, dgate, ws, wsb, None)


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(dh=None), L.ERR_NULL), (dict(dy=None), L.ERR_NULL), (dict(dwpost=None), L.ERR_NULL),
    (dict(dwpre=None), L.ERR_NULL), (dict(dgate=None), L.ERR_NULL), (dict(dho=MIS4), L.ERR_ALIGN),
    (dict(dgate=MIS4), L.ERR_ALIGN), (dict(ws=None), L.ERR_WORKSPACE), (dict(wsb=64), L.ERR_WORKSPACE),
    (dict(ws=P + 8), L.ERR_ALIGN)])
def test_block_norm_backward_rejects(lib, kw, code):
    assert norm_bwd(lib, **kw) == code


def test_block_norm_backward_bytes(lib):
    f = lib.sherry_block_norm_backward_bytes
    assert f(0, 64, 0, 1) == NONE and f(4, 64, L.GATE_ROWS, 3) == NONE
    # column sums of at most ~512 workgroups of each reduced operand, and 3 floats a row
    assert f(8192, 2048, L.GATE_ROWS, 1024) <= 3 * 520 * 2048 * 4 + 8192 * 12
    assert f(1, 2048, L.GATE_NONE, 1) >= 2 * 2048 * 4


def ad(lib, decode, n=64, k=256, gran=L.PER_GROUP, g=128, packed=P, alpha=P, x=P, m=4, y=P, yd=L.BF16, a=P, b=P,
       scale=P, ranks=P, ids=P, count=2, rank=16, ws=P, wsb=1 << 40):
    if decode:
        return lib.sherry_adapter_gemv(n, k, gran, g, packed, alpha, x, m, y, yd, a, b, scale, ranks, ids, count, rank,
                                       ws, wsb, None)
    return lib.sherry_adapter_gemm(n, k, gran, g, packed, alpha, x, m, y, a, b, scale, ranks, ids, count, rank, ws, wsb,
                                   None)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(m=0), L.ERR_BATCH), (dict(rank=0), L.ERR_ARG), (dict(rank=12), L.ERR_ARG), (dict(rank=264), L.ERR_ARG),
    (dict(count=0), L.ERR_ARG), (dict(n=0), L.ERR_SHAPE), (dict(k=200), L.ERR_SHAPE), (dict(gran=9), L.ERR_SHAPE),
    (dict(a=None), L.ERR_NULL), (dict(b=None), L.ERR_NULL), (dict(scale=None), L.ERR_NULL), (dict(ids=None), L.ERR_NULL),
    (dict(packed=None), L.ERR_NULL), (dict(x=None), L.ERR_NULL), (dict(y=None), L.ERR_NULL),
    (dict(a=P + 8), L.ERR_ALIGN), (dict(b=P + 8), L.ERR_ALIGN), (dict(ids=MIS4), L.ERR_ALIGN),
    (dict(ranks=MIS4), L.ERR_ALIGN), (dict(x=P + 8), L.ERR_ALIGN),
    (dict(ws=None), L.ERR_WORKSPACE), (dict(wsb=16), L.ERR_WORKSPACE), (dict(ws=P + 8), L.ERR_ALIGN)])
def test_adapter_rejects(lib, decode, kw, code):
    assert ad(lib, decode, **kw) == code


def test_adapter_decode_limits(lib):
    assert ad(lib, True, m=17) == L.ERR_BATCH
    assert ad(lib, True, yd=L.I8) == L.ERR_DTYPE
    assert lib.sherry_adapter_workspace_bytes(64, 256, L.PER_GROUP, 128, 17, 16, 1) == NONE
    assert lib.sherry_adapter_workspace_bytes(64, 256, L.PER_GROUP, 128, 17, 16, 0) < 1 << 30
    assert lib.sherry_adapter_workspace_bytes(64, 256, L.PER_GROUP, 128, 17, 15, 0) == NONE


def muon(lib, count=1, n=64, k=64, w=P, g=P, buf=P, dt=L.F32, wo=P, bo=P, lr=0.1, mom=0.9, nes=1, wd=0.0, scale=1.0,
         steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, ws=P, wsb=1 << 40):
    return lib.sherry_muon_step(count, n, k, w, g, buf, dt, wo, bo, lr, mom, nes, wd, scale, steps, a, b, c, eps, ws,
                                wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), L.ERR_ARG), (dict(n=0), L.ERR_ARG), (dict(k=16385), L.ERR_ARG), (dict(steps=0), L.ERR_ARG),
    (dict(steps=17), L.ERR_ARG), (dict(dt=L.I8), L.ERR_DTYPE), (dict(w=None), L.ERR_NULL), (dict(g=None), L.ERR_NULL),
    (dict(buf=None), L.ERR_NULL), (dict(wo=None), L.ERR_NULL), (dict(bo=None), L.ERR_NULL),
    (dict(lr=float("nan")), L.ERR_ARG), (dict(eps=-1.0), L.ERR_ARG), (dict(a=float("inf")), L.ERR_ARG),
    (dict(w=MIS4), L.ERR_ALIGN), (dict(ws=None), L.ERR_WORKSPACE), (dict(wsb=16), L.ERR_WORKSPACE),
    (dict(ws=P + 8), L.ERR_ALIGN)])
def test_muon_rejects(lib, kw, code):
    assert muon(lib, **kw) == code


def test_orthogonalize_rejects(lib):
    def call(count=1, n=64, k=64, g=P, dt=L.F32, out=P, ws=P, wsb=1 << 40, steps=5):
        return lib.sherry_orthogonalize(count, n, k, g, dt, out, steps, 3.0, -4.0, 2.0, 1e-7, ws, wsb, None)
    assert call(n=-1) == L.ERR_ARG and call(count=70000) == L.ERR_ARG and call(steps=0) == L.ERR_ARG
    assert call(g=None) == L.ERR_NULL and call(out=None) == L.ERR_NULL and call(dt=5) == L.ERR_DTYPE
    assert call(ws=None) == L.ERR_WORKSPACE
    assert lib.sherry_muon_workspace_bytes(1, 0, 4) == NONE
    assert lib.sherry_muon_workspace_bytes(2, 512, 2048) > 2 * 5 * 512 * 2048 * 4 // 2


def test_binding_rejects_host_tensors():
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        S.block_norm(t, torch.ones(64))
    with pytest.raises(ValueError):
        S.orthogonalize(t)
    with pytest.raises(ValueError):
        S.muon_step(t, t, t, 0.1)
    pw = S.PackedWeight(torch.zeros(64 * 256 * 5 // 32, dtype=torch.uint8), torch.zeros(128), 64, 256)
    ads = S.AdapterSet(torch.zeros(1, 8, 256), torch.zeros(1, 64, 8), torch.zeros(1))
    with pytest.raises(ValueError):
        S.adapter_gemv(pw, torch.zeros(1, 256), ads, torch.zeros(1, dtype=torch.int32))


REFUSED = [((3.3, -0.4, 0.0), 2), ((2.83, 0.0, 0.0), 2), ((8.3, -23.6, 17.3), 1), ((8.3, -23.6, 17.3), 5),
           ((1.0, 9.0, 0.0), 1), ((3.0, -4.0, 2.0), 5), ((1e30, -1e30, 1e30), 2)]


@pytest.mark.parametrize("coeffs,steps", REFUSED)
def test_muon_refuses_coefficients_that_leave_its_range(lib, coeffs, steps):
    """A singular value that reaches 2.82 before the last step, or |b t + c t^2| that reaches 8."""
    a, b, c = coeffs
    assert muon(lib, a=a, b=b, c=c, steps=steps) == L.ERR_ARG
    assert lib.sherry_orthogonalize(1, 64, 64, P, L.BF16, P, steps, a, b, c, 1e-7, P, 1 << 40, None) == L.ERR_ARG


@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (96, 100), (128, 128), (300, 300), (16, 2048), (600, 600), (1, 16384)])
def test_muon_workspace_follows_the_count(lib, n, k):
    """Bytes grow with the matrices at most by the padding of the tiles that their own sides admit (1.4 times the
    products of 64-tiles), without a jump, and not past what 2^26 elements of a time need."""
    f = lib.sherry_muon_workspace_bytes
    counts = sorted({min(65535, max(1, int(2 ** (i / 4)))) for i in range(65)} | {7811, 7812, 7813, 62499, 62500, 65535})
    up = lambda x, t: -(-x // t) * t  # noqa: E731
    r, l = min(n, k), max(n, k)
    one = 4 * n * k + 3 * 4 * up(r, 64) * up(l, 64) * 1.4 + 5 * 4 * up(r, 64) ** 2 * 1.4   # u; X and its copies; A and the like
    for c in counts:
        assert f(c, n, k) <= c * one * 1.01 + (32 << 20), (c, f(c, n, k))   # and partials of split K, sums
        assert f(c, n, k) < 4 << 30, (c, f(c, n, k))


def test_muon_refuses_overlapping_outputs(lib):
    a, b, c, d = (0x10000000 * i for i in range(1, 5))
    size = 64 * 64 * 4
    good = dict(a=1.5, b=-0.5, c=0.0, ws=None)           # in order but for the workspace
    assert muon(lib, w=a, g=b, buf=c, wo=a, bo=c, **good) == L.ERR_WORKSPACE
    good["ws"] = P
    for kw in (dict(wo=a, bo=a), dict(wo=d, bo=a), dict(wo=d, bo=d), dict(wo=a + 16, bo=c), dict(wo=a - size + 4, bo=c),
               dict(wo=a, bo=c + 16), dict(wo=b + 8, bo=c), dict(wo=d, bo=d + 64)):
        assert muon(lib, w=a, g=b, buf=c, **kw, **good) == L.ERR_ARG, kw
    for out in (a + 4, a - 4, a + size - 4):
        assert lib.sherry_orthogonalize(1, 64, 64, a, L.F32, out, 5, 1.5, -0.5, 0.0, 1e-7, P, 1 << 40, None) == L.ERR_ARG
