"""Low-rank adapters of many requests beside one packed projection.

A packed ternary weight is not edited after packing; a tuned variant of it is
served as an adapter.  Requests of one batch share the packed weight and bring
their own adapter each.
"""

from __future__ import annotations

from dataclasses import dataclass

from . import (_activations, _check_pw, _gran, _need_gpu, _need_out, _on_stream, _ptr, _stream, _torch,
               _workspace, _y_dtype)
from ._lib import check, load


@dataclass
class AdapterSet:
    """The adapters of one projection [N, K], stacked."""
    a: object               # torch.bfloat16 [C, R, K]
    b: object               # torch.bfloat16 [C, N, R]
    scale: object           # torch.float32 [C]
    rank: object = None     # torch.int32 [C]: ranks in use (None: all R)


def _operand(t, name, dtype, shape, dev):
    if t.dtype != dtype or t.device != dev or t.shape != shape or not t.is_contiguous():
        _need_gpu(t, name, dev)
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _adapted(pw, x, ad, ids, decode, y_dtype, stream, out):
    torch = _torch()
    _check_pw(pw)
    dev, n, k = pw.packed.device, pw.n, pw.k
    if decode and x.dim() == 1:
        x = x.unsqueeze(0)
    ydt, code = _y_dtype(y_dtype)
    gran = _gran(pw.granularity)
    x = _activations(x, k, dev)
    m = x.shape[0]
    if ad.a.dim() != 3:
        raise ValueError(f"adapters' a must be [C, R, {k}], got {tuple(ad.a.shape)}")
    c, r = ad.a.shape[:2]
    if c < 1 or r % 8 != 0 or not 8 <= r <= 256:
        raise ValueError(f"adapters need C >= 1 and a stored rank R of 8..256, a multiple of 8: got C {c}, R {r}")
    bf16, i32 = torch.bfloat16, torch.int32
    tail = (_operand(ad.a, "a", bf16, (c, r, k), dev), _operand(ad.b, "b", bf16, (c, n, r), dev),
            _operand(ad.scale, "scale", torch.float32, (c,), dev),
            None if ad.rank is None else _operand(ad.rank, "rank", i32, (c,), dev),
            _operand(ids, "ids", i32, (m,), dev), c, r)
    if out is not None:
        _need_out(out, "out", ydt, m * n, dev)
    y = out if out is not None else torch.empty((m, n), dtype=ydt, device=dev)
    lib = load()
    nbytes = lib.sherry_adapter_workspace_bytes(n, k, gran, pw.group_size, m, r, int(decode))
    ws = _workspace(nbytes, dev) if nbytes != (1 << 64) - 1 else None
    head = (n, k, gran, pw.group_size, _ptr(pw.packed), _ptr(pw.alpha), _ptr(x), m, y.data_ptr())
    tail += (_ptr(ws), 0 if ws is None else nbytes, _stream(stream))
    check(lib.sherry_adapter_gemv(*head, code, *tail) if decode else lib.sherry_adapter_gemm(*head, *tail))
    return y


def _on(stream, *args):
    """The call on ``stream`` (its temporaries belong to it), or on the current one."""
    if stream is None:
        return _adapted(*args[:6], None, args[6])
    with _on_stream(stream):
        return _adapted(*args[:6], stream, args[6])


def adapter_gemv(pw, x, adapters: AdapterSet, ids, y_dtype="bfloat16", stream=None, out=None):
    """y[m] = x[m] @ (T*alpha)^T + scale_c * B_c (A_c x[m]), c = ids[m], for a
    decode batch ``x`` [M, K] bf16 (M = 1..16).  ``ids`` int32 [M] on the GPU;
    a token whose id is outside [0, C) gets the projection alone."""
    return _on(stream, pw, x, adapters, ids, True, y_dtype, out)


def adapter_gemm(pw, x, adapters: AdapterSet, ids, stream=None, out=None):
    """The same for prefill activations ``x`` [M, K] bf16 -> [M, N] bf16,
    M >= 1, on MFMA.  Tokens of one request stand together in earnest; any
    order of ``ids`` is right."""
    return _on(stream, pw, x, adapters, ids, False, "bfloat16", out)
