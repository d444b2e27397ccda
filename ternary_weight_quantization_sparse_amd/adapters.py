"""Low-rank adapters of many requests beside one packed projection.

A packed ternary weight is not edited after packing; a tuned variant of it is
served as an adapter.  Requests of one batch share the packed weight and bring
their own adapter each.
"""

from __future__ import annotations

from dataclasses import dataclass

from . import (_activations, _check_pw, _gran, _need_out, _on_stream, _ptr, _stream, _torch,
               _workspace, _y_dtype)
from ._lib import check, load


@dataclass
class AdapterSet:
    """The adapters of one projection [N, K], stacked."""
    a: object               # torch.bfloat16 [C, R, K]
    b: object               # torch.bfloat16 [C, N, R]
    scale: object           # torch.float32 [C]
    rank: object = None     # torch.int32 [C]: ranks in use (None: all R)


def _check_adapters(ad: AdapterSet, pw, ids, tokens):
    torch = _torch()
    dev = pw.packed.device
    if ad.a.dim() != 3 or ad.b.dim() != 3 or ad.a.shape[2] != pw.k or ad.b.shape[1] != pw.n \
            or ad.b.shape[0] != ad.a.shape[0] or ad.b.shape[2] != ad.a.shape[1]:
        raise ValueError(f"adapters of a [{pw.n}, {pw.k}] weight are a [C, R, {pw.k}] and b [C, {pw.n}, R], got "
                         f"{tuple(ad.a.shape)} and {tuple(ad.b.shape)}")
    c, r = int(ad.a.shape[0]), int(ad.a.shape[1])
    if c < 1 or r % 8 != 0 or not 8 <= r <= 256:
        raise ValueError(f"adapters need C >= 1 and a stored rank R of 8..256, a multiple of 8: got C {c}, R {r}")
    _need_out(ad.a, "a", torch.bfloat16, c * r * pw.k, dev)
    _need_out(ad.b, "b", torch.bfloat16, c * r * pw.n, dev)
    _need_out(ad.scale, "scale", torch.float32, c, dev)
    if ad.rank is not None:
        _need_out(ad.rank, "rank", torch.int32, c, dev)
    if ids.dim() != 1 or ids.shape[0] != tokens:
        raise ValueError(f"ids must be [{tokens}], got {tuple(ids.shape)}")
    _need_out(ids, "ids", torch.int32, tokens, dev)
    return c, r


def _adapted(pw, x, ad, ids, decode, y_dtype, stream, out):
    torch = _torch()
    _check_pw(pw)
    dev = pw.packed.device
    if decode and x.dim() == 1:
        x = x.unsqueeze(0)
    ydt, code = _y_dtype(y_dtype)
    gran = _gran(pw.granularity)
    lib = load()
    with _on_stream(stream):
        x = _activations(x, pw.k, dev)
        m = int(x.shape[0])
        c, r = _check_adapters(ad, pw, ids, m)
        if out is not None:
            _need_out(out, "out", ydt, m * pw.n, dev)
        y = out if out is not None else torch.empty((m, pw.n), dtype=ydt, device=dev)
        nbytes = int(lib.sherry_adapter_workspace_bytes(pw.n, pw.k, gran, pw.group_size, m, r, int(decode)))
        ws = _workspace(nbytes if nbytes != (1 << 64) - 1 else 0, dev)
        head = (pw.n, pw.k, gran, pw.group_size, _ptr(pw.packed), _ptr(pw.alpha), _ptr(x), m, _ptr(y))
        tail = (_ptr(ad.a), _ptr(ad.b), _ptr(ad.scale), _ptr(ad.rank), _ptr(ids), c, r, _ptr(ws),
                0 if ws is None else ws.numel(), _stream(stream))
        if decode:
            check(lib.sherry_adapter_gemv(*head, code, *tail))
        else:
            check(lib.sherry_adapter_gemm(*head, *tail))
    return y


def adapter_gemv(pw, x, adapters: AdapterSet, ids, y_dtype="bfloat16", stream=None, out=None):
    """y[m] = x[m] @ (T*alpha)^T + scale_c * B_c (A_c x[m]), c = ids[m], for a
    decode batch ``x`` [M, K] bf16 (M = 1..16).  ``ids`` int32 [M] on the GPU;
    a token whose id is outside [0, C) gets the projection alone."""
    return _adapted(pw, x, adapters, ids, True, y_dtype, stream, out)


def adapter_gemm(pw, x, adapters: AdapterSet, ids, stream=None, out=None):
    """The same for prefill activations ``x`` [M, K] bf16 -> [M, N] bf16,
    M >= 1, on MFMA.  Tokens of one request stand together in earnest; any
    order of ``ids`` is right."""
    return _adapted(pw, x, adapters, ids, False, "bfloat16", stream, out)
