"""Orthogonalised updates of latent weights: Newton-Schulz steps on the
momentum, and the weight update they feed."""

from __future__ import annotations

import math

from . import _lib, _need_gpu, _need_out, _on_stream, _ptr, _stream, _torch, _workspace, _written
from ._lib import check, load

#: Quintic coefficients (a, b, c) of X <- a X + (b A + c A A) X, A = X X^T: a
#: steep slope at 0, so that small singular values rise in few steps.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def _matrices(t, name):
    torch = _torch()
    _need_gpu(t, name)
    code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [N, K] or [C, N, K], got {tuple(t.shape)}")
    n, k = (int(s) for s in t.shape[-2:])
    return code, (1 if t.dim() == 2 else int(t.shape[0])), n, k


def _ws(count, n, k, device):
    nbytes = int(load().sherry_muon_workspace_bytes(count, n, k))
    return _workspace(nbytes if nbytes != (1 << 64) - 1 else 0, device)


def _coeffs(coeffs):
    a, b, c = NEWTON_SCHULZ if coeffs is None else coeffs
    return float(a), float(b), float(c)


def orthogonalize(g, steps: int = 5, coeffs=None, eps: float = 1e-7, stream=None, out=None):
    """``steps`` Newton-Schulz steps on a matrix ``g`` [N, K], or on each of
    [C, N, K] at once (fp32 or bf16): every singular value that is not far
    below the largest comes near 1.  Returns g's shape and dtype (``out``, which may be g).
    ``coeffs`` (a, b, c) that can raise a singular value above 2.82 before the
    last step, or |b t + c t^2| (t its square) above 7.98, raise ValueError."""
    torch = _torch()
    code, count, n, k = _matrices(g, "g")
    with _on_stream(stream):
        src = g.contiguous()
        if out is not None:
            _need_out(out, "out", g.dtype, g.numel(), g.device)
        res = out if out is not None else torch.empty_like(src)
        ws = _ws(count, n, k, g.device)
        check(load().sherry_orthogonalize(count, n, k, _ptr(src), code, _ptr(res), int(steps), *_coeffs(coeffs),
                                          float(eps), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    if out is not None:
        _written(out)
    return res


def muon_step(w, grad, buf, lr: float, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
              scale=None, steps: int = 5, coeffs=None, eps: float = 1e-7, stream=None, out=None):
    """One update of latent weights ``w`` [N, K] or [C, N, K] (fp32 or bf16):

        buf' = momentum * buf + grad,   u = grad + momentum * buf'  (buf' without nesterov)
        w' = w * (1 - lr * weight_decay) - lr * scale * orthogonalize(u)

    ``scale`` defaults to sqrt(max(1, N / K)); ``coeffs`` as for `orthogonalize`.  Returns ``(w', buf')``, new
    tensors or ``out``: ``out=(w, buf)`` updates in place."""
    torch = _torch()
    code, count, n, k = _matrices(w, "w")
    for name, t in (("grad", grad), ("buf", buf)):
        _need_gpu(t, name, w.device)
        if t.shape != w.shape or t.dtype != w.dtype:
            raise ValueError(f"{name} must be {w.dtype} {tuple(w.shape)} like w, got {t.dtype} {tuple(t.shape)}")
    if scale is None:
        scale = math.sqrt(max(1.0, n / max(k, 1)))
    with _on_stream(stream):
        if out is not None:
            for name, t in zip(("out[0]", "out[1]"), out):
                _need_out(t, name, w.dtype, w.numel(), w.device)
        ws_, gs, bs = w.contiguous(), grad.contiguous(), buf.contiguous()
        w_out, buf_out = out if out is not None else (torch.empty_like(ws_), torch.empty_like(bs))
        work = _ws(count, n, k, w.device)
        check(load().sherry_muon_step(count, n, k, _ptr(ws_), _ptr(gs), _ptr(bs), code, _ptr(w_out), _ptr(buf_out),
                                      float(lr), float(momentum), int(nesterov), float(weight_decay), float(scale),
                                      int(steps), *_coeffs(coeffs), float(eps), _ptr(work),
                                      0 if work is None else work.numel(), _stream(stream)))
    if out is not None:
        _written(w_out, buf_out)
    return w_out, buf_out
