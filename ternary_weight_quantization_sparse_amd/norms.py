"""Norms before and after a block, fused with its gate and the residual scale.

For a row of the residual stream ``h`` and the block's output ``y`` (x^ =
x / sqrt(mean(x^2) + eps)):

    h' = res_scale * h + gate * (w_post * y^),    n = w_pre * h'^

``n`` is what the next block's projections read.
"""

from __future__ import annotations

from . import _lib, _need_gpu, _on_stream, _ptr, _stream, _torch
from ._lib import check, load


_CODES = {}


def _codes():
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: _lib.F32, torch.bfloat16: _lib.BF16})
    return _CODES


def _contiguous(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _like(t, h, name):
    """An operand of h's shape, dtype and device."""
    if t.dtype != h.dtype or t.shape != h.shape or t.device != h.device:
        _need_gpu(t, name, h.device)
        raise ValueError(f"{name} must be {h.dtype} {tuple(h.shape)} like h, got {t.dtype} {tuple(t.shape)}")


def _layout(h, w_pre, y, w_post, gate, res_scale):
    """Checks one call's operands; (rows, D, dtype code, weight dtype code, gate
    kind, rows that share a gate row)."""
    if not h.is_cuda:
        _need_gpu(h, "h")
    codes, dev, dtype, shape = _codes(), h.device, h.dtype, h.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"h must be [..., D], got {tuple(shape)}")
    dim = shape[-1]
    rows = h.numel() // dim
    code = codes.get(dtype)
    if code is None:
        raise ValueError(f"h must be float32 or bfloat16, got {dtype}")
    if y is not None:
        _like(y, h, "y")
    elif w_pre is None:
        raise ValueError("nothing to do: neither a block output y nor a norm w_pre")
    elif w_post is not None or gate is not None or res_scale != 1.0:
        raise ValueError("w_post, gate and res_scale belong to a block output y")
    w_code = None
    for w in (w_post, w_pre):
        if w is None:
            continue
        c = codes.get(w.dtype)
        if c is None or w.shape != (dim,) or w.device != dev or (w_code is not None and w_code != c):
            name = "w_pre" if w is w_pre else "w_post"
            _need_gpu(w, name, dev)
            raise ValueError(f"w_post and w_pre must be [{dim}], both float32 or both bfloat16, got {name} "
                             f"{w.dtype} {tuple(w.shape)}")
        w_code = c
    kind, gate_rows = _lib.GATE_NONE, 1
    if gate is not None:
        if gate.dtype != dtype or gate.device != dev:
            _need_gpu(gate, "gate", dev)
            raise ValueError(f"gate must be {dtype} like h, got {gate.dtype}")
        shape = gate.shape
        if shape == (dim,):
            kind = _lib.GATE_CHANNEL
        elif shape == (rows, 1):
            kind = _lib.GATE_TOKEN
        elif len(shape) == 2 and shape[1] == dim and shape[0] > 0 and rows % shape[0] == 0:
            kind, gate_rows = _lib.GATE_ROWS, max(rows // shape[0], 1)
        else:
            raise ValueError(f"gate must be [{dim}] (a channel), [{rows}, 1] (a token) or [S, {dim}] with S dividing "
                             f"{rows} rows, got {tuple(shape)}")
    return rows, dim, code, w_code or 0, kind, gate_rows


def _forward(layout, h, w_pre, y, w_post, gate, res_scale, eps, stream):
    rows, dim, code, w_code, kind, gate_rows = layout
    empty_like = _torch().empty_like
    h_ = _contiguous(h)
    y, w_pre, w_post, gate = _contiguous(y), _contiguous(w_pre), _contiguous(w_post), _contiguous(gate)
    h_out = h if y is None else empty_like(h_)
    n = None if w_pre is None else empty_like(h_)
    if rows:
        check(load().sherry_block_norm(rows, dim, h_.data_ptr(), _ptr(y), code, _ptr(w_post), _ptr(w_pre), w_code,
                                       _ptr(gate), kind, gate_rows, res_scale, eps,
                                       None if y is None else h_out.data_ptr(), _ptr(n), _stream(stream)))
    return h_out, n


def _backward(layout, dh_out, dn, h, w_pre, y, w_post, gate, res_scale, eps, stream):
    """Gradients of checked operands; dh_out and dn are h's shape and dtype."""
    rows, dim, code, w_code, kind, gate_rows = layout
    torch = _torch()
    empty_like = torch.empty_like
    if w_pre is None:
        dn = None
    dh_out, dn, h, y = _contiguous(dh_out), _contiguous(dn), _contiguous(h), _contiguous(y)
    w_pre, w_post, gate = _contiguous(w_pre), _contiguous(w_post), _contiguous(gate)
    dh = empty_like(h)
    dw_pre = None if w_pre is None else empty_like(w_pre)
    dy = None if y is None else empty_like(y)
    dw_post = None if w_post is None else empty_like(w_post)
    dgate = None if gate is None else empty_like(gate)
    if rows:
        lib = load()
        nbytes = lib.sherry_block_norm_backward_bytes(rows, dim, kind, gate_rows)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=h.device)
        check(lib.sherry_block_norm_backward(
            rows, dim, h.data_ptr(), _ptr(y), _ptr(dh_out), _ptr(dn), code, _ptr(w_post), _ptr(w_pre), w_code,
            _ptr(gate), kind, gate_rows, res_scale, eps, dh.data_ptr(), _ptr(dy), _ptr(dw_post), _ptr(dw_pre),
            _ptr(dgate), ws.data_ptr(), nbytes, _stream(stream)))
    else:
        for t in (dw_pre, dw_post, dgate):
            if t is not None:
                t.zero_()
    return dh, dw_pre, dy, dw_post, dgate


def block_norm(h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6, stream=None):
    """``(h', n)`` for the residual stream ``h`` [..., D] (fp32 or bf16).

    ``y`` the block's output (None: only the norm of h, and h' is h);
    ``w_post`` [D] the norm after the block (None: y as it is); ``gate`` [D],
    [rows, 1] or [S, D] for S equal runs of rows; ``w_pre`` [D] the norm before
    the next block (None: n is None).  Sums and norms are fp32, each output is
    rounded once."""
    layout = _layout(h, w_pre, y, w_post, gate, res_scale)
    if stream is None:
        return _forward(layout, h, w_pre, y, w_post, gate, res_scale, eps, None)
    with _on_stream(stream):
        return _forward(layout, h, w_pre, y, w_post, gate, res_scale, eps, stream)


def block_norm_backward(dh_out, dn, h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0,
                        eps: float = 1e-6, stream=None):
    """Gradients ``(dh, dw_pre, dy, dw_post, dgate)`` of `block_norm` from those
    of its outputs (either may be None: no gradient), None for absent operands.
    h' is recomputed from y and h in fp32, and sums over rows and over a gate's
    broadcast are fp32 in a fixed order."""
    layout = _layout(h, w_pre, y, w_post, gate, res_scale)
    for t, name in ((dh_out, "dh_out"), (dn, "dn")):
        if t is not None:
            _like(t, h, name)
    with _on_stream(stream):
        return _backward(layout, dh_out, dn, h, w_pre, y, w_post, gate, res_scale, eps, stream)


def _make_ad():
    torch = _torch()

    class Gradients(torch.autograd.Function):
        """The gradients in a graph of their own, which cannot be differentiated:
        they depend on h, y, w_post, w_pre and gate, so without it a second
        derivative would be wrong in silence."""

        @staticmethod
        def forward(ctx, *args):
            return _backward(*args)

        @staticmethod
        def backward(ctx, *grads):
            raise RuntimeError("block_norm_ad has first derivatives only")

    class BlockNorm(torch.autograd.Function):
        """`block_norm` with `block_norm_backward` as its gradient."""

        @staticmethod
        def forward(ctx, h, w_pre, y, w_post, gate, res_scale, eps):
            ctx.save_for_backward(h, w_pre, y, w_post, gate)
            ctx.set_materialize_grads(False)
            layout = _layout(h, w_pre, y, w_post, gate, res_scale)
            ctx.args = layout, res_scale, eps
            out, n = _forward(layout, h, w_pre, y, w_post, gate, res_scale, eps, None)
            return (h.view_as(h) if y is None else out), n

        @staticmethod
        def backward(ctx, dh_out, dn):
            if dh_out is None and dn is None:
                return (None,) * 7
            layout, res_scale, eps = ctx.args
            grads = Gradients.apply if torch.is_grad_enabled() else _backward   # create_graph, or not
            dh, dw_pre, dy, dw_post, dgate = grads(layout, dh_out, dn, *ctx.saved_tensors, res_scale, eps, None)
            return dh, dw_pre, dy, dw_post, dgate, None, None

    return BlockNorm


_AD = None


def block_norm_ad(h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6):
    """Differentiable `block_norm` (forward and backward each in the library's kernels)."""
    global _AD
    if _AD is None:
        _AD = _make_ad()
    return _AD.apply(h, w_pre, y, w_post, gate, res_scale, eps)
