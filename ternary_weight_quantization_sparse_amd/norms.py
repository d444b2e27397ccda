"""Norms before and after a block, fused with its gate and the residual scale.

For a row of the residual stream ``h`` and the block's output ``y`` (x^ =
x / sqrt(mean(x^2) + eps)):

    h' = res_scale * h + gate * (w_post * y^),    n = w_pre * h'^

``n`` is what the next block's projections read.
"""

from __future__ import annotations

from . import _lib, _need_gpu, _on_stream, _ptr, _stream, _torch, _workspace
from ._lib import check, load


def _dtype_code(t, name):
    torch = _torch()
    code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


class _Norm:
    """Checked operands of one call: contiguous, two-dimensional, on one GPU."""

    def __init__(self, h, w_pre, y, w_post, gate, res_scale, eps):
        _need_gpu(h, "h")
        dev = h.device
        if h.dim() < 1 or h.shape[-1] < 1:
            raise ValueError(f"h must be [..., D], got {tuple(h.shape)}")
        self.shape, self.dim = h.shape, int(h.shape[-1])
        self.rows = h.numel() // self.dim
        self.code = _dtype_code(h, "h")
        if y is None and w_pre is None:
            raise ValueError("nothing to do: neither a block output y nor a norm w_pre")
        if y is None and (w_post is not None or gate is not None or res_scale != 1.0):
            raise ValueError("w_post, gate and res_scale belong to a block output y")
        if y is not None:
            _need_gpu(y, "y", dev)
            if y.shape != h.shape or y.dtype != h.dtype:
                raise ValueError(f"y must be {h.dtype} {tuple(h.shape)} like h, got {y.dtype} {tuple(y.shape)}")
        self.w_code = _lib.F32
        for name, w in (("w_post", w_post), ("w_pre", w_pre)):
            if w is None:
                continue
            _need_gpu(w, name, dev)
            if tuple(w.shape) != (self.dim,):
                raise ValueError(f"{name} must be [{self.dim}], got {tuple(w.shape)}")
            self.w_code = _dtype_code(w, name)
        if w_post is not None and w_pre is not None and w_post.dtype != w_pre.dtype:
            raise ValueError("w_post and w_pre must have one dtype")
        self.kind, self.gate_rows = _lib.GATE_NONE, 1
        if gate is not None:
            _need_gpu(gate, "gate", dev)
            if gate.dtype != h.dtype:
                raise ValueError(f"gate must be {h.dtype} like h, got {gate.dtype}")
            if tuple(gate.shape) == (self.dim,):
                self.kind = _lib.GATE_CHANNEL
            elif gate.dim() == 2 and gate.shape[1] == self.dim and gate.shape[0] > 0 \
                    and self.rows % gate.shape[0] == 0 and (self.dim > 1 or gate.shape[0] != self.rows):
                self.kind, self.gate_rows = _lib.GATE_ROWS, max(self.rows // int(gate.shape[0]), 1)
            elif tuple(gate.shape) == (self.rows, 1):
                self.kind = _lib.GATE_TOKEN
            else:
                raise ValueError(f"gate must be [{self.dim}] (a channel), [{self.rows}, 1] (a token) or [S, {self.dim}] "
                                 f"with S dividing {self.rows} rows, got {tuple(gate.shape)}")
        self.h, self.y, self.w_post, self.w_pre, self.gate = (
            None if t is None else t.contiguous() for t in (h, y, w_post, w_pre, gate))
        self.res_scale, self.eps = float(res_scale), float(eps)

    def like(self, t, name):
        """An incoming gradient of an output: h's shape and dtype."""
        if t is None:
            return None
        _need_gpu(t, name, self.h.device)
        if t.shape != self.shape or t.dtype != self.h.dtype:
            raise ValueError(f"{name} must be {self.h.dtype} {tuple(self.shape)}, got {t.dtype} {tuple(t.shape)}")
        return t.contiguous()


def block_norm(h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6, stream=None):
    """``(h', n)`` for the residual stream ``h`` [..., D] (fp32 or bf16).

    ``y`` the block's output (None: only the norm of h, and h' is h);
    ``w_post`` [D] the norm after the block (None: y as it is); ``gate`` [D],
    [rows, 1] or [S, D] for S equal runs of rows; ``w_pre`` [D] the norm before
    the next block (None: n is None).  Sums and norms are fp32, each output is
    rounded once."""
    torch = _torch()
    with _on_stream(stream):
        a = _Norm(h, w_pre, y, w_post, gate, res_scale, eps)
        h_out = torch.empty_like(a.h) if y is not None else h
        n = torch.empty_like(a.h) if w_pre is not None else None
        if a.rows:
            check(load().sherry_block_norm(
                a.rows, a.dim, _ptr(a.h), _ptr(a.y), a.code, _ptr(a.w_post), _ptr(a.w_pre), a.w_code, _ptr(a.gate),
                a.kind, a.gate_rows, a.res_scale, a.eps, None if y is None else _ptr(h_out), _ptr(n), _stream(stream)))
    return h_out, n


def block_norm_backward(dh_out, dn, h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0,
                        eps: float = 1e-6, stream=None):
    """Gradients ``(dh, dw_pre, dy, dw_post, dgate)`` of `block_norm` from those
    of its outputs (either may be None: zero), None for absent operands.
    h' is recomputed from y and h in fp32, and sums over rows and over a gate's
    broadcast are fp32 in a fixed order."""
    torch = _torch()
    with _on_stream(stream):
        a = _Norm(h, w_pre, y, w_post, gate, res_scale, eps)
        dh_out, dn = a.like(dh_out, "dh_out"), a.like(dn, "dn")
        if a.w_pre is None:
            dn = None
        dh = torch.empty_like(a.h)
        made = [None if t is None else torch.empty_like(t) for t in (a.w_pre, a.y, a.w_post, a.gate)]
        if a.rows:
            lib = load()
            ws = _workspace(int(lib.sherry_block_norm_backward_bytes(a.rows, a.dim, a.kind, a.gate_rows)), h.device)
            dw_pre, dy, dw_post, dgate = made
            check(lib.sherry_block_norm_backward(
                a.rows, a.dim, _ptr(a.h), _ptr(a.y), _ptr(dh_out), _ptr(dn), a.code, _ptr(a.w_post), _ptr(a.w_pre),
                a.w_code, _ptr(a.gate), a.kind, a.gate_rows, a.res_scale, a.eps, _ptr(dh), _ptr(dy), _ptr(dw_post),
                _ptr(dw_pre), _ptr(dgate), _ptr(ws), ws.numel(), _stream(stream)))
        else:
            for t in made:
                if t is not None:
                    t.zero_()
    return (dh, *made)


def _make_ad():
    torch = _torch()

    class BlockNorm(torch.autograd.Function):
        """`block_norm` with `block_norm_backward` as its gradient."""

        @staticmethod
        def forward(ctx, h, w_pre, y, w_post, gate, res_scale, eps):
            ctx.save_for_backward(h, w_pre, y, w_post, gate)
            ctx.args = (res_scale, eps)
            ctx.set_materialize_grads(False)
            out, n = block_norm(h, w_pre, y, w_post, gate, res_scale, eps)
            return (h.view_as(h) if y is None else out), n

        @staticmethod
        def backward(ctx, dh_out, dn):
            h, w_pre, y, w_post, gate = ctx.saved_tensors
            if dh_out is None and dn is None:
                return (None,) * 7
            return (*block_norm_backward(dh_out, dn, h, w_pre, y, w_post, gate, *ctx.args), None, None)

    return BlockNorm


_AD = None


def block_norm_ad(h, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6):
    """Differentiable `block_norm` (forward and backward each in the library's kernels)."""
    global _AD
    if _AD is None:
        _AD = _make_ad()
    return _AD.apply(h, w_pre, y, w_post, gate, res_scale, eps)
