"""The packed product with what follows it: bias, activation and residual.

    y = f(x (T alpha)^T + bias) + res_scale * residual

or, for a gate and its values packed as one weight (what `quantize_pack_fused`
makes of the two, or a `PackedWeight` of their rows [gate; values]):

    y = f(z_gate) * z_values + res_scale * residual
"""

from __future__ import annotations

from . import FusedWeight, _gran, _lib, _need_current, _need_gpu, _on_stream, _stream, _torch, _written, _y_dtype
from ._lib import check, load

_NONE = (1 << 64) - 1
_BF16_OUT = None


def _bf16_out():
    global _BF16_OUT
    _BF16_OUT = _torch().bfloat16, _lib.BF16
    return _BF16_OUT


def _apart(t, count, size):
    """Whether ``count`` parts of ``size`` elements do not stand back to back from the start of ``t``."""
    return t.numel() < count * size or (count > 1 and t.dim() > 1 and t.numel() != count * size and t[0].numel() != size)


def _planes(packed, alpha, n, k, granularity, group_size, count, dev, name=""):
    """Checks the planes and scales of ``count`` packed weights [n, k]; their granularity's code."""
    torch = _torch()
    gran = _lib.GRANULARITY.get(granularity)
    if gran is None:
        gran = _gran(granularity)
    if n < 1 or k < 1 or (gran == _lib.PER_GROUP and group_size < 1):
        raise ValueError(f"{name}packed weight [{n}, {k}], group size {group_size}: not a shape")
    nbytes = n * k // 32 * 5
    scales = n * (k // group_size) if gran == _lib.PER_GROUP else n if gran == _lib.PER_CHANNEL else 1
    if packed.dtype != torch.uint8 or packed.device != dev or not packed.is_contiguous() or _apart(packed, count, nbytes):
        _need_gpu(packed, name + "packed", dev)
        raise ValueError(f"{name}packed must be a contiguous uint8 tensor of {count} x {nbytes} bytes")
    if alpha.dtype != torch.float32 or alpha.device != dev or not alpha.is_contiguous() or _apart(alpha, count, scales):
        _need_gpu(alpha, name + "alpha", dev)
        raise ValueError(f"{name}alpha must be a contiguous float32 tensor of {count} x {scales} scales")
    return gran


def _activation(name):
    try:
        return _lib.ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(_lib.ACTIVATIONS)}, got {name!r}") from None


def _rows(t, name, shape, dev):
    """A bf16 operand or output of this shape."""
    torch = _torch()
    if t.dtype != torch.bfloat16 or t.shape != shape or t.device != dev:
        _need_gpu(t, name, dev)
        raise ValueError(f"{name} must be bfloat16 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _place(out, dtype, shape, dev, like):
    """The caller's output, or a new one (of ``like``'s type if that is it: half the time)."""
    if out is None:
        return like.new_empty(shape) if dtype is like.dtype else _torch().empty(shape, dtype=dtype, device=dev)
    if out.dtype != dtype or out.shape != shape or out.device != dev or not out.is_contiguous():
        _need_gpu(out, "out", dev)
        raise ValueError(f"out must be contiguous {dtype} {tuple(shape)}, got {out.dtype} {tuple(out.shape)}")
    return out


def _linear(pw, x, bias, activation, gated, residual, res_scale, decode, y_dtype, stream, out):
    torch = _torch()
    if isinstance(pw, FusedWeight):
        if gated and (len(pw.sizes) != 2 or pw.sizes[0] != pw.sizes[1]):
            raise ValueError(f"a gated product needs two members of the same rows, a gate and its values, got {pw.sizes}")
        pw = pw.pw
    packed, n, k = pw.packed, pw.n, pw.k
    dev = packed.device
    if not packed.is_cuda:
        _need_gpu(packed, "packed")
    _need_current(dev)
    gran = _planes(packed, pw.alpha, n, k, pw.granularity, pw.group_size, 1, dev)
    act = _activation(activation)
    if gated and n % 2:
        raise ValueError(f"a gated product needs an even number of rows [gate; values], got {n}")
    if decode and x.dim() == 1:
        x = x.unsqueeze(0)
        residual = residual if residual is None or residual.dim() != 1 else residual.unsqueeze(0)
    m, outs = x.shape[0] if x.dim() == 2 else -1, n // 2 if gated else n
    x = _rows(x, "x", (m, k), dev)
    y = _place(out, y_dtype[0], (m, outs), dev, x)
    res = None
    if residual is not None:
        residual = _rows(residual, "residual", (m, outs), dev)
        res = residual.data_ptr()
    elif res_scale != 1.0:
        raise ValueError("res_scale belongs to a residual")
    b, b_code = None, 0
    if bias is not None:
        b_code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}.get(bias.dtype)
        if b_code is None or bias.shape != (n,) or bias.device != dev:
            _need_gpu(bias, "bias", dev)
            raise ValueError(f"bias must be float32 or bfloat16 [{n}], got {bias.dtype} {tuple(bias.shape)}")
        bias = bias if bias.is_contiguous() else bias.contiguous()
        b = bias.data_ptr()
    lib = load()
    head = (n, k, gran, pw.group_size, packed.data_ptr(), pw.alpha.data_ptr(), x.data_ptr(), m, y.data_ptr())
    tail = (b, b_code, act, bool(gated), res, res_scale)
    if decode:
        check(lib.sherry_linear_gemv(*head, y_dtype[1], *tail, _stream(stream)))
    else:
        nbytes = lib.sherry_workspace_bytes(_lib.OP_GEMM, n, k, gran, pw.group_size, m, 1)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if 0 < nbytes < _NONE else None
        check(lib.sherry_linear_gemm(*head, *tail, None if ws is None else ws.data_ptr(), 0 if ws is None else nbytes,
                                     _stream(stream)))
    if out is not None:
        _written(out)
    return y


def _on(stream, *args):
    if stream is None:
        return _linear(*args[:-1], None, args[-1])
    with _on_stream(stream):
        return _linear(*args[:-1], stream, args[-1])


def linear_gemv(pw, x, bias=None, activation: str = "none", gated: bool = False, residual=None, res_scale: float = 1.0,
                y_dtype="bfloat16", stream=None, out=None):
    """The product of a decode batch ``x`` [B, K] bf16 (B = 1..16) with its epilogue, in one launch and with one
    rounding.

    ``pw`` a `PackedWeight`, or a `FusedWeight`, whose members' rows are stacked (gated: the gate and its values).
    ``bias`` [N] fp32 or bf16; ``activation`` none, relu, relu2 (squared), silu, gelu or gelu_tanh; ``gated``: the
    weight's rows are [gate; values] and y is [B, N/2]; ``residual`` bf16 of y's shape.  ``out`` may be ``residual``
    (the residual stream updated in place)."""
    kind = _BF16_OUT if y_dtype == "bfloat16" else _y_dtype(y_dtype)
    return _on(stream, pw, x, bias, activation, gated, residual, res_scale, True, kind or _bf16_out(), out)


def linear_gemm(pw, x, bias=None, activation: str = "none", gated: bool = False, residual=None, res_scale: float = 1.0,
                stream=None, out=None):
    """The same for prefill activations ``x`` [M, K] bf16 -> bf16 [M, N or N/2], on MFMA."""
    return _on(stream, pw, x, bias, activation, gated, residual, res_scale, False, _BF16_OUT or _bf16_out(), out)
