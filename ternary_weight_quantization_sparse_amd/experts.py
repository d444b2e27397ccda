"""A mixture-of-experts layer of packed ternary experts, for the few tokens of
a decode step.

    l = x router^T;   s = softmax(l) or sigmoid(l);   the top_k largest of s (or of s + bias)
    y = sum_j w_j down_j (f(gate_j x) * (up_j x)) + shared experts + residual

Every expert is a packed weight like any other; the layer's are stacked.
"""

from __future__ import annotations

from dataclasses import dataclass

from . import _lib, _need_current, _need_gpu, _on_stream, _stream, _torch, _written, _y_dtype, quantize_pack
from ._lib import check, load
from .linear import _activation, _place, _planes, _rows


@dataclass
class PackedExperts:
    """Packed planes and scales of ``count`` weights [N, K], one after another."""
    packed: object          # torch.uint8 [count, N*K*5/32]
    alpha: object           # torch.float32 [count, num_scales]
    count: int
    n: int
    k: int
    granularity: str = "per_group"
    group_size: int = 128


def quantize_pack_experts(w, granularity: str = "per_group", group_size: int = 128, stream=None) -> PackedExperts:
    """`quantize_pack` of each latent weight of ``w`` [E, N, K] (fp32 or bf16), stacked."""
    torch = _torch()
    if w.dim() != 3 or w.shape[0] < 1:
        raise ValueError(f"experts must be [E, N, K], got {tuple(w.shape)}")
    with _on_stream(stream):
        parts = [quantize_pack(e, granularity, group_size, stream) for e in w]
        packed, alpha = torch.stack([p.packed for p in parts]), torch.stack([p.alpha for p in parts])
    return PackedExperts(packed, alpha, len(parts), parts[0].n, parts[0].k, granularity, group_size)


def moe_decode(x, router, up: PackedExperts, down: PackedExperts, top_k: int, shared: int = 0,
               scoring: str = "softmax", normalize: bool = True, bias=None, scale: float = 1.0,
               activation: str = "silu", residual=None, y_dtype="bfloat16", stream=None, out=None):
    """The whole layer for tokens ``x`` [M, D] bf16, M = 1..16.

    ``router`` [E, D] fp32 or bf16.  ``up`` holds E + shared weights [2H, D], rows [gate; up] (or [H, D]: no gate,
    h = f(up x)), ``down`` as many [D, H]; the ``shared`` last ones serve every token with the weight 1.
    ``scoring`` softmax or sigmoid; ``normalize``: a token's weights are divided by their sum; ``scale`` multiplies
    them.  ``bias`` fp32 [E] is added to the scores for the choice alone; an expert of bias -inf is off.  Among
    equals the lower index is chosen.  ``residual`` bf16 [M, D]; ``out`` may be ``residual`` or ``x``.
    No token's values reach another's result; the order of its fp32 sums follows the experts that the batch uses."""
    if stream is None:
        return _moe(x, router, up, down, top_k, shared, scoring, normalize, bias, scale, activation, residual, y_dtype,
                    None, out)
    with _on_stream(stream):
        return _moe(x, router, up, down, top_k, shared, scoring, normalize, bias, scale, activation, residual, y_dtype,
                    stream, out)


def _moe(x, router, up, down, top_k, shared, scoring, normalize, bias, scale, activation, residual, y_dtype, stream,
         out):
    torch = _torch()
    dev, dim, hidden, total = x.device, down.n, down.k, up.count
    if not x.is_cuda:
        _need_gpu(x, "x")
    _need_current(dev)
    if x.dim() != 2:
        raise ValueError(f"x must be [M, {dim}], got {tuple(x.shape)}")
    m = x.shape[0]
    x = _rows(x, "x", (m, dim), dev)
    if up.k != dim or up.n not in (hidden, 2 * hidden) or down.count != total:
        raise ValueError(f"experts must be up [2H or H, D] and down [D, H], as many of each: got {total} x "
                         f"[{up.n}, {up.k}] and {down.count} x [{dim}, {hidden}]")
    up_gran = _planes(up.packed, up.alpha, up.n, up.k, up.granularity, up.group_size, total, dev, "up: ")
    down_gran = _planes(down.packed, down.alpha, dim, hidden, down.granularity, down.group_size, total, dev, "down: ")
    experts = total - shared
    r_code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}.get(router.dtype)
    if r_code is None or router.shape != (experts, dim) or router.device != dev:
        _need_gpu(router, "router", dev)
        raise ValueError(f"router must be float32 or bfloat16 [{experts}, {dim}], got {router.dtype} "
                         f"{tuple(router.shape)}")
    router = router if router.is_contiguous() else router.contiguous()
    if scoring not in _lib.SCORING:
        raise ValueError(f"scoring must be softmax or sigmoid, got {scoring!r}")
    if bias is not None:
        if bias.dtype != torch.float32 or bias.shape != (experts,) or bias.device != dev:
            _need_gpu(bias, "bias", dev)
            raise ValueError(f"bias must be float32 [{experts}], got {bias.dtype} {tuple(bias.shape)}")
        bias = bias if bias.is_contiguous() else bias.contiguous()
    if residual is not None:
        residual = _rows(residual, "residual", (m, dim), dev)
    ydt, y_code = (x.dtype, _lib.BF16) if y_dtype == "bfloat16" else _y_dtype(y_dtype)
    y = _place(out, ydt, (m, dim), dev, x)
    lib = load()
    nbytes = lib.sherry_moe_workspace_bytes(m, dim, hidden, experts, shared, top_k)
    ws = x.new_empty(nbytes if nbytes != (1 << 64) - 1 else 0, dtype=torch.uint8)
    check(lib.sherry_moe_decode(
        m, dim, hidden, x.data_ptr(), router.data_ptr(), r_code, experts, shared, top_k, _lib.SCORING[scoring],
        bool(normalize), None if bias is None else bias.data_ptr(), scale, _activation(activation), up.n != hidden,
        up.packed.data_ptr(), up.alpha.data_ptr(), up_gran, up.group_size, down.packed.data_ptr(),
        down.alpha.data_ptr(), down_gran, down.group_size, None if residual is None else residual.data_ptr(),
        y.data_ptr(), y_code, ws.data_ptr(), nbytes, _stream(stream)))
    if out is not None:
        _written(out)
    return y
