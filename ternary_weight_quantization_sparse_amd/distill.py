"""Distillation of a student from a teacher's top logits.

Ternary weights are learned from a teacher of full precision; what is kept of
it for each token are its largest logits.  For a row of student logits s, the
teacher's logits u_j of ids i_j and a temperature t (q = softmax(s / t)):

    kd = t^2 (sum_j p_j log(p_j / q_ij) + rest log(rest / q_rest))
    loss = kd_weight * kd + (1 - kd_weight) * (-log softmax(s)_label)

p is the softmax of u / t over the slots and rest is 0; or, with the teacher's
own normaliser, p_j = exp(u_j / t - teacher_lse) and rest what they leave of 1,
held against the student's mass outside the ids.
"""

from __future__ import annotations

from . import _lib, _need_current, _need_gpu, _on_stream, _ptr, _stream, _torch, _written
from ._lib import check, load


_HEAD = 6     # floats of a row's statistics before its slots


def _floats(t, name, shape, dev):
    torch = _torch()
    _need_gpu(t, name, dev)
    code = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}.get(t.dtype)
    if code is None or t.shape != shape:
        raise ValueError(f"{name} must be float32 or bfloat16 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return code


def _indexes(t, name, shape, dev):
    torch = _torch()
    _need_gpu(t, name, dev)
    if t.dtype not in (torch.int32, torch.int64) or t.shape != shape:
        raise ValueError(f"{name} must be int32 or int64 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return int(t.dtype == torch.int64)


def _rows(t, vocab):
    """[..., V] as rows of V consecutive elements: (tensor, rows, elements from one row to the next)."""
    if t.is_contiguous():
        return t, t.numel() // vocab, vocab
    flat = t.reshape(-1, vocab) if t.dim() != 2 else t
    rows, stride = flat.shape[0], flat.stride(0)
    if vocab > 1 and flat.stride(1) != 1 or rows > 1 and stride < vocab:   # (broadcast rows too)
        return flat.contiguous(), rows, vocab
    return flat, rows, (stride if rows > 1 else vocab)


def _layout(logits, ids, labels):
    """(vocab, leading shape, slots, dtype code, int64 ids, int64 labels) of checked operands."""
    dev, shape = logits.device, logits.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"logits must be [..., V], got {tuple(shape)}")
    code = _floats(logits, "logits", shape, dev)
    _need_current(dev)
    lead = shape[:-1]
    if ids.dim() != len(shape) or ids.shape[-1] < 1:
        raise ValueError(f"ids must be {[*lead]} + [slots], got {tuple(ids.shape)}")
    slots = ids.shape[-1]
    ids_64 = _indexes(ids, "ids", (*lead, slots), dev)
    return shape[-1], lead, slots, code, ids_64, 0 if labels is None else _indexes(labels, "labels", lead, dev)


def _contiguous(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _forward(layout, logits, teacher, ids, temperature, teacher_lse, labels, kd_weight, want_stats, stream):
    vocab, lead, slots, code, ids_64, labels_64 = layout
    torch = _torch()
    dev = logits.device
    t_code = _floats(teacher, "teacher", ids.shape, dev)
    if teacher_lse is not None and (teacher_lse.dtype != torch.float32 or teacher_lse.shape != lead
                                    or teacher_lse.device != dev):
        _need_gpu(teacher_lse, "teacher_lse", dev)
        raise ValueError(f"teacher_lse must be float32 {tuple(lead)}, got {teacher_lse.dtype} {tuple(teacher_lse.shape)}")
    flat, rows, stride = _rows(logits, vocab)
    teacher, ids, teacher_lse, labels = _contiguous(teacher), _contiguous(ids), _contiguous(teacher_lse), _contiguous(labels)
    loss = torch.empty(lead, dtype=torch.float32, device=dev)
    stats = torch.empty((rows, _HEAD + slots), dtype=torch.float32, device=dev) if want_stats else None
    if rows:
        lib = load()
        nbytes = lib.sherry_distill_workspace_bytes(rows, vocab, code)
        ws = torch.empty(nbytes if nbytes != (1 << 64) - 1 else 0, dtype=torch.uint8, device=dev)
        check(lib.sherry_distill_loss(rows, vocab, flat.data_ptr(), stride, code, teacher.data_ptr(), t_code,
                                      ids.data_ptr(), ids_64, slots, temperature, _ptr(teacher_lse), _ptr(labels),
                                      labels_64, kd_weight, loss.data_ptr(), _ptr(stats), ws.data_ptr(), nbytes,
                                      _stream(stream)))
    return loss, stats


def _backward(layout, g, logits, ids, stats, temperature, labels, kd_weight, out, stream):
    """The gradient of checked operands."""
    vocab, _, slots, code, ids_64, labels_64 = layout
    flat, rows, stride = _rows(logits, vocab)
    if out is None:
        out, out_stride = logits.new_empty(logits.shape), vocab
    else:
        place, _, out_stride = _rows(out, vocab)
        if place.data_ptr() != out.data_ptr():
            raise ValueError("out must have rows of consecutive elements at one distance")
    g, ids, labels = _contiguous(g), _contiguous(ids), _contiguous(labels)
    if rows:
        check(load().sherry_distill_loss_backward(
            rows, vocab, g.data_ptr(), flat.data_ptr(), stride, code, ids.data_ptr(), ids_64, slots, temperature,
            _ptr(labels), labels_64, kd_weight, stats.data_ptr(), out.data_ptr(), out_stride, _stream(stream)))
    return out


def distill_loss(logits, teacher, ids, temperature: float = 1.0, teacher_lse=None, labels=None, kd_weight: float = 1.0,
                 with_stats: bool = False, stream=None):
    """The loss of each row, float32 [...], for student ``logits`` [..., V] (fp32 or bf16; rows may stand apart, as in a
    padded vocabulary), the teacher's top logits ``teacher`` [..., J] of ``ids`` [..., J] (int32 or int64; an id outside
    [0, V) is an empty slot).

    ``teacher_lse`` float32 [...]: the logarithm of the sum of exp(u / temperature) over the teacher's whole vocabulary
    (None: p is normalised over the slots).  ``labels`` [...] (int32 or int64; outside [0, V): none) with the weight
    1 - kd_weight.  A row without slots and label has the loss 0.  J is at most 1024.
    ``with_stats``: (loss, what `distill_loss_backward` needs)."""
    if stream is None:
        out = _forward(_layout(logits, ids, labels), logits, teacher, ids, temperature, teacher_lse, labels, kd_weight,
                       with_stats, None)
    else:
        with _on_stream(stream):
            out = _forward(_layout(logits, ids, labels), logits, teacher, ids, temperature, teacher_lse, labels,
                           kd_weight, with_stats, stream)
    return out if with_stats else out[0]


def distill_loss_backward(g, logits, ids, stats, temperature: float = 1.0, labels=None, kd_weight: float = 1.0,
                          stream=None, out=None):
    """The gradient of the logits, their shape and dtype, from that of the losses ``g`` float32 [...] and the ``stats``
    of the forward pass with the same arguments.  ``out`` may be ``logits``.  A row whose g is 0 gets zeros, whatever
    it holds."""
    with _on_stream(stream):
        layout = _layout(logits, ids, labels)
        torch, dev, lead, slots = _torch(), logits.device, layout[1], layout[2]
        if g.dtype != torch.float32 or g.shape != lead or g.device != dev:
            _need_gpu(g, "g", dev)
            raise ValueError(f"g must be float32 {tuple(lead)}, got {g.dtype} {tuple(g.shape)}")
        rows = logits.numel() // layout[0]
        if stats.dtype != torch.float32 or stats.shape != (rows, _HEAD + slots) or not stats.is_contiguous() \
                or stats.device != dev:
            _need_gpu(stats, "stats", dev)
            raise ValueError(f"stats must be those of the forward pass, float32 {(rows, _HEAD + slots)}")
        if out is not None and (out.dtype != logits.dtype or out.shape != logits.shape or out.device != dev):
            _need_gpu(out, "out", dev)
            raise ValueError(f"out must be {logits.dtype} {tuple(logits.shape)}, got {out.dtype} {tuple(out.shape)}")
        grad = _backward(layout, g, logits, ids, stats, temperature, labels, kd_weight, out, stream)
        if out is not None:
            _written(out)
        return grad


def _make_ad():
    torch = _torch()

    class Gradient(torch.autograd.Function):
        """The gradient in a graph of its own, which cannot be differentiated: it
        depends on the logits, so without it a second derivative would be wrong in silence."""

        @staticmethod
        def forward(ctx, *args):
            return _backward(*args)

        @staticmethod
        def backward(ctx, *grads):
            raise RuntimeError("distill_loss_ad has first derivatives only")

    class DistillLoss(torch.autograd.Function):
        """`distill_loss` with `distill_loss_backward` as the gradient of the logits."""

        @staticmethod
        def forward(ctx, logits, teacher, ids, temperature, teacher_lse, labels, kd_weight):
            layout = _layout(logits, ids, labels)
            loss, stats = _forward(layout, logits, teacher, ids, temperature, teacher_lse, labels, kd_weight, True, None)
            ctx.save_for_backward(logits, ids, stats, labels)
            ctx.args = layout, temperature, kd_weight
            return loss

        @staticmethod
        def backward(ctx, g):
            logits, ids, stats, labels = ctx.saved_tensors
            layout, temperature, kd_weight = ctx.args
            _need_current(logits.device)
            grad = Gradient.apply if torch.is_grad_enabled() else _backward   # create_graph, or not
            return grad(layout, g, logits, ids, stats, temperature, labels, kd_weight, None, None), None, None, None, \
                None, None, None

    return DistillLoss


_AD = None


def distill_loss_ad(logits, teacher, ids, temperature: float = 1.0, teacher_lse=None, labels=None,
                    kd_weight: float = 1.0):
    """Differentiable `distill_loss` (forward and backward each in the library's kernels).  The teacher's operands are
    constants: ones that require a gradient are refused."""
    global _AD
    if any(t is not None and t.requires_grad for t in (teacher, teacher_lse)):
        raise ValueError("the teacher is a constant: detach teacher and teacher_lse")
    if _AD is None:
        _AD = _make_ad()
    return _AD.apply(logits, teacher, ids, temperature, teacher_lse, labels, kd_weight)
