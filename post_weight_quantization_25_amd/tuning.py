"""The tuning operators (C ABI in ``include/gptq_tuning.h``): products grouped by expert on
stored layers, the gradient through them, and cross entropy and distillation at a stored
head with their gradients.

Argument checks and marshalling only, as in the package's module.  Work is queued on
``stream`` (default: the current stream of the operands' device, which need not be the
current device); buffers made here are allocated on that stream.

Nothing here is recorded for autograd: results of operands that ask for a gradient carry no
graph.  A program that uses autograd calls ``linear_grouped_backward``, or takes dx from the
losses, in a ``torch.autograd.Function`` of its own.  Gradients in bfloat16 are formed from
weights (and softmax values) in one fp16 part, 2^-11 of each; ``out_dtype`` or ``dx_dtype``
float32 or float16 takes two, 2^-23.
"""
from __future__ import annotations

import torch

from . import _DT, Quantized, _check, _tensor, _workspace, lib
from .serving import _On, _rows, _out, _stored

_HALF = (torch.bfloat16, torch.float16)


def _experts(offsets, device) -> int:
    if offsets is None:
        return 1
    _tensor(offsets, "offsets", torch.int32, None, device)
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must hold n_experts + 1 int32")
    return offsets.numel() - 1


def _activations(x: torch.Tensor, name: str, width: int):
    ld = _rows(x, name)
    if x.dtype not in _HALF or x.shape[1] != width:
        raise ValueError(f"{name} must be bf16/f16 with {width} columns")
    n = x.shape[0]
    return (ld if n > 1 else width), n                # one row's pitch leads nowhere (a view's may be beyond the limit)


def _layers(q: Quantized, offsets, device):
    e, rows = _experts(offsets, device), _stored(q, "q", device)
    if rows % e:
        raise ValueError(f"q has {rows} rows, which {e} experts do not share evenly")
    return e, rows // e


def linear_grouped_workspace_size(n_rows: int, n_experts: int, d_row: int, d_col: int, group_size: int = 128) -> int:
    return lib.gptqt_linear_grouped_workspace_size(n_rows, n_experts, d_row, d_col, group_size)


def linear_grouped(q: Quantized, x: torch.Tensor, offsets: torch.Tensor | None = None, out_dtype=torch.float32,
                   out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = What_e x[t] for the rows t of expert e, offsets[e] <= t < offsets[e + 1]
    (gptqt_linear_grouped).  ``q`` holds the experts' rows one after another (``torch.cat`` of
    their codes, scales and zeros); ``offsets``: n_experts + 1 int32 on the device, or None for
    one expert that takes all rows.  Rows of no expert are left as they were in ``out`` (in a
    buffer made here: undefined).  x (bf16/f16) may be strided."""
    dev = x.device
    e, d_row = _layers(q, offsets, dev)
    ldx, n = _activations(x, "x", q.d_col)
    with _On(dev, stream) as s:
        out = _out(out, n, d_row, out_dtype, dev, x)
        ws = _workspace(linear_grouped_workspace_size(n, e, d_row, q.d_col, q.group_size), dev, ws)
        _check(lib.gptqt_linear_grouped(q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), e, d_row, q.d_col,
                                        q.bits, q.group_size, x.data_ptr(), _DT[x.dtype], n, ldx,
                                        None if offsets is None else offsets.data_ptr(), out.data_ptr(),
                                        _DT[out.dtype], None if ws is None else ws.data_ptr(),
                                        0 if ws is None else ws.numel(), s), "gptqt_linear_grouped")
    return out


def linear_grouped_backward_workspace_size(n_rows: int, n_experts: int, d_row: int, d_col: int, group_size: int = 128) -> int:
    return lib.gptqt_linear_grouped_backward_workspace_size(n_rows, n_experts, d_row, d_col, group_size)


def linear_grouped_backward(q: Quantized, dy: torch.Tensor, offsets: torch.Tensor | None = None, out_dtype=None,
                            out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """dx[t] = What_e^T dy[t]: the gradient through ``linear_grouped``, and with ``offsets`` None
    through ``linear`` or any other product on ``q`` (gptqt_linear_grouped_backward).  dy
    (bf16/f16) may be strided; ``out_dtype``: dy's unless given."""
    dev = dy.device
    e, d_row = _layers(q, offsets, dev)
    ld, n = _activations(dy, "dy", d_row)
    with _On(dev, stream) as s:
        out = _out(out, n, q.d_col, dy.dtype if out_dtype is None else out_dtype, dev, dy)
        ws = _workspace(linear_grouped_backward_workspace_size(n, e, d_row, q.d_col, q.group_size), dev, ws)
        _check(lib.gptqt_linear_grouped_backward(
            q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), e, d_row, q.d_col, q.bits, q.group_size,
            dy.data_ptr(), _DT[dy.dtype], n, ld, None if offsets is None else offsets.data_ptr(), out.data_ptr(),
            _DT[out.dtype], None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s),
            "gptqt_linear_grouped_backward")
    return out


def _apart(outputs, inputs):
    """The outputs that the caller gives overlap no input and not each other: a token's weight, entries
    and activations are read by several workgroups, others of which write."""
    def spans(tensors):
        return [(name, t.data_ptr(), t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.itemsize)
                for name, t in tensors if t is not None and t.numel()]
    mine, theirs = spans(outputs), spans(inputs)
    for i, (name, at, end) in enumerate(mine):
        for other, a, b in mine[i + 1:] + theirs:
            if at < b and a < end:
                raise ValueError(f"{name} overlaps {other}")


def _head(q, x, weights, loss, dx, grad, dx_dtype, entries):
    """Checks what both losses share and makes their outputs; the head's words, x's pitch."""
    dev = x.device
    vocab = _stored(q, "q", dev)
    ldx, n = _activations(x, "x", q.d_col)
    if weights is not None:
        _tensor(weights, "weights", torch.float32, (n,), dev)
    given = [("loss", loss), ("dx", dx)]
    if loss is None:
        loss = torch.empty(n, dtype=torch.float32, device=dev)
    _tensor(loss, "loss", torch.float32, (n,), dev)
    if grad:
        dx = _out(dx, n, q.d_col, x.dtype if dx_dtype is None else dx_dtype, dev, x)
    elif dx is not None:
        raise ValueError("dx without grad")
    if given[0][1] is not None or given[1][1] is not None:
        _apart(given, [("x", x), ("weights", weights)] + entries)
    return vocab, ldx, n, loss, dx


def cross_entropy_workspace_size(n_tokens: int, d: int, vocab: int, group_size: int = 128, grad: bool = True) -> int:
    return lib.gptqt_cross_entropy_workspace_size(n_tokens, d, vocab, group_size, int(bool(grad)))


def cross_entropy(q: Quantized, x: torch.Tensor, targets: torch.Tensor, weights: torch.Tensor | None = None,
                  grad: bool = True, dx_dtype=None, loss: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None):
    """Cross entropy at a stored head and its gradient, in pieces of the vocabulary
    (gptqt_cross_entropy): returns (loss, dx), loss[t] = w_t (logsumexp(What x[t]) - its target's
    logit) in fp32 and dx the gradient of their sum in x's dtype or ``dx_dtype`` (None without
    ``grad``).  A target (int32) outside the vocabulary or a weight of 0 masks its token.  For a
    mean over the tokens give weights of 1 / n.  x (bf16/f16) may be strided."""
    dev = x.device
    _tensor(targets, "targets", torch.int32, x.shape[:1], dev)
    with _On(dev, stream) as s:
        vocab, ldx, n, loss, dx = _head(q, x, weights, loss, dx, grad, dx_dtype, [("targets", targets)])
        ws = _workspace(cross_entropy_workspace_size(n, q.d_col, vocab, q.group_size, grad), dev, ws)
        _check(lib.gptqt_cross_entropy(
            q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), vocab, q.d_col, q.bits, q.group_size,
            x.data_ptr(), _DT[x.dtype], n, ldx, targets.data_ptr(), None if weights is None else weights.data_ptr(),
            loss.data_ptr(), None if dx is None else dx.data_ptr(), 0 if dx is None else _DT[dx.dtype],
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s), "gptqt_cross_entropy")
    return loss, dx


def distill_workspace_size(n_tokens: int, d: int, vocab: int, top_k: int, group_size: int = 128, grad: bool = True) -> int:
    return lib.gptqt_distill_workspace_size(n_tokens, d, vocab, group_size, top_k, int(bool(grad)))


def distill(q: Quantized, x: torch.Tensor, ids: torch.Tensor, top: torch.Tensor, temperature: float = 1.0,
            weights: torch.Tensor | None = None, grad: bool = True, dx_dtype=None, loss: torch.Tensor | None = None,
            dx: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Distillation from a teacher's top logits at a stored head, and its gradient
    (gptqt_distill): ``top`` (n x k, f32/bf16/f16) are the teacher's logits of the words ``ids``
    (int32; outside the vocabulary: no entry).  Returns (loss, dx) as ``cross_entropy`` does,
    loss[t] = w_t T^2 sum_j p_j (log p_j - log q_j) with p the softmax of the entries / T and q
    that of the whole vocabulary's logits / T."""
    dev = x.device
    if ids.dim() != 2 or top.dtype not in _DT:
        raise ValueError("ids must be n_tokens x top_k, top f32/bf16/f16")
    k = ids.shape[1]
    _tensor(ids, "ids", torch.int32, (x.shape[0], k), dev)
    _tensor(top, "top", None, (x.shape[0], k), dev)
    with _On(dev, stream) as s:
        vocab, ldx, n, loss, dx = _head(q, x, weights, loss, dx, grad, dx_dtype, [("ids", ids), ("top", top)])
        ws = _workspace(distill_workspace_size(n, q.d_col, vocab, k, q.group_size, grad), dev, ws)
        _check(lib.gptqt_distill(
            q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), vocab, q.d_col, q.bits, q.group_size,
            x.data_ptr(), _DT[x.dtype], n, ldx, ids.data_ptr(), top.data_ptr(), _DT[top.dtype], k, float(temperature),
            None if weights is None else weights.data_ptr(), loss.data_ptr(), None if dx is None else dx.data_ptr(),
            0 if dx is None else _DT[dx.dtype], None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
            s), "gptqt_distill")
    return loss, dx
