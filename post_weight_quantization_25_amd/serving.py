"""The serving operators (C ABI in ``include/gptq_serving.h``): the norm that writes 8-bit
rows, the product on stored codes with 8-bit rows, the product with low-rank adapters
beside it, and a mixture-of-experts layer on stored codes.

Argument checks and marshalling only, as in the package's module.  Work is queued on
``stream`` (default: the current stream of the operands' device, which need not be the
current device); buffers made here are allocated on that stream.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _DT, Quantized, _check, _check_quantized, _dev, _n_groups, _tensor, _workspace, code_bytes, lib


_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream   # current_stream(i).cuda_stream without the object


class _On:
    """The operands' device made current and ``stream`` made the current stream, where they
    are not already; gives the stream's handle."""
    __slots__ = ("index", "inner")

    def __init__(self, device, stream):
        self.index, self.inner = device.index, ()
        if stream is not None or self.index != _current_device():
            self.inner = (torch.cuda.device(device),)
            if stream is not None:
                if stream.device != device:
                    raise ValueError(f"stream is on {stream.device}, the operands on {device}")
                self.inner += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self.inner:
            c.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        for c in reversed(self.inner):
            c.__exit__(*exc)


def _rows(t: torch.Tensor, name: str, dtype=None, shape=None, device=None) -> int:
    """A 2-D device tensor of rows with unit column stride; its row pitch in elements."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D device tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    n, d = t.shape
    if n == 0 or d == 0:
        return d
    s0, s1 = t.stride()
    if (s1 != 1 and d > 1) or (s0 < d and n > 1):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return max(s0, d)


@dataclass
class Int8Rows:
    """Rows of 8-bit codes with one scale each: row t stands for q[t] * scale[t]."""
    q: torch.Tensor          # int8, n_tokens x d (rows may be strided)
    scale: torch.Tensor      # float32, n_tokens


def _shared(o, ldo: int, name: str, x, ldx: int, r, ldr: int):
    """An output that is an input's buffer must have its row pitch."""
    if o.shape[0] < 2:
        return
    at = o.data_ptr()
    if (at == x.data_ptr() and ldo != ldx) or (r is not None and at == r.data_ptr() and ldo != ldr):
        raise ValueError(f"{name} shares a buffer with an input of another row pitch")


def rmsnorm_int8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 residual_out: torch.Tensor | None = None, normed: torch.Tensor | None = None,
                 out: Int8Rows | None = None, stream=None):
    """h = x + residual; RMS norm of h times ``weight``, as 8-bit rows (gptqs_rmsnorm_int8).
    Returns (Int8Rows, h); h is x itself without a residual, else ``residual_out`` (made
    here when not given; it may be ``residual`` or ``x``).  ``normed``: a buffer of x's
    dtype that also receives the normalised rows (it may be ``x`` or ``residual``, not
    ``residual_out``).  Rows may be strided."""
    if x.dtype not in _DT:
        raise ValueError("x must be f32/bf16/f16")
    dev, dt = x.device, x.dtype
    ldx = _rows(x, "x")
    shape = n, d = x.shape
    _tensor(weight, "weight", (dt, torch.float32), (d,), dev)
    ldr = 0 if residual is None else _rows(residual, "residual", dt, shape, dev)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without a residual")
    ldn = 0
    if normed is not None:
        ldn = _rows(normed, "normed", dt, shape, dev)
        if residual_out is not None and normed.data_ptr() == residual_out.data_ptr() and n and d:
            raise ValueError("normed and residual_out must be different buffers")
    with _On(dev, stream) as s:
        ldo = 0
        if residual_out is not None:
            ldo = _rows(residual_out, "residual_out", dt, shape, dev)
            _shared(residual_out, ldo, "residual_out", x, ldx, residual, ldr)
        elif residual is not None:
            residual_out, ldo = torch.empty(shape, dtype=dt, device=dev), d
        if normed is not None:
            _shared(normed, ldn, "normed", x, ldx, residual, ldr)
        if out is None:
            out, ldq = Int8Rows(torch.empty(shape, dtype=torch.int8, device=dev),
                                torch.empty(n, dtype=torch.float32, device=dev)), d
        else:
            ldq = _rows(out.q, "out.q", torch.int8, shape, dev)
            _tensor(out.scale, "out.scale", torch.float32, (n,), dev)
        if d == 0:
            out.scale.fill_(1.0)     # the library leaves rows of no columns alone
        _check(lib.gptqs_rmsnorm_int8(
            x.data_ptr(), _DT[dt], ldx, None if residual is None else residual.data_ptr(), ldr, weight.data_ptr(),
            _DT[weight.dtype], eps, n, d, None if residual_out is None else residual_out.data_ptr(), ldo,
            None if normed is None else normed.data_ptr(), ldn, out.q.data_ptr(), ldq,
            out.scale.data_ptr(), s), "gptqs_rmsnorm_int8")
    return out, (x if residual is None else residual_out)


def _stored(q: Quantized, name: str, device) -> int:
    """q is a layer on an integer grid with whole arrays on ``device``; its rows."""
    if q.fp4:
        raise ValueError(f"{name} is on the E2M1 grid; the products read integer-grid codes")
    c, S, Z = q.codes, q.scales, q.zeros
    d_row = c.shape[0]
    groups = (d_row, _n_groups(q.group_size, q.d_col))
    if not (c.dtype is torch.uint8 and S.dtype is Z.dtype is torch.float16 and c.device == S.device == Z.device == device
            and c.shape == (d_row, code_bytes(q.bits, q.d_col)) and S.shape == Z.shape == groups
            and c.is_contiguous() and S.is_contiguous() and Z.is_contiguous()):
        _dev(c, f"{name}.codes")
        _check_quantized(q, name, d_row, device)   # says which
    return d_row


def _out(out, n: int, d_row: int, out_dtype, device, x):
    if out is None:
        if out_dtype not in _DT:
            raise ValueError("out_dtype must be f32/bf16/f16")
        return torch.empty((n, d_row), dtype=out_dtype, device=device)
    _tensor(out, "out", tuple(_DT), (n, d_row), device)
    if n and d_row and x.shape[1]:                # a workgroup writes its rows of y while others read x
        at, xat = out.data_ptr(), x.data_ptr()
        if at < xat + ((n - 1) * x.stride(0) + x.shape[1]) * x.itemsize and xat < at + out.nbytes:
            raise ValueError("out overlaps x")
    return out


def linear_int8(q: Quantized, x: Int8Rows, out_dtype=torch.float32, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """y = (x.q * x.scale) What^T on the stored format and the 8-bit rows (gptqs_linear_int8):
    int8 products, exact integer sums per group, fp32 across groups.  x.q may be strided."""
    dev = x.q.device
    ldx = _rows(x.q, "x.q", torch.int8)
    n, d_col = x.q.shape
    if d_col != q.d_col:
        raise ValueError(f"x.q has {d_col} columns, the layer {q.d_col}")
    _tensor(x.scale, "x.scale", torch.float32, (n,), dev)
    d_row = _stored(q, "q", dev)
    with _On(dev, stream) as s:
        out = _out(out, n, d_row, out_dtype, dev, x.q)
        if d_col == 0:
            out.zero_()              # a sum of nothing; the library leaves it alone
        _check(lib.gptqs_linear_int8(q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), d_row, d_col, q.bits,
                                     q.group_size, x.q.data_ptr(), ldx, x.scale.data_ptr(), n, out.data_ptr(),
                                     _DT[out.dtype], s), "gptqs_linear_int8")
    return out


def linear_lora_workspace_size(n_tokens: int, d_col: int, rank: int) -> int:
    return lib.gptqs_linear_lora_workspace_size(n_tokens, d_col, rank)


def linear_lora(q: Quantized, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor,
                scaling: torch.Tensor | None = None, out_dtype=torch.float32, out: torch.Tensor | None = None,
                ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = What x[t] + scaling[a] B[a] (A[a] x[t]), a = ids[t] (gptqs_linear_lora): the
    projection is shared, the adapters (A: n_adapters x rank x d_col, B: n_adapters x d_row
    x rank, x's dtype) are the tokens' own; a token whose id (int32) is outside the table
    takes the projection alone.  x (bf16/f16) may be strided."""
    dev, dt = x.device, x.dtype
    ldx = _rows(x, "x")
    n, d_col = x.shape
    if dt not in (torch.bfloat16, torch.float16) or d_col != q.d_col:
        raise ValueError(f"x must be bf16/f16 with the layer's {q.d_col} columns")
    d_row = _stored(q, "q", dev)
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A and B must be n_adapters x rank x d_col and n_adapters x d_row x rank")
    m, rank, _ = A.shape
    _tensor(A, "A", dt, (m, rank, d_col), dev)
    _tensor(B, "B", dt, (m, d_row, rank), dev)
    _tensor(ids, "ids", torch.int32, (n,), dev)
    if scaling is not None:
        _tensor(scaling, "scaling", torch.float32, (m,), dev)
    with _On(dev, stream) as s:
        out = _out(out, n, d_row, out_dtype, dev, x)
        if d_col == 0:
            out.zero_()              # a sum of nothing; the library leaves it alone
        ws = _workspace(linear_lora_workspace_size(n, d_col, rank) if m else 0, dev, ws)
        _check(lib.gptqs_linear_lora(q.codes.data_ptr(), q.scales.data_ptr(), q.zeros.data_ptr(), d_row, d_col, q.bits,
                                     q.group_size, x.data_ptr(), _DT[dt], n, ldx, A.data_ptr(), B.data_ptr(), m, rank,
                                     ids.data_ptr(), None if scaling is None else scaling.data_ptr(), out.data_ptr(),
                                     _DT[out.dtype], None if ws is None else ws.data_ptr(),
                                     0 if ws is None else ws.numel(), s), "gptqs_linear_lora")
    return out


def moe_workspace_size(n_tokens: int, d: int, f: int, n_experts: int, top_k: int) -> int:
    return lib.gptqs_moe_workspace_size(n_tokens, d, f, n_experts, top_k)


def moe(x: torch.Tensor, router: torch.Tensor, up: Quantized, down: Quantized, top_k: int, renormalize: bool = True,
        out_dtype=torch.float32, out: torch.Tensor | None = None, ids: torch.Tensor | None = None,
        weights: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """A mixture-of-experts layer for a few tokens on stored experts (gptqs_moe): router
    (n_experts x d, x's dtype), softmax and top-k, silu(gate) * up, down, weighted sum.
    ``up`` holds every expert's gate rows, then its up rows, as one layer of n_experts * 2 f
    rows and d columns; ``down`` one of n_experts * d rows and f columns (``torch.cat`` of
    the experts' codes, scales and zeros).  x (bf16/f16) may be strided.  Returns (y, ids,
    weights): the chosen experts per token in falling order of their logits, int32, and
    their weights, fp32."""
    dev, dt = x.device, x.dtype
    ldx = _rows(x, "x")
    n, d = x.shape
    if dt not in (torch.bfloat16, torch.float16):
        raise ValueError("x must be bf16/f16")
    if router.dim() != 2:
        raise ValueError("router must be n_experts x d")
    e = router.shape[0]
    _tensor(router, "router", dt, (e, d), dev)
    if (up.bits, up.group_size) != (down.bits, down.group_size):
        raise ValueError("up and down must have the same bits and group size")
    f = down.d_col
    up_rows, down_rows = _stored(up, "up", dev), _stored(down, "down", dev)
    if (up_rows, up.d_col, down_rows) != (e * 2 * f, d, e * d):
        raise ValueError(f"up must be {e * 2 * f} x {d} and down {e * d} x {f}, not {up_rows} x {up.d_col} and "
                         f"{down_rows} x {f}")
    with _On(dev, stream) as s:
        out = _out(out, n, d, out_dtype, dev, x)
        if ids is None:
            ids = torch.empty((n, top_k), dtype=torch.int32, device=dev)
        _tensor(ids, "ids", torch.int32, (n, top_k), dev)
        if weights is None:
            weights = torch.empty((n, top_k), dtype=torch.float32, device=dev)
        _tensor(weights, "weights", torch.float32, (n, top_k), dev)
        ws = _workspace(moe_workspace_size(n, d, f, e, top_k), dev, ws)
        _check(lib.gptqs_moe(x.data_ptr(), _DT[dt], n, d, ldx, router.data_ptr(), e, top_k, int(bool(renormalize)), f,
                             up.codes.data_ptr(), up.scales.data_ptr(), up.zeros.data_ptr(), down.codes.data_ptr(),
                             down.scales.data_ptr(), down.zeros.data_ptr(), up.bits, up.group_size, out.data_ptr(),
                             _DT[out.dtype], ids.data_ptr(), weights.data_ptr(),
                             None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s), "gptqs_moe")
    return out, ids, weights
