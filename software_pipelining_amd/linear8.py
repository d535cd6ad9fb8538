"""The 8-bit linear layer's operators of libtilepipe: the root-mean-square norm
with the residual's addition, its gradient, the block quantiser and the
block-scaled product (the C ABI's section "8-bit linear layers").

Matrices are 2-D GPU tensors with unit column stride and any row stride of at
least their columns. 8-bit results are ``torch.float8_e4m3fn`` or
``torch.float8_e5m2`` with a float32 scale for each block of 128; a number is
its 8-bit value times its block's scale. The functions are not recorded by
autograd: a training step calls the gradients itself.

Outputs and workspaces come from torch's allocator. Work is enqueued on the
device's current stream, or on ``stream``: then the outputs belong to that
stream, and the inputs are marked as used on it.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from .tilepipe import _check, _load

BLOCK = 128
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_EIGHT = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 4}
_CODES = {"same": -1, "e4m3": 3, "e5m2": 4}
_FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}

try:        # the direct calls; without them every call goes the long way below
    from . import _linear8 as _direct
except ImportError:
    _direct = None

_empty = torch.empty
_tuple = tuple.__new__        # a NamedTuple of a tuple, without going through its own __new__
_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice


class RmsNorm(NamedTuple):
    """out: the norm's output; scale: its blocks' scales (None unless 8-bit);
    sum: x + residual (None without a residual); rstd: for the gradient (None
    unless asked for)."""
    out: torch.Tensor
    scale: Optional[torch.Tensor]
    sum: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


class BlockQuantized(NamedTuple):
    """q, scale: x in blocks along its rows (or in squares); qt, scale_t: x
    transposed in blocks along its own rows. Those not asked for are None."""
    q: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    qt: Optional[torch.Tensor]
    scale_t: Optional[torch.Tensor]


def _matrix(t, name: str, types) -> int:
    """Row stride of a matrix in elements; raises unless t is one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of "
                        f"{', '.join(str(k) for k in types)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (libtilepipe has no CPU path)")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D view")
    rows, cols = t.shape
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        return max(1, cols)      # one row: any stride will do
    if row < cols:
        raise ValueError(f"the rows of {name} overlap")
    return row


def _like(t, name: str, x) -> int:
    """Row stride of a matrix of x's shape, type and device."""
    s = _matrix(t, name, (x.dtype,))
    if t.shape != x.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(x.shape)}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}; expected {x.device}")
    return s


def _vector(t, name: str, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {shape}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}; expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _format(name: str):
    try:
        return _FORMATS[name]
    except KeyError:
        raise ValueError(f"unknown out_format {name!r}; expected one of {sorted(_FORMATS)}") from None


def _eight_bit_empty(rows: int, cols: int, dtype, device):
    """Rows on a stride of a multiple of 16 bytes."""
    if cols % 16 == 0:
        return _empty(rows, cols, dtype=dtype, device=device)
    return torch.empty_strided((rows, cols), (cols + 15 & ~15, 1), dtype=dtype, device=device)


def _elsewhere(fn, stream, inputs, *args, **kwargs):
    """fn with `stream` current, its inputs marked as used there."""
    for t in inputs:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.device != stream.device:
            raise ValueError(f"stream is on {stream.device}; expected {t.device}")
    with torch.cuda.stream(stream):
        for t in inputs:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        return fn(*args, **kwargs)


def _call(name: str, device, *args) -> None:
    index = device.index
    fn = getattr(_load(), name)
    if index == _get_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def rms_norm(x, weight, eps: float = 1e-6, residual=None, out_format: str = "same",
             save_rstd: bool = False, stream=None) -> RmsNorm:
    """Root-mean-square norm of each row of s = x + residual (or of x):
    y = s * rstd * weight with rstd = 1 / sqrt(mean(s^2) + eps).

    x, residual: (rows, cols) bfloat16, float16 or float32, weight: (cols,) of
    the same type. out_format "same" gives y in x's type, "e4m3" or "e5m2" in
    8 bits with a scale for each row and 128 columns, rounded from 32 bits.
    With a residual, ``sum`` is s in x's type."""
    if stream is not None:
        return _elsewhere(rms_norm, stream, (x, weight, residual), x, weight, eps, residual,
                          out_format, save_rstd)
    if _direct is not None:
        got = _direct.rms_norm(x, weight, eps, residual, _CODES.get(out_format, -2), save_rstd)
        if got is not None:
            return _tuple(RmsNorm, got)
    xs = _matrix(x, "x", _DTYPES)
    rows, cols = x.shape
    dtype, device = x.dtype, x.device
    _vector(weight, "weight", (cols,), dtype, device)
    code = _DTYPES[dtype]
    total = scale = rstd = None
    rs = ss = 0
    if residual is not None:
        rs = _like(residual, "residual", x)
        total, ss = _empty(rows, cols, dtype=dtype, device=device), max(1, cols)
    if out_format == "same":
        out, os_, out_code = _empty(rows, cols, dtype=dtype, device=device), max(1, cols), code
    else:
        eight = _format(out_format)
        out, out_code = _eight_bit_empty(rows, cols, eight, device), _EIGHT[eight]
        os_ = max(1, cols + 15 & ~15)
        scale = _empty(rows, -(-cols // BLOCK), dtype=torch.float32, device=device)
    if save_rstd:
        rstd = _empty(rows, dtype=torch.float32, device=device)
    if rows and cols:
        _call("tp_rms_norm", device, x.data_ptr(), xs, _ptr(residual), rs, weight.data_ptr(), rows, cols,
              code, eps, _ptr(total), ss, out.data_ptr(), os_, out_code, _ptr(scale), _ptr(rstd))
    elif rstd is not None:
        rstd.fill_(float("nan"))        # the mean of no columns
    return RmsNorm(out, scale, total, rstd)


def rms_norm_backward(dy, x, weight, rstd, dsum=None, stream=None):
    """Gradients of rms_norm: (dx, dweight). dy: the gradient of its output, x:
    its input (``sum`` where there was a residual), rstd: as it saved it,
    dsum: the gradient that reaches that sum another way, added to dx. dx (the
    gradient of x and of the residual) has x's type, dweight is float32."""
    if stream is not None:
        return _elsewhere(rms_norm_backward, stream, (dy, x, weight, rstd, dsum), dy, x, weight, rstd,
                          dsum)
    if _direct is not None:
        got = _direct.rms_norm_backward(dy, x, weight, rstd, dsum)
        if got is not None:
            return got
    xs = _matrix(x, "x", _DTYPES)
    dys = _like(dy, "dy", x)
    dss = 0 if dsum is None else _like(dsum, "dsum", x)
    rows, cols = x.shape
    dtype, device = x.dtype, x.device
    _vector(weight, "weight", (cols,), dtype, device)
    _vector(rstd, "rstd", (rows,), torch.float32, device)
    code = _DTYPES[dtype]
    dx = _empty(rows, cols, dtype=dtype, device=device)
    dw = _empty(cols, dtype=torch.float32, device=device)
    if cols:
        need = _load().tp_rms_norm_backward_workspace_bytes(rows, cols, code)
        ws = _empty(need, dtype=torch.uint8, device=device)
        _call("tp_rms_norm_backward", device, dy.data_ptr(), dys, x.data_ptr(), xs, weight.data_ptr(),
              rstd.data_ptr(), _ptr(dsum), dss, rows, cols, code, dx.data_ptr(), max(1, cols),
              dw.data_ptr(), ws.data_ptr(), need)
    return dx, dw


def block_quantize(x, out_format: str = "e4m3", square: bool = False, straight: bool = True,
                   transposed: bool = False, stream=None) -> BlockQuantized:
    """x (rows, cols) in 8 bits with a scale for each block of 128.

    straight: ``q`` (rows, cols) with ``scale`` (rows, ceil(cols / 128)), or
    with square (ceil(rows / 128), ceil(cols / 128)). transposed: ``qt``
    (cols, rows), x transposed in blocks along its own rows, with ``scale_t``.
    x is read once for both. 8-bit rows lie on a stride of a multiple of 16
    bytes."""
    if stream is not None:
        return _elsewhere(block_quantize, stream, (x,), x, out_format, square, straight, transposed)
    if _direct is not None:
        got = _direct.block_quantize(x, _CODES.get(out_format, -2), square, straight, transposed)
        if got is not None:
            return _tuple(BlockQuantized, got)
    xs = _matrix(x, "x", _DTYPES)
    if not straight and not transposed:
        raise ValueError("nothing to make: neither straight nor transposed")
    eight = _format(out_format)
    rows, cols = x.shape
    device = x.device
    down, across = -(-rows // BLOCK), -(-cols // BLOCK)
    q = scale = qt = scale_t = None
    if straight:
        q = _eight_bit_empty(rows, cols, eight, device)
        scale = _empty(down if square else rows, across, dtype=torch.float32, device=device)
    if transposed:
        qt = _eight_bit_empty(cols, rows, eight, device)
        scale_t = _empty(across if square else cols, down, dtype=torch.float32, device=device)
    if rows and cols:
        _call("tp_block_quantize", device, x.data_ptr(), xs, rows, cols, _DTYPES[x.dtype], int(bool(square)),
              _EIGHT[eight], _ptr(q), cols + 15 & ~15, _ptr(scale), _ptr(qt), rows + 15 & ~15,
              _ptr(scale_t))
    return BlockQuantized(q, scale, qt, scale_t)


def block_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, stream=None):
    """(m, n) = A B^T of 8-bit matrices a (m, k) and b (n, k), each e4m3 or
    e5m2, with a_scale (m, ceil(k / 128)) and b_scale (n, ceil(k / 128)) or, for
    a weight in squares, (ceil(n / 128), ceil(k / 128)). Blocks are added in
    float32 and rounded once to out_dtype (bfloat16, float16 or float32). So are
    the 128 products of a block for float16 and float32; for bfloat16 the 8-bit
    matrix instructions add them, each eight to within 2^-13 of its largest
    product for each of the others."""
    if stream is not None:
        return _elsewhere(block_matmul, stream, (a, a_scale, b, b_scale), a, a_scale, b, b_scale, out_dtype)
    if _direct is not None:
        got = _direct.block_matmul(a, a_scale, b, b_scale, _DTYPES.get(out_dtype, -1))
        if got is not None:
            return got
    a_s = _matrix(a, "a", _EIGHT)
    b_s = _matrix(b, "b", _EIGHT)
    m, k = a.shape
    n = b.shape[0]
    device = a.device
    if b.shape[1] != k:
        raise ValueError(f"a has {k} columns and b {b.shape[1]}")
    if b.device != device:
        raise ValueError(f"b is on {b.device}; expected {device}")
    if out_dtype not in _DTYPES:
        raise TypeError(f"out_dtype must be one of {', '.join(str(t) for t in _DTYPES)}")
    blocks = -(-k // BLOCK)
    _vector(a_scale, "a_scale", (m, blocks), torch.float32, device)
    square = isinstance(b_scale, torch.Tensor) and tuple(b_scale.shape) == (-(-n // BLOCK), blocks)
    if not square:
        _vector(b_scale, "b_scale", (n, blocks), torch.float32, device)
    else:
        _vector(b_scale, "b_scale", (-(-n // BLOCK), blocks), torch.float32, device)
    out = _empty(m, n, dtype=out_dtype, device=device)
    if m and n:
        need = _load().tp_block_matmul_workspace_bytes(m, n, k, _DTYPES[out_dtype])
        ws = _empty(need, dtype=torch.uint8, device=device) if need > 0 else None
        _call("tp_block_matmul", device, a.data_ptr(), a_s, _EIGHT[a.dtype], a_scale.data_ptr(),
              b.data_ptr(), b_s, _EIGHT[b.dtype], b_scale.data_ptr(), int(square), m, n, k,
              out.data_ptr(), n, _DTYPES[out_dtype], _ptr(ws), max(0, need))
    return out
