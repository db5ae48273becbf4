"""The expert layer above the tables, and the bound on its gradients
(include/tbe_experts.h): a router, token rows sorted by expert and back,
8-bit block-scaled matrix products over experts, and the global gradient norm
with clipping.

The `tbe_*` functions have the names of the C entry points they call, check
types, shapes, devices and strides, and pass raw pointers and the current
stream.  `route`, `ExpertRows`, `F8Matrix`, `quantize_f8`, `matmul_f8` and
`clip_grad_norm` allocate their results; what they allocate themselves is not
checked again.  There is no fallback: without the library every call raises.
"""
from __future__ import annotations

import array
import ctypes as C
import functools
import operator
from typing import Optional, Sequence

import torch

from ._experts_abi import (TBE_F8_BLOCK, TBE_F8_SQUARE, TBE_MAX_CHOICES, TBE_MAX_EXPERTS,
                           TBE_ROUTE_RENORMALIZE)
from ._lib import ITYPE_OF_TORCH, WDTYPE_OF_TORCH, _check, _stream, lib

_F8 = torch.float8_e4m3fn


def _up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


# The short ways to the current device and stream (current_stream() builds an object: 2.7 us
# against 0.1), where this torch has them; nothing of it is needed to import the package.
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _matrix(t, name, dtypes=WDTYPE_OF_TORCH, dims=2):
    """(pointer, row stride in elements) of a tensor whose last axis is contiguous
    (rows may be strided, and do not overlap)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    width = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), width
    if t.numel() and width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    ld = t.stride(-2) if shape[-2] > 1 else width
    if ld < width:
        raise ValueError(f"rows of {name} must not overlap")
    return t.data_ptr(), ld


def _whole(t, name, dtypes, shape):
    """Pointer of a contiguous tensor of one of `dtypes` and of `shape`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on(stream, first, *tensors):
    """The stream to launch on: `stream`, or the current one of the device that all
    tensors are on, which has to be the current device."""
    d = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on one device")
    if d < 0:
        raise ValueError("tensors must be device tensors")
    if d != _get_device():
        raise ValueError(f"tensors are on device {d}, not on the current device")
    return _raw_stream(d) if stream is None else _stream(stream)


_I32, _F32 = (torch.int32,), (torch.float32,)


def _counts(*counts):
    """Counts that the library takes in 32 bits (its binding would drop the bits above)."""
    for n in counts:
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"a count of {n} does not fit 32 bits")


def _width(t, name, dims=2):
    """Size of the last of a tensor's `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    return t.shape[-1]


# ---------------------------------------------------------------------- router


def tbe_route(logits: torch.Tensor, k: int, valid: Optional[torch.Tensor], flags: int,
              ids: torch.Tensor, weights: torch.Tensor, stream=None) -> None:
    p, ld = _matrix(logits, "logits")
    n, e = logits.shape
    _counts(k, e)
    st = _on(stream, logits, valid, ids, weights)
    v = None
    if valid is not None:
        v = _whole(valid, "valid", (torch.uint8, torch.bool), (n,))
    _check("tbe_route", lib().tbe_route(
        n, e, k, WDTYPE_OF_TORCH[logits.dtype], p, ld, v, flags,
        _whole(ids, "ids", _I32, (n, k)), _whole(weights, "weights", _F32, (n, k)),
        st))


def tbe_route_backward(logits: torch.Tensor, ids: torch.Tensor, grad_weights: torch.Tensor,
                       flags: int, grad_logits: torch.Tensor, stream=None) -> None:
    (p, ld), (g, ldg) = _matrix(logits, "logits"), _matrix(grad_logits, "grad_logits")
    n, e = logits.shape
    k = _width(ids, "ids")
    _counts(k, e)
    if grad_logits.shape != logits.shape or grad_logits.dtype != logits.dtype:
        raise ValueError("grad_logits must have the logits' shape and dtype")
    st = _on(stream, logits, ids, grad_weights, grad_logits)
    _check("tbe_route_backward", lib().tbe_route_backward(
        n, e, k, WDTYPE_OF_TORCH[logits.dtype], p, ld, _whole(ids, "ids", _I32, (n, k)),
        _whole(grad_weights, "grad_weights", _F32, (n, k)), flags, g, ldg,
        st))


def route(logits: torch.Tensor, k: int, valid: Optional[torch.Tensor] = None,
          renormalize: bool = False):
    """(ids int32 [N, k], weights float32 [N, k]) of the k largest logits of each
    token: softmax weights over all experts, or over the chosen ones
    (`renormalize`).  valid: uint8 or bool [N], tokens with 0 get no expert."""
    p, ld = _matrix(logits, "logits")
    n, e = logits.shape
    _counts(k, e)
    st = _on(None, logits, valid)
    v = None
    if valid is not None:
        v = _whole(valid, "valid", (torch.uint8, torch.bool), (n,))
    shape, dev = (n, k), logits.device
    ids = torch.empty(shape, dtype=torch.int32, device=dev)
    weights = torch.empty(shape, dtype=torch.float32, device=dev)
    _check("tbe_route", lib().tbe_route(
        n, e, k, WDTYPE_OF_TORCH[logits.dtype], p, ld, v, TBE_ROUTE_RENORMALIZE if renormalize else 0,
        ids.data_ptr(), weights.data_ptr(), st))
    return ids, weights


def route_backward(logits: torch.Tensor, ids: torch.Tensor, grad_weights: torch.Tensor,
                   renormalize: bool = False) -> torch.Tensor:
    """Gradient with respect to the logits of `route`'s weights."""
    p, ld = _matrix(logits, "logits")
    n, e = logits.shape
    shape = (n, _width(ids, "ids"))
    _counts(shape[1], e)
    st = _on(None, logits, ids, grad_weights)
    i, w = _whole(ids, "ids", _I32, shape), _whole(grad_weights, "grad_weights", _F32, shape)
    grad = torch.empty_like(logits, memory_format=torch.contiguous_format)
    _check("tbe_route_backward", lib().tbe_route_backward(
        n, e, shape[1], WDTYPE_OF_TORCH[logits.dtype], p, ld, i, w,
        TBE_ROUTE_RENORMALIZE if renormalize else 0, grad.data_ptr(), e, st))
    return grad


# ------------------------------------------------------------- rows by expert


@functools.lru_cache(maxsize=256)  # a function of its sizes alone
def tbe_expert_rows(tokens: int, k: int, experts: int, align: int) -> int:
    _counts(k, experts, align)
    n = C.c_int64()
    _check("tbe_expert_rows", lib().tbe_expert_rows(tokens, k, experts, align, C.byref(n)))
    return n.value


@functools.lru_cache(maxsize=256)
def tbe_expert_sort_workspace_size(tokens: int, k: int, experts: int, align: int) -> int:
    _counts(k, experts, align)
    n = C.c_size_t()
    _check("tbe_expert_sort_workspace_size",
           lib().tbe_expert_sort_workspace_size(tokens, k, experts, align, C.byref(n)))
    return n.value


def tbe_expert_sort(ids: torch.Tensor, experts: int, align: int, offsets: torch.Tensor,
                    slots: torch.Tensor, source: torch.Tensor, ws: Optional[torch.Tensor],
                    stream=None) -> None:
    _width(ids, "ids")
    n, k = ids.shape
    rows = tbe_expert_rows(n, k, experts, align)
    p = _whole(ids, "ids", tuple(ITYPE_OF_TORCH), (n, k))
    st = _on(stream, ids, offsets, slots, source, ws)
    _check("tbe_expert_sort", lib().tbe_expert_sort(
        n, k, experts, align, ITYPE_OF_TORCH[ids.dtype], p,
        _whole(offsets, "offsets", _I32, (experts + 1,)), _whole(slots, "slots", _I32, (n, k)),
        _whole(source, "source", _I32, (rows,)), None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel() * ws.element_size(),
        st))


def tbe_expert_dispatch(x: torch.Tensor, slots: torch.Tensor, source: torch.Tensor,
                        out: torch.Tensor, stream=None) -> None:
    (p, ldx), (o, ldo) = _matrix(x, "x"), _matrix(out, "out", (x.dtype,))
    n, w = x.shape
    rows = out.shape[0]
    if out.shape[1] != w:
        raise ValueError("x and out must have one width")
    k = _width(slots, "slots")
    _counts(k)
    st = _on(stream, x, slots, source, out)
    _check("tbe_expert_dispatch", lib().tbe_expert_dispatch(
        n, k, rows, w, WDTYPE_OF_TORCH[x.dtype], p, ldx, _whole(slots, "slots", _I32, (n, k)),
        _whole(source, "source", _I32, (rows,)), o, ldo, st))


def tbe_expert_dispatch_f8(x: torch.Tensor, slots: torch.Tensor, source: torch.Tensor,
                           values: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    p, ldx = _matrix(x, "x")
    n, w = x.shape
    rows, k = _width(source, "source", 1), _width(slots, "slots")
    _counts(k)
    st = _on(stream, x, slots, source, values, scales)
    vs, ss = F8Matrix.shapes(rows, w)
    _check("tbe_expert_dispatch_f8", lib().tbe_expert_dispatch_f8(
        n, k, rows, w, WDTYPE_OF_TORCH[x.dtype], p, ldx, _whole(slots, "slots", _I32, (n, k)),
        _whole(source, "source", _I32, (rows,)), _whole(values, "values", (_F8,), vs),
        _whole(scales, "scales", (torch.uint8,), ss), st))


def tbe_expert_combine(y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor],
                       out: torch.Tensor, stream=None) -> None:
    (p, ldy), (o, ldo) = _matrix(y, "y"), _matrix(out, "out", (y.dtype,))
    rows, w = y.shape
    n, k = out.shape[0], _width(slots, "slots")
    _counts(k)
    if out.shape[1] != w:
        raise ValueError("y and out must have one width")
    st = _on(stream, y, slots, weights, out)
    _check("tbe_expert_combine", lib().tbe_expert_combine(
        n, k, rows, w, WDTYPE_OF_TORCH[y.dtype], p, ldy, _whole(slots, "slots", _I32, (n, k)),
        None if weights is None else _whole(weights, "weights", _F32, (n, k)), o, ldo,
        st))


def tbe_expert_combine_backward(grad_out: torch.Tensor, y: torch.Tensor, slots: torch.Tensor,
                                source: torch.Tensor, weights: torch.Tensor,
                                grad_y: torch.Tensor, grad_weights: torch.Tensor,
                                stream=None) -> None:
    g, ldg = _matrix(grad_out, "grad_out")
    same = (grad_out.dtype,)
    (p, ldy), (o, ldo) = _matrix(y, "y", same), _matrix(grad_y, "grad_y", same)
    rows, w = y.shape
    n, k = grad_out.shape[0], _width(slots, "slots")
    _counts(k)
    if grad_out.shape[1] != w or grad_y.shape != y.shape:
        raise ValueError("grad_out, y and grad_y must have one width, grad_y the rows of y")
    st = _on(stream, grad_out, y, slots, source, weights, grad_y, grad_weights)
    _check("tbe_expert_combine_backward", lib().tbe_expert_combine_backward(
        n, k, rows, w, WDTYPE_OF_TORCH[y.dtype], g, ldg, p, ldy,
        _whole(slots, "slots", _I32, (n, k)), _whole(source, "source", _I32, (rows,)),
        _whole(weights, "weights", _F32, (n, k)), o, ldo,
        _whole(grad_weights, "grad_weights", _F32, (n, k)), st))


class ExpertRows:
    """One sort of a batch's choices by expert, and the row traffic through it.

    ids [N, k] (int32 or int64; outside [0, experts): dropped).  Segments start
    on multiples of `align` rows (128 where `matmul_f8_segments` is to take
    them).  offsets [experts + 1], slots [N, k] and source [rows] stay on the
    device."""

    def __init__(self, ids: torch.Tensor, experts: int, align: int = 1):
        if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
            raise ValueError("ids must be a tensor of 2 dimensions")
        n, k = shape = ids.shape
        self.tokens, self.k, self.experts, self.align = n, k, experts, align
        self.rows = rows = tbe_expert_rows(n, k, experts, align)
        need = tbe_expert_sort_workspace_size(n, k, experts, align)
        p, st = _whole(ids, "ids", ITYPE_OF_TORCH, shape), _on(None, ids)
        dev, i32 = ids.device, torch.int32
        self.offsets = torch.empty(experts + 1, dtype=i32, device=dev)
        self.slots = torch.empty(shape, dtype=i32, device=dev)
        self.source = torch.empty(rows, dtype=i32, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _check("tbe_expert_sort", lib().tbe_expert_sort(
            n, k, experts, align, ITYPE_OF_TORCH[ids.dtype], p, self.offsets.data_ptr(),
            self.slots.data_ptr(), self.source.data_ptr(), ws.data_ptr() if need else None, need,
            st))

    def _rows(self, t: torch.Tensor, name: str, rows: int):
        """(pointer, row stride, width, type code) of a matrix of `rows` rows."""
        p, ld = _matrix(t, name)
        if t.shape[0] != rows:
            raise ValueError(f"{name} must have {rows} rows, not {t.shape[0]}")
        return p, ld, t.shape[1], WDTYPE_OF_TORCH[t.dtype]

    def _weights(self, weights):
        return _whole(weights, "weights", _F32, (self.tokens, self.k))

    def dispatch(self, x: torch.Tensor) -> torch.Tensor:
        """Token rows [N, W] to expert rows [rows, W]; rows without a choice are zero."""
        p, ld, w, code = self._rows(x, "x", self.tokens)
        st = _on(None, x, self.slots)
        out = x.new_empty((self.rows, w))
        _check("tbe_expert_dispatch", lib().tbe_expert_dispatch(
            self.tokens, self.k, self.rows, w, code, p, ld, self.slots.data_ptr(), self.source.data_ptr(),
            out.data_ptr(), w, st))
        return out

    def dispatch_f8(self, x: torch.Tensor) -> "F8Matrix":
        """quantize_f8(dispatch(x)) in one pass over the tokens."""
        p, ld, w, code = self._rows(x, "x", self.tokens)
        st = _on(None, x, self.slots)
        m = F8Matrix.empty(self.rows, w, x.device)
        _check("tbe_expert_dispatch_f8", lib().tbe_expert_dispatch_f8(
            self.tokens, self.k, self.rows, w, code, p, ld, self.slots.data_ptr(), self.source.data_ptr(),
            m.values.data_ptr(), m.scales.data_ptr(), st))
        return m

    def _combine(self, y, weights):
        p, ld, w, code = self._rows(y, "y", self.rows)
        st = _on(None, y, self.slots, weights)
        wp = None if weights is None else self._weights(weights)
        out = y.new_empty((self.tokens, w))
        _check("tbe_expert_combine", lib().tbe_expert_combine(
            self.tokens, self.k, self.rows, w, code, p, ld, self.slots.data_ptr(), wp, out.data_ptr(), w,
            st))
        return out

    def dispatch_backward(self, grad_rows: torch.Tensor) -> torch.Tensor:
        """Gradient of dispatch: every token's expert rows summed."""
        return self._combine(grad_rows, None)

    def combine(self, y: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """Expert rows [rows, W] to token rows [N, W], weighted by weights [N, k]."""
        if weights is None:
            raise TypeError("weights must be a torch tensor")
        return self._combine(y, weights)

    def combine_backward(self, grad_out: torch.Tensor, y: torch.Tensor, weights: torch.Tensor):
        """(grad_y, grad_weights) of combine."""
        g, ldg, w, code = self._rows(grad_out, "grad_out", self.tokens)
        p, ld, wy, ycode = self._rows(y, "y", self.rows)
        if wy != w or ycode != code:
            raise ValueError("grad_out and y must have one width and dtype")
        st = _on(None, grad_out, y, self.slots, weights)
        wp = self._weights(weights)
        grad_y = y.new_empty((self.rows, w))
        grad_w = torch.empty((self.tokens, self.k), dtype=torch.float32, device=y.device)
        _check("tbe_expert_combine_backward", lib().tbe_expert_combine_backward(
            self.tokens, self.k, self.rows, w, code, g, ldg, p, ld, self.slots.data_ptr(), self.source.data_ptr(), wp,
            grad_y.data_ptr(), w, grad_w.data_ptr(), st))
        return grad_y, grad_w


# --------------------------------------------------------------- 8-bit product


class F8Matrix:
    """A matrix [rows, cols], or one for each expert, in the 8-bit form: values
    e4m3 [..., rows, cols rounded up to 128], scales uint8 [..., rows or (square)
    ceil(rows / 128), blocks of 128 columns rounded up to 4].  A value stands for
    value * 2^(scale - 127), or NaN at a scale of 255."""

    __slots__ = ("values", "scales", "rows", "cols", "square")

    def __init__(self, values: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                 square: bool = False):
        vs, ss = self.shapes(rows, cols, square, tuple(values.shape[:-2]))
        if not values.is_cuda or not scales.is_cuda:
            raise ValueError("values and scales must be device tensors")
        if values.get_device() != scales.get_device():
            raise ValueError("values and scales must be on one device")
        _whole(values, "values", (_F8,), vs)
        _whole(scales, "scales", (torch.uint8,), ss)
        self.values, self.scales = values, scales
        self.rows, self.cols, self.square = int(rows), int(cols), bool(square)

    @staticmethod
    def shapes(rows: int, cols: int, square: bool = False, batch: Sequence[int] = ()):
        """Shapes of the values and the scales."""
        blocks = (cols + 127) // 128
        sr = (rows + 127) // 128 if square else rows
        return (*batch, rows, blocks * 128), (*batch, sr, (blocks + 3) // 4 * 4)

    @classmethod
    def empty(cls, rows: int, cols: int, device, square: bool = False,
              batch: Sequence[int] = ()) -> "F8Matrix":
        vs, ss = cls.shapes(rows, cols, square, batch)
        m = cls.__new__(cls)
        m.values = torch.empty(vs, dtype=_F8, device=device)
        m.scales = torch.empty(ss, dtype=torch.uint8, device=device)
        m.rows, m.cols, m.square = rows, cols, square
        return m

    def float(self) -> torch.Tensor:
        """The values it stands for, in float32 [..., rows, cols] (for checks: plain torch)."""
        blocks = self.values.shape[-1] // TBE_F8_BLOCK
        e = self.scales[..., :blocks].to(torch.int32)
        e = e.repeat_interleave(TBE_F8_BLOCK, dim=-1)
        if self.square:
            e = e.repeat_interleave(TBE_F8_BLOCK, dim=-2)[..., :self.rows, :]
        # the byte is float32's exponent field, but for its ends: 2^-127 is subnormal there, and
        # 255 is no number
        by = (e << 23).masked_fill(e == 0, 1 << 22).masked_fill(e == 255, 0x7fc00000)
        by = by.view(torch.float32)
        return (self.values.float() * by)[..., :self.cols]


def tbe_quantize_f8(x: torch.Tensor, flags: int, row: Optional[F8Matrix],
                    col: Optional[F8Matrix], stream=None) -> None:
    dims = x.dim() if isinstance(x, torch.Tensor) else 0
    if dims not in (2, 3):
        raise ValueError("x must be a tensor of 2 or 3 dimensions")
    p, ldx = _matrix(x, "x", dims=dims)
    batch = x.shape[0] if dims == 3 else 1
    r, c = x.shape[-2:]
    lead = tuple(x.shape[:-2])
    square = bool(flags & TBE_F8_SQUARE)
    ptr = [None] * 4
    st = _on(stream, x)
    for i, (m, mr, mc) in enumerate(((row, r, c), (col, c, r))):
        if m is None:
            continue
        vs, ss = F8Matrix.shapes(mr, mc, square, lead)
        _on(stream, x, m.values, m.scales)
        ptr[2 * i] = _whole(m.values, "values", (_F8,), vs)
        ptr[2 * i + 1] = _whole(m.scales, "scales", (torch.uint8,), ss)
    _check("tbe_quantize_f8", lib().tbe_quantize_f8(
        batch, r, c, WDTYPE_OF_TORCH[x.dtype], p, ldx,
        x.stride(0) if dims == 3 and batch > 1 else 0, flags, *ptr, st))


def _quantize(x, square, rows, cols):
    """New 8-bit forms of x: by rows and / or of its transpose."""
    dims = x.dim() if isinstance(x, torch.Tensor) else 0
    if dims not in (2, 3):
        raise ValueError("x must be a tensor of 2 or 3 dimensions")
    p, ldx = _matrix(x, "x", dims=dims)
    st = _on(None, x)
    r, c = x.shape[-2:]
    lead, dev = tuple(x.shape[:-2]), x.device
    batch = lead[0] if lead else 1
    row = F8Matrix.empty(r, c, dev, square, lead) if rows else None
    col = F8Matrix.empty(c, r, dev, square, lead) if cols else None
    _check("tbe_quantize_f8", lib().tbe_quantize_f8(
        batch, r, c, WDTYPE_OF_TORCH[x.dtype], p, ldx, x.stride(0) if batch > 1 else 0,
        TBE_F8_SQUARE if square else 0,
        row.values.data_ptr() if rows else None, row.scales.data_ptr() if rows else None,
        col.values.data_ptr() if cols else None, col.scales.data_ptr() if cols else None, st))
    return row, col


def quantize_f8(x: torch.Tensor, transpose: bool = False, square: bool = False) -> F8Matrix:
    """The 8-bit form of x [..., R, C] with blocks of 128 along its columns, or of
    its transpose (blocks along the rows).  square: one scale per 128 x 128."""
    return _quantize(x, square, not transpose, transpose)[1 if transpose else 0]


def quantize_f8_pair(x: torch.Tensor, square: bool = False):
    """(quantize_f8(x), quantize_f8(x, transpose=True)) from one read of x."""
    return _quantize(x, square, True, True)


def _out_type(dtype):
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"8-bit products are stored in float16 or bfloat16, not {dtype}")
    return WDTYPE_OF_TORCH[dtype]


def tbe_matmul_f8(a: F8Matrix, b: F8Matrix, offsets: Optional[torch.Tensor], out: torch.Tensor,
                  stream=None) -> None:
    experts = b.values.shape[0] if b.values.dim() == 3 else 1
    _counts(experts)
    if a.values.dim() != 2 or a.square or b.values.dim() > 3:
        raise ValueError("a must be one matrix with a scale a row, b one or one an expert")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    dt = _out_type(out.dtype)
    o, ldo = _matrix(out, "out", (out.dtype,))
    if out.shape != (a.rows, b.rows):
        raise ValueError(f"out must be [{a.rows}, {b.rows}]")
    st = _on(stream, a.values, a.scales, b.values, b.scales, offsets, out)
    if offsets is None and experts != 1:
        raise ValueError("several experts need offsets")
    _check("tbe_matmul_f8", lib().tbe_matmul_f8(
        experts, a.rows, b.rows, a.cols, a.values.data_ptr(), a.scales.data_ptr(),
        b.values.data_ptr(), b.scales.data_ptr(), int(b.square),
        None if offsets is None else _whole(offsets, "offsets", _I32, (experts + 1,)), dt, o,
        ldo, st))


def matmul_f8(a: F8Matrix, b: F8Matrix, offsets: Optional[torch.Tensor] = None,
              dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a [M, K] times the transpose of b [N, K], or of b[e] [E, N, K] for the rows
    [offsets[e], offsets[e + 1]) of each expert; rows of no expert are zero."""
    out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.values.device)
    tbe_matmul_f8(a, b, offsets, out)
    return out


def tbe_matmul_f8_segments(a: F8Matrix, b: F8Matrix, offsets: torch.Tensor, out: torch.Tensor,
                           stream=None) -> None:
    if a.values.dim() != 2 or b.values.dim() != 2 or a.square or b.square:
        raise ValueError("a and b must be single matrices with a scale a row")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    dt = _out_type(out.dtype)
    experts = _width(offsets, "offsets", 1) - 1
    _counts(experts)
    st = _on(stream, a.values, a.scales, b.values, b.scales, offsets, out)
    _check("tbe_matmul_f8_segments", lib().tbe_matmul_f8_segments(
        experts, a.rows, b.rows, a.cols, a.values.data_ptr(), a.scales.data_ptr(),
        b.values.data_ptr(), b.scales.data_ptr(),
        _whole(offsets, "offsets", _I32, (experts + 1,)), dt,
        _whole(out, "out", (out.dtype,), (experts, a.rows, b.rows)), st))


def matmul_f8_segments(a: F8Matrix, b: F8Matrix, offsets: torch.Tensor,
                       dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """out[e] = a[:, s] b[:, s]^T over the segment s of each expert: a [P, M] and
    b [Q, M] with blocks along the M rows (quantize_f8(..., transpose=True)),
    segments on multiples of 128.  The gradient of an expert's weights."""
    out = torch.empty((_width(offsets, "offsets", 1) - 1, a.rows, b.rows), dtype=dtype,
                      device=a.values.device)
    tbe_matmul_f8_segments(a, b, offsets, out)
    return out


# -------------------------------------------------------- gradient norm, clipping


@functools.lru_cache(maxsize=64)
def _clip_workspace(n: int) -> int:
    return tbe_clip_workspace_size([0] * n)  # a function of their number


def tbe_clip_workspace_size(sizes: Sequence[int]) -> int:
    n = C.c_size_t()
    _check("tbe_clip_workspace_size", lib().tbe_clip_workspace_size(
        len(sizes), (C.c_int64 * len(sizes))(*sizes), C.byref(n)))
    return n.value


_numel, _data_ptr, _dtype = torch.Tensor.numel, torch.Tensor.data_ptr, operator.attrgetter("dtype")
_contiguous, _device = torch.Tensor.is_contiguous, torch.Tensor.get_device


def _tensor_list(ts, name):
    """(sizes, type codes, pointers) of contiguous tensors, as arrays."""
    if not all(map(_contiguous, ts)):
        raise ValueError(f"{name} must be contiguous")
    try:
        codes = array.array("i", map(WDTYPE_OF_TORCH.__getitem__, map(_dtype, ts)))
    except KeyError:
        raise TypeError(f"{name} must be float32, float16 or bfloat16") from None
    return array.array("q", map(_numel, ts)), codes, array.array("Q", map(_data_ptr, ts))


def tbe_clip_grad_norm(grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]],
                       max_norm: float, norm: torch.Tensor, ws: torch.Tensor,
                       stream=None) -> None:
    st = _on(stream, norm, ws)
    if len({norm.get_device(), *map(_device, grads), *map(_device, outs or ())}) > 1:
        raise ValueError("all tensors must be on one device")
    sizes, codes, ptrs = _tensor_list(grads, "grads")
    o = None
    if outs is not None:
        osizes, ocodes, optrs = _tensor_list(outs, "outs")
        if osizes != sizes or ocodes != codes:
            raise ValueError("outs must have the sizes and dtypes of grads")
        o = optrs.buffer_info()[0]
    _check("tbe_clip_grad_norm", lib().tbe_clip_grad_norm(
        len(grads), ptrs.buffer_info()[0], o, sizes.buffer_info()[0], codes.buffer_info()[0],
        max_norm, _whole(norm, "norm", _F32, ()), ws.data_ptr(), ws.numel() * ws.element_size(),
        st))


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float,
                   outs: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """The 2-norm over all gradients (device scalar); every gradient times
    min(1, max_norm / (norm + 1e-6)) is written to `outs`, or in place."""
    dev = grads[0].device if len(grads) else torch.device("cuda", _get_device())
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws = torch.empty(_clip_workspace(len(grads)), dtype=torch.uint8, device=dev)
    tbe_clip_grad_norm(grads, outs, max_norm, norm, ws)
    return norm
