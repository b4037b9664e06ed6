"""Operators around a linear layer whose weight Muon trains: layer norm with its
gradient, and 4-bit microscaled (MX) quantisation with the layer's products.

Argument marshalling over the C ABI (include/muon.h), like the rest of the
binding.  Calls run on the tensors' device, on ``stream`` or that device's
current stream, and allocate their results and scratch there.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MUON_BF16, MUON_FP16, MUON_FP32, check

__all__ = ["MxMatrix", "muon_layer_norm", "muon_layer_norm_backward", "muon_mx_quantize", "muon_mx_dequantize",
           "muon_mx_product"]

_DTYPES = {torch.bfloat16: MUON_BF16, torch.float32: MUON_FP32, torch.float16: MUON_FP16}


def _on_stream(body, tensors, stream):
    """body(raw stream) on the device of ``tensors``, with ``stream`` current while it allocates."""
    index = tensors[0].device.index
    for t in tensors:
        if t.device.index != index:
            raise ValueError("all tensors must be on one device")
    if stream is None and index == torch.cuda.current_device():
        return body(torch.cuda.current_stream(index).cuda_stream)
    with torch.cuda.device(index):
        if stream is None:
            stream = torch.cuda.current_stream(index)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=index)
        elif stream.device.index != index:
            raise ValueError("stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            for t in tensors:
                t.record_stream(stream)
            return body(stream.cuda_stream)


def _matrix(t, name, dtype=None):
    """Checks a 2-D CUDA matrix whose rows are contiguous; returns its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows > 1 and ld < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld if rows > 1 else cols


def _rows_of(t, name, dtype=None, shape=None):
    """A tensor (..., cols) as a matrix of rows, without copying."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dim() != 2:
        try:
            t = t.view(t.shape[:-1].numel(), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name} of more than two dimensions must be viewable as rows of its last one") from None
    return t, _matrix(t, name, dtype)


def _vector(t, name, n, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in (torch.float32, dtype):
        raise ValueError(f"{name} must be fp32 or {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values")


def _statistic(t, name, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise ValueError(f"{name} must be an fp32 CUDA tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {tuple(shape)}")


def muon_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm over the last dimension: ``(y, mean, rstd)``.

    ``x`` (..., cols) bf16, fp16 or fp32, rows contiguous (a matrix may have a
    row stride).  ``weight`` and ``bias``: cols values of x's type or fp32, or
    None for 1 and 0.  ``y`` has x's type and shape (or is ``out``, which must
    not overlap x); ``mean`` and ``rstd`` are fp32, one a row, as the backward
    pass takes them.
    """
    m, ld = _rows_of(x, "x")
    rows, cols = m.shape
    if cols == 0:
        raise ValueError("x must have at least one column")
    tensors = [x]
    params = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        _vector(t, name, cols, x.dtype)
        if params not in (None, t.dtype):
            raise ValueError("weight and bias must have one type")
        params = t.dtype
        tensors.append(t)
    if out is not None:
        mo, ldo = _rows_of(out, "out", x.dtype, x.shape)
        tensors.append(out)

    def body(s):
        y, o, lo = (out, mo, ldo) if out is not None else (torch.empty(x.shape, dtype=x.dtype, device=x.device),) * 2 + (cols,)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        check(_lib.lib().muon_layer_norm(
            rows, cols, m.data_ptr(), ld, _DTYPES[x.dtype], None if weight is None else weight.data_ptr(),
            None if bias is None else bias.data_ptr(), _DTYPES[params or torch.float32], eps, o.data_ptr(), lo,
            mean.data_ptr(), rstd.data_ptr(), s))
        return y, mean, rstd

    return _on_stream(body, tensors, stream)


def muon_layer_norm_backward(dy, x, mean, rstd, weight=None, bias=False, params=True, out=None, stream=None):
    """Gradients of ``muon_layer_norm``: ``(dx, dweight, dbias)``.

    ``dy`` and ``x`` of one type and shape, ``mean`` and ``rstd`` as the forward
    pass returned them.  ``dx`` has x's type and shape (or is ``out``).
    ``dweight`` has weight's type (None where ``weight`` is None or ``params`` is
    False); ``dbias`` the same type (fp32 where there is no weight), or None
    unless ``bias`` is true.
    """
    m, ld = _rows_of(x, "x")
    g, ldg = _rows_of(dy, "dy", x.dtype, x.shape)
    rows, cols = m.shape
    if cols == 0:
        raise ValueError("x must have at least one column")
    _statistic(mean, "mean", x.shape[:-1])
    _statistic(rstd, "rstd", x.shape[:-1])
    tensors = [x, dy, mean, rstd]
    if weight is not None:
        _vector(weight, "weight", cols, x.dtype)
        tensors.append(weight)
    ptype = torch.float32 if weight is None else weight.dtype
    want_w, want_b = weight is not None and params, bool(bias) and params
    if out is not None:
        mo, ldo = _rows_of(out, "out", x.dtype, x.shape)
        tensors.append(out)

    def body(s):
        lib = _lib.lib()
        dx, o, lo = (out, mo, ldo) if out is not None else (torch.empty(x.shape, dtype=x.dtype, device=x.device),) * 2 + (cols,)
        dw = torch.empty(cols, dtype=ptype, device=x.device) if want_w else None
        db = torch.empty(cols, dtype=ptype, device=x.device) if want_b else None
        need, scratch = ctypes.c_longlong(0), None
        if want_w or want_b:
            check(lib.muon_layer_norm_scratch_bytes(rows, cols, ctypes.byref(need)))
            if need.value:
                scratch = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        check(lib.muon_layer_norm_backward(
            rows, cols, g.data_ptr(), ldg, m.data_ptr(), ld, _DTYPES[x.dtype],
            None if weight is None else weight.data_ptr(), _DTYPES[ptype], mean.data_ptr(), rstd.data_ptr(), o.data_ptr(), lo,
            None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
            None if scratch is None else scratch.data_ptr(), need.value, s))
        return dx, dw, db

    return _on_stream(body, tensors, stream)


class MxMatrix:
    """A matrix in 4 bits: E2M1 values in blocks of 32 along its rows, a power-of-two scale byte for each.

    ``data``: uint8 (rows, 16 * ceil(cols / 32)), two values a byte, the even
    column in the low half.  ``scales``: uint8 (ceil(rows / 128),
    ceil(cols / 128), 32, 16); the byte of block 4 C + b of row
    128 R + 32 j + r is ``scales[R, C, r, 4 j + b]`` and stands for
    2^(byte - 127).  Places beyond the matrix hold zeros.
    """

    __slots__ = ("rows", "cols", "_buffer", "_data", "_scales", "_at")

    def __init__(self, data, scales, rows, cols):
        rows, cols = int(rows), int(cols)
        for t, name, shape in ((data, "data", self._data_shape(rows, cols)), (scales, "scales", self._scales_shape(rows, cols))):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise ValueError(f"{name} must be a uint8 tensor")
            if t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} of a {rows} x {cols} matrix must be contiguous, {shape}, got {tuple(t.shape)}")
        if scales.device != data.device:
            raise ValueError("data and scales must be on one device")
        self.rows, self.cols, self._buffer, self._data, self._scales, self._at = rows, cols, None, data, scales, None

    @staticmethod
    def _data_shape(rows, cols):
        return (rows, (cols + 31) // 32 * 16)

    @staticmethod
    def _scales_shape(rows, cols):
        return ((rows + 127) // 128, (cols + 127) // 128, 32, 16)

    @staticmethod
    def _bytes(rows, cols):
        """Bytes of data and of scales; both multiples of 16."""
        return rows * ((cols + 31) // 32 * 16), (rows + 127) // 128 * ((cols + 127) // 128) * 512

    @classmethod
    def _within(cls, buffer, at, rows, cols):
        """The matrix whose data and scales start at byte ``at`` of a uint8 buffer."""
        q = cls.__new__(cls)
        q.rows, q.cols, q._buffer, q._data, q._scales, q._at = rows, cols, buffer, None, None, at
        return q

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        """An uninitialised matrix, for ``out`` of ``muon_mx_quantize``."""
        rows, cols = int(rows), int(cols)
        return cls._within(torch.empty(sum(cls._bytes(rows, cols)), dtype=torch.uint8, device=device), 0, rows, cols)

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def data(self):
        if self._data is None:
            self._data = self._buffer[self._at: self._at + self._bytes(self.rows, self.cols)[0]].view(
                self._data_shape(self.rows, self.cols))
        return self._data

    @property
    def scales(self):
        if self._scales is None:
            d, s = self._bytes(self.rows, self.cols)
            self._scales = self._buffer[self._at + d: self._at + d + s].view(self._scales_shape(self.rows, self.cols))
        return self._scales

    @property
    def device(self):
        return (self._data if self._buffer is None else self._buffer).device

    def _tensors(self):
        return [self._buffer] if self._buffer is not None else [self._data, self._scales]

    def _pointers(self):
        if self._buffer is not None:
            p = self._buffer.data_ptr() + self._at
            return p, p + self._bytes(self.rows, self.cols)[0]
        return self._data.data_ptr(), self._scales.data_ptr()

    def __repr__(self):
        return f"MxMatrix({self.rows} x {self.cols}, {self.device})"


def _mx(q, name):
    if not isinstance(q, MxMatrix):
        raise ValueError(f"{name} must be an MxMatrix")
    if q.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA matrix")


def _array(kind, values):
    return (kind * max(1, len(values)))(*values)


def muon_mx_quantize(x, rows=True, cols=False, out=None, stream=None):
    """4-bit forms of a matrix, or of a list of matrices in one launch.

    ``x``: CUDA matrices of one type (bf16, fp16 or fp32), rows contiguous (a
    row stride is allowed).  ``rows``: the form with blocks along the rows;
    ``cols``: the form of the transpose (cols x rows), blocks along x's columns.
    Both come from one read of x.  Returns, for each matrix, the ``MxMatrix`` of
    the one form or the pair ``(row form, column form)``; ``out`` of the same
    structure is written in place of new ones.
    """
    single = isinstance(x, torch.Tensor)
    xs = [x] if single else list(x)
    if not rows and not cols:
        raise ValueError("no form is wanted: rows or cols must be true")
    if not xs:
        return []
    dtype = xs[0].dtype if isinstance(xs[0], torch.Tensor) else None
    strides = [_matrix(t, f"x[{i}]", dtype) for i, t in enumerate(xs)]
    shapes = [tuple(t.shape) for t in xs]
    given, tensors = None, list(xs)
    if out is not None:
        given = [out] if single else list(out)
        if len(given) != len(xs):
            raise ValueError("one out for each matrix is required")
        given = [tuple(g) if rows and cols else (g,) for g in given]
        for i, (g, (r, c)) in enumerate(zip(given, shapes)):
            want = ([(r, c)] if rows else []) + ([(c, r)] if cols else [])
            for q, w in zip(g, want):
                _mx(q, f"out[{i}]")
                if q.shape != w:
                    raise ValueError(f"out[{i}] must be {w}, got {q.shape}")
                tensors += q._tensors()
            if len(g) != len(want):
                raise ValueError(f"out[{i}] must hold {len(want)} forms")

    def body(s):
        forms = given
        if forms is None:
            at, places = 0, []
            for r, c in shapes:
                for a, b in ([(r, c)] if rows else []) + ([(c, r)] if cols else []):
                    places.append((at, a, b))
                    at += sum(MxMatrix._bytes(a, b))
            buffer = torch.empty(at, dtype=torch.uint8, device=xs[0].device)
            made = [MxMatrix._within(buffer, *place) for place in places]
            forms = list(zip(made[0::2], made[1::2])) if rows and cols else [(q,) for q in made]
        row = [f[0]._pointers() for f in forms] if rows else None
        col = [f[-1]._pointers() for f in forms] if cols else None
        V, L = ctypes.c_void_p, ctypes.c_int64

        def column(pairs, k):
            return None if pairs is None else _array(V, [p[k] for p in pairs])

        check(_lib.lib().muon_mx_quantize(
            len(xs), _array(V, [t.data_ptr() for t in xs]), _array(L, [v for sh in shapes for v in sh]), _array(L, strides),
            _DTYPES[dtype], column(row, 0), column(row, 1), column(col, 0), column(col, 1), s))
        if out is not None:
            return out
        got = forms if rows and cols else [f[0] for f in forms]
        return got[0] if single else got

    return _on_stream(body, tensors, stream)


def muon_mx_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values of an ``MxMatrix``, or of each of a list in one launch, as contiguous
    matrices of ``dtype``: exact in bf16 and fp32, rounded in fp16."""
    single = isinstance(q, MxMatrix)
    qs = [q] if single else list(q)
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bf16, fp16 or fp32, got {dtype}")
    if not qs:
        return []
    tensors = []
    for i, m in enumerate(qs):
        _mx(m, f"q[{i}]")
        tensors += m._tensors()

    def body(s):
        ys = [torch.empty(m.shape, dtype=dtype, device=m.device) for m in qs]
        places = [m._pointers() for m in qs]
        V = ctypes.c_void_p
        check(_lib.lib().muon_mx_dequantize(
            len(qs), _array(V, [p[0] for p in places]), _array(V, [p[1] for p in places]),
            _array(ctypes.c_int64, [v for m in qs for v in m.shape]), _array(V, [y.data_ptr() for y in ys]), _DTYPES[dtype], s))
        return ys[0] if single else ys

    return _on_stream(body, tensors, stream)


def muon_mx_product(a, b, dtype=torch.bfloat16, out=None, stream=None):
    """``a @ b.T`` of two ``MxMatrix`` (m x k and n x k): (m, n) of ``dtype``, or ``out`` (whose type it then is).

    For a linear layer y = x W^T: y = product(rows of x, rows of W), dx =
    product(rows of dy, columns of W), dW = product(columns of dy, columns of x).
    """
    _mx(a, "a")
    _mx(b, "b")
    m, k = a.shape
    n = b.rows
    if b.cols != k:
        raise ValueError(f"a and b must have equal columns, got {k} and {b.cols}")
    tensors = a._tensors() + b._tensors()
    if out is not None:
        ldo = _matrix(out, "out")
        if out.shape != (m, n):
            raise ValueError(f"out must be {(m, n)}, got {tuple(out.shape)}")
        dtype = out.dtype
        tensors.append(out)
    elif dtype not in _DTYPES:
        raise ValueError(f"dtype must be bf16, fp16 or fp32, got {dtype}")

    def body(s):
        y, ld = (out, ldo) if out is not None else (torch.empty(m, n, dtype=dtype, device=a.device), n)
        check(_lib.lib().muon_mx_product(m, n, k, *a._pointers(), *b._pointers(), y.data_ptr(), ld, _DTYPES[dtype], s))
        return y

    return _on_stream(body, tensors, stream)
