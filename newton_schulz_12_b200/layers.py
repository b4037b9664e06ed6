"""Operators around a linear layer whose weight Muon trains: layer norm with its
gradient, and 4-bit microscaled (MX) quantisation with the layer's products.

Argument marshalling over the C ABI (include/muon.h), like the rest of the
binding.  Calls run on the tensors' device, on ``stream`` or that device's
current stream, and allocate their results and scratch there.  Like the rest of
the binding they are not recorded by autograd: results never require a
gradient, whatever the inputs do, and the gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
import functools
from array import array

import torch

from . import _lib
from ._lib import MUON_BF16, MUON_FP16, MUON_FP32, check

__all__ = ["MxMatrix", "muon_layer_norm", "muon_layer_norm_backward", "muon_mx_quantize", "muon_mx_dequantize",
           "muon_mx_product"]

_DTYPES = {torch.bfloat16: MUON_BF16, torch.float32: MUON_FP32, torch.float16: MUON_FP16}


def _on_stream(body, tensors, stream):
    """body(raw stream) on the device of ``tensors``, with ``stream`` current while it allocates."""
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index:
            raise ValueError("all tensors must be on one device")
    if stream is None and index == torch.cuda.current_device():
        return body(torch.cuda.current_stream(index).cuda_stream if _raw_stream is None else _raw_stream(index))
    with torch.cuda.device(index):
        if stream is None:
            stream = torch.cuda.current_stream(index)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=index)
        elif stream.device.index != index:
            raise ValueError("stream belongs to another device than the tensors")
        if stream.cuda_stream == torch.cuda.current_stream(index).cuda_stream:
            return body(stream.cuda_stream)
        with torch.cuda.stream(stream):
            for t in tensors:  # made on another stream, as far as the allocator knows
                t.record_stream(stream)
            return body(stream.cuda_stream)


#: The current stream's handle without making a Stream object of it (1.2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _tensor(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _matrix(t, name, dtype=None):
    """Checks a 2-D CUDA matrix whose rows are contiguous; returns its rows, columns and row stride."""
    _tensor(t, name)
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise ValueError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    elif t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows > 1:
        if ld < cols:
            raise ValueError(f"{name} must not have overlapping rows")
        return rows, cols, ld
    return rows, cols, cols


def _rows_of(t, name, dtype=None, shape=None):
    """A tensor (..., cols) as a matrix of rows, without copying: its address, rows, columns and row stride."""
    _tensor(t, name)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have at least one dimension")
        try:
            t = t.view(t.shape[:-1].numel(), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name} of more than two dimensions must be viewable as rows of its last one") from None
    return (t.data_ptr(), *_matrix(t, name, dtype))


def _vector(t, name, n, dtype):
    _tensor(t, name)
    if t.dtype != dtype and t.dtype != torch.float32:
        raise ValueError(f"{name} must be fp32 or {dtype}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values")
    return t.data_ptr()


def _statistic(t, name, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise ValueError(f"{name} must be an fp32 CUDA tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {tuple(shape)}")
    return t.data_ptr()


def _like(x):
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def muon_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm over the last dimension: ``(y, mean, rstd)``.

    ``x`` (..., cols) bf16, fp16 or fp32, rows contiguous (a matrix may have a
    row stride).  ``weight`` and ``bias``: cols values of x's type or fp32, or
    None for 1 and 0.  ``y`` has x's type and shape (or is ``out``, which must
    not overlap x); ``mean`` and ``rstd`` are fp32, one a row, as the backward
    pass takes them.
    """
    xp, rows, cols, ld = _rows_of(x, "x")
    if cols == 0:
        raise ValueError("x must have at least one column")
    tensors = [x]
    wp = bp = op = None
    params = torch.float32
    if weight is not None:
        wp, params = _vector(weight, "weight", cols, x.dtype), weight.dtype
        tensors.append(weight)
    if bias is not None:
        bp = _vector(bias, "bias", cols, x.dtype)
        if weight is not None and bias.dtype != params:
            raise ValueError("weight and bias must have one type")
        params = bias.dtype
        tensors.append(bias)
    if out is not None:
        op, _, _, ldo = _rows_of(out, "out", x.dtype, x.shape)
        tensors.append(out)

    def body(s):
        y, yp, ldy = out, op, cols
        if out is None:
            y = _like(x)
            yp = y.data_ptr()
        else:
            ldy = ldo
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        if x.dim() != 2:
            mean = mean.view(x.shape[:-1])
        rstd = torch.empty_like(mean)
        check(_lib.lib().muon_layer_norm(rows, cols, xp, ld, _DTYPES[x.dtype], wp, bp, _DTYPES[params], eps, yp, ldy,
                                         mean.data_ptr(), rstd.data_ptr(), s))
        return y, mean, rstd

    return _on_stream(body, tensors, stream)


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(device, rows, cols):
    """Bytes of scratch of a backward pass on the current device, ``device``."""
    need = ctypes.c_longlong(0)
    check(_lib.lib().muon_layer_norm_scratch_bytes(rows, cols, ctypes.byref(need)))
    return need.value


def muon_layer_norm_backward(dy, x, mean, rstd, weight=None, bias=False, params=True, out=None, stream=None):
    """Gradients of ``muon_layer_norm``: ``(dx, dweight, dbias)``.

    ``dy`` and ``x`` of one type and shape, ``mean`` and ``rstd`` as the forward
    pass returned them.  ``dx`` has x's type and shape (or is ``out``).
    ``dweight`` has weight's type (None where ``weight`` is None or ``params`` is
    False); ``dbias`` the same type (fp32 where there is no weight), or None
    unless ``bias`` is true.
    """
    xp, rows, cols, ld = _rows_of(x, "x")
    gp, _, _, ldg = _rows_of(dy, "dy", x.dtype, x.shape)
    if cols == 0:
        raise ValueError("x must have at least one column")
    stats = x.shape[:-1]
    mp, rp = _statistic(mean, "mean", stats), _statistic(rstd, "rstd", stats)
    tensors = [x, dy, mean, rstd]
    wp = op = None
    ptype = torch.float32
    if weight is not None:
        wp, ptype = _vector(weight, "weight", cols, x.dtype), weight.dtype
        tensors.append(weight)
    want_w, want_b = weight is not None and params, bool(bias) and params
    if out is not None:
        op, _, _, ldo = _rows_of(out, "out", x.dtype, x.shape)
        tensors.append(out)

    def body(s):
        lib = _lib.lib()
        dx, dxp, lddx = out, op, cols
        if out is None:
            dx = _like(x)
            dxp = dx.data_ptr()
        else:
            lddx = ldo
        dw = db = scratch = dwp = dbp = sp = None
        nbytes = 0
        if want_w or want_b:
            nbytes = _scratch_bytes(x.get_device(), rows, cols)
            scratch = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
            sp = scratch.data_ptr() if nbytes else None
        if want_w:
            dw = torch.empty_like(weight)
            dwp = dw.data_ptr()
        if want_b:
            db = torch.empty(cols, dtype=ptype, device=x.device) if weight is None else torch.empty_like(weight)
            dbp = db.data_ptr()
        check(lib.muon_layer_norm_backward(rows, cols, gp, ldg, xp, ld, _DTYPES[x.dtype], wp, _DTYPES[ptype], mp, rp, dxp,
                                           lddx, dwp, dbp, sp, nbytes, s))
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
        self._check(data, "data", self._data_shape(rows, cols), rows, cols)
        self._check(scales, "scales", self._scales_shape(rows, cols), rows, cols)
        if scales.get_device() != data.get_device():
            raise ValueError("data and scales must be on one device")
        self.rows, self.cols, self._buffer, self._data, self._scales, self._at = rows, cols, None, data, scales, None

    @staticmethod
    def _check(t, name, shape, rows, cols):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8:
            raise ValueError(f"{name} must be a uint8 tensor")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} of a {rows} x {cols} matrix must be contiguous, {shape}, got {tuple(t.shape)}")

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
            return p, p + self.rows * ((self.cols + 31) >> 5) * 16
        return self._data.data_ptr(), self._scales.data_ptr()

    def __repr__(self):
        return f"MxMatrix({self.rows} x {self.cols}, {self.device})"


def _mx(q, name):
    if not isinstance(q, MxMatrix):
        raise ValueError(f"{name} must be an MxMatrix")
    if not (q._data if q._buffer is None else q._buffer).is_cuda:
        raise ValueError(f"{name} must be a CUDA matrix")


def _marshal_quantize(xs, sizes, row, col):
    """muon_mx_quantize's host arrays, made once: returns call(raw stream).  ``row`` and ``col``: the
    forms' (data, scales) addresses, or empty."""
    values = array("q", [t.data_ptr() for t in xs])
    values.extend([v for r, c, _ in sizes for v in (r, c)])
    values.extend([ld for _, _, ld in sizes])
    for pairs in (row, col):
        values.extend([d for d, _ in pairs])
        values.extend([q for _, q in pairs])
    count, n, p = len(xs), 8 * len(xs), values.buffer_info()[0]
    rd = p + 4 * n if row else None
    cd = p + (6 if row else 4) * n if col else None
    dtype, fn = _DTYPES[xs[0].dtype], _lib.lib().muon_mx_quantize

    def call(s, values=values):  # keeps the arrays
        check(fn(count, p, p + n, p + 3 * n, dtype, rd, rd and rd + n, cd, cd and cd + n, s))

    return call


def _quantize_one(x, rows, cols, stream):
    """New forms of one matrix, with few steps: a token's call is as long as its Python."""
    r, c, ld = _matrix(x, "x")

    def body(s):
        tiles = ((r + 127) >> 7) * ((c + 127) >> 7) * 512
        rdata, cdata = r * ((c + 31) >> 5) * 16, c * ((r + 31) >> 5) * 16
        second = rdata + tiles if rows else 0
        buffer = torch.empty(second + cdata + tiles if cols else second, dtype=torch.uint8, device=x.device)
        b = buffer.data_ptr()
        values = array("q", (x.data_ptr(), r, c, ld, b, b + rdata, b + second, b + second + cdata))
        v = values.buffer_info()[0]
        check(_lib.lib().muon_mx_quantize(
            1, v, v + 8, v + 24, _DTYPES[x.dtype], v + 32 if rows else None, v + 40 if rows else None,
            v + 48 if cols else None, v + 56 if cols else None, s))
        if not cols:
            return MxMatrix._within(buffer, 0, r, c)
        col = MxMatrix._within(buffer, second, c, r)
        return (MxMatrix._within(buffer, 0, r, c), col) if rows else col

    return _on_stream(body, [x], stream)


def muon_mx_quantize(x, rows=True, cols=False, out=None, stream=None):
    """4-bit forms of a matrix, or of a list of matrices in one launch.

    ``x``: CUDA matrices of one type (bf16, fp16 or fp32), rows contiguous (a
    row stride is allowed).  ``rows``: the form with blocks along the rows;
    ``cols``: the form of the transpose (cols x rows), blocks along x's columns.
    Both come from one read of x.  Returns, for each matrix, the ``MxMatrix`` of
    the one form or the pair ``(row form, column form)``; ``out`` of the same
    structure is written in place of new ones.
    """
    if not rows and not cols:
        raise ValueError("no form is wanted: rows or cols must be true")
    single = isinstance(x, torch.Tensor)
    if single and out is None:
        return _quantize_one(x, rows, cols, stream)
    xs = [x] if single else list(x)
    if not xs:
        return []
    dtype = xs[0].dtype if isinstance(xs[0], torch.Tensor) else None
    if dtype not in _DTYPES:
        raise ValueError(f"x must be bf16, fp16 or fp32 CUDA matrices, got {dtype}")
    sizes = [_matrix(t, "x", dtype) for t in xs]
    given, tensors = None, list(xs)
    if out is not None:
        given = [out] if single else list(out)
        if len(given) != len(xs):
            raise ValueError("one out for each matrix is required")
        for i, g in enumerate(given):
            if rows and cols and not isinstance(g, (tuple, list)):
                raise ValueError(f"out[{i}] must be the pair (row form, column form)")
        given = [tuple(g) if rows and cols else (g,) for g in given]
        for i, (g, (r, c, _)) in enumerate(zip(given, sizes)):
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
            # every form's data and scales in one buffer, each at a multiple of 16 bytes
            at, made, row, col = 0, [], [], []
            for r, c, _ in sizes:
                tiles = ((r + 127) >> 7) * ((c + 127) >> 7) * 512
                if rows:
                    data = r * ((c + 31) >> 5) * 16
                    made.append((at, r, c))
                    row.append((at, at + data))
                    at += data + tiles
                if cols:
                    data = c * ((r + 31) >> 5) * 16
                    made.append((at, c, r))
                    col.append((at, at + data))
                    at += data + tiles
            buffer = torch.empty(at, dtype=torch.uint8, device=xs[0].device)
            base = buffer.data_ptr()
            made = [MxMatrix._within(buffer, *place) for place in made]
            forms = list(zip(made[0::2], made[1::2])) if rows and cols else made
        else:
            base = 0
            row = [f[0]._pointers() for f in given] if rows else []
            col = [f[-1]._pointers() for f in given] if cols else []
        _marshal_quantize(xs, sizes, [(base + d, base + q) for d, q in row], [(base + d, base + q) for d, q in col])(s)
        return forms if out is None else out

    return _on_stream(body, tensors, stream)


def muon_mx_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values of an ``MxMatrix``, or of each of a list in one launch, as contiguous
    matrices of ``dtype``: exact in bf16 and fp32, rounded in fp16.

    The matrices of a list are views of one allocation.
    """
    single = isinstance(q, MxMatrix)
    qs = [q] if single else list(q)
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bf16, fp16 or fp32, got {dtype}")
    if not qs:
        return []
    tensors, last = [], None
    for m in qs:
        if not isinstance(m, MxMatrix) or m._buffer is None or m._buffer is not last:  # one check for each buffer
            _mx(m, "q")
            tensors += m._tensors()
            last = m._buffer

    def body(s):
        # one allocation, each matrix on a 16-byte boundary
        size = dtype.itemsize
        unit = 16 // size
        at, places, data, scales, shapes = 0, [], [], [], []
        for m in qs:
            r, c = m.rows, m.cols
            places.append((at, r, c))
            at += -(-r * c // unit) * unit
            d, q = m._pointers()
            data.append(d)
            scales.append(q)
            shapes += (r, c)
        flat = torch.empty(at, dtype=dtype, device=tensors[0].device)
        base, strided = flat.data_ptr(), flat.as_strided
        values = array("q", data + scales + shapes + [base + size * o for o, _, _ in places])
        n, p = 8 * len(qs), values.buffer_info()[0]
        check(_lib.lib().muon_mx_dequantize(len(qs), p, p + n, p + 2 * n, p + 4 * n, _DTYPES[dtype], s))
        ys = [strided((r, c), (c, 1), o) for o, r, c in places]
        return ys[0] if single else ys

    return _on_stream(body, tensors, stream)


def muon_mx_product(a, b, dtype=torch.bfloat16, out=None, stream=None):
    """``a @ b.T`` of two ``MxMatrix`` (m x k and n x k): (m, n) of ``dtype``, or ``out`` (whose type it then is).

    For a linear layer y = x W^T: y = product(rows of x, rows of W), dx =
    product(rows of dy, columns of W), dW = product(columns of dy, columns of x).
    """
    _mx(a, "a")
    _mx(b, "b")
    m, k, n = a.rows, a.cols, b.rows
    if b.cols != k:
        raise ValueError(f"a and b must have equal columns, got {k} and {b.cols}")
    tensors = a._tensors() + b._tensors()
    if out is not None:
        _, _, ldo = _matrix(out, "out")
        if out.shape != (m, n):
            raise ValueError(f"out must be {(m, n)}, got {tuple(out.shape)}")
        dtype = out.dtype
        tensors.append(out)
    elif dtype not in _DTYPES:
        raise ValueError(f"dtype must be bf16, fp16 or fp32, got {dtype}")

    def body(s):
        y, ld = (out, ldo) if out is not None else (torch.empty((m, n), dtype=dtype, device=a.device), n)
        check(_lib.lib().muon_mx_product(m, n, k, *a._pointers(), *b._pointers(), y.data_ptr(), ld, _DTYPES[dtype], s))
        return y

    return _on_stream(body, tensors, stream)
