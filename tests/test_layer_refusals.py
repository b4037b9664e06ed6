"""What the layer operators refuse, before any device work: the C ABI by status, the binding by ValueError."""
import ctypes

import pytest
import torch

import newton_schulz_12_b200 as nsb
from newton_schulz_12_b200 import _lib

NULL = ctypes.c_void_p(0)
X, Y, Z, V, S1, S2 = 0x10000, 0x200000, 0x400000, 0x600000, 0x610000, 0x620000


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def refused(lib, code, word, rc):
    assert rc == code, (rc, lib.muon_last_error())
    assert word in lib.muon_last_error().decode(), lib.muon_last_error()


def forward(lib, rows=4, cols=64, x=X, ldx=64, dtype=0, w=V, b=V + 512, pdtype=1, eps=1e-5, y=Y, ldy=64, mean=S1, rstd=S2):
    return lib.muon_layer_norm(rows, cols, x, ldx, dtype, w, b, pdtype, eps, y, ldy, mean, rstd, NULL)


def backward(lib, rows=4, cols=64, dy=Z, lddy=64, x=X, ldx=64, dtype=0, w=V, pdtype=1, mean=S1, rstd=S2, dx=Y, lddx=64,
             dw=None, db=None, scratch=None, nbytes=0):
    return lib.muon_layer_norm_backward(rows, cols, dy, lddy, x, ldx, dtype, w, pdtype, mean, rstd, dx, lddx, dw, db,
                                        scratch, nbytes, NULL)


def test_layer_norm_arguments(lib):
    refused(lib, -2, "rows", forward(lib, rows=-1))
    refused(lib, -2, "cols", forward(lib, cols=0))
    refused(lib, -2, "cols", forward(lib, cols=1 << 31, ldx=1 << 32, ldy=1 << 32))
    refused(lib, -1, "dtype", forward(lib, dtype=3))
    refused(lib, -1, "param_dtype", forward(lib, pdtype=2))
    refused(lib, -1, "param_dtype", forward(lib, dtype=1, pdtype=0))
    for eps in (float("nan"), float("inf"), -1e-5):
        refused(lib, -1, "eps", forward(lib, eps=eps))
    refused(lib, -2, "stride", forward(lib, ldx=63))
    refused(lib, -2, "stride", forward(lib, ldy=10))
    refused(lib, -1, "x is NULL", forward(lib, x=None))
    refused(lib, -1, "mean", forward(lib, mean=None))
    refused(lib, -1, "rstd", forward(lib, rstd=S2 + 2))
    refused(lib, -1, "aligned", forward(lib, x=X + 1))
    refused(lib, -1, "weight", forward(lib, w=V + 2))
    refused(lib, -1, "overlap", forward(lib, y=X))
    refused(lib, -1, "overlap", forward(lib, y=X + 64 * 4 * 2 - 2))
    refused(lib, -1, "overlap", forward(lib, y=V + 512 + 250 - 510))
    assert forward(lib, rows=0, x=None, y=None, mean=None, rstd=None) == 0


def test_layer_norm_backward_arguments(lib):
    refused(lib, -2, "rows", backward(lib, rows=1 << 31))
    refused(lib, -1, "dtype", backward(lib, dtype=-1))
    refused(lib, -2, "dy", backward(lib, lddy=3))
    refused(lib, -2, "dx", backward(lib, lddx=3))
    refused(lib, -1, "dy is NULL", backward(lib, dy=None))
    refused(lib, -1, "mean", backward(lib, mean=None))
    refused(lib, -1, "overlap", backward(lib, dx=Z))
    refused(lib, -1, "overlap", backward(lib, dx=X))
    refused(lib, -1, "dweight", backward(lib, dw=S1 + 1))
    assert backward(lib, rows=0, dy=None, x=None, mean=None, rstd=None, dx=None) == 0
    refused(lib, -1, "bytes", lib.muon_layer_norm_scratch_bytes(4, 4, None))


def quantize(lib, shapes, x=X, strides=None, dtype=0, row=(Y, Z), col=(None, None), count=1):
    arr = lambda p: None if p is None else _lib.ptr_array([p])  # noqa: E731
    st = None if strides is None else (ctypes.c_int64 * 1)(strides)
    return lib.muon_mx_quantize(count, arr(x), _lib.shape_array(shapes), st, dtype, arr(row[0]), arr(row[1]), arr(col[0]),
                                arr(col[1]), NULL)


def test_mx_quantize_arguments(lib):
    refused(lib, -1, "count", quantize(lib, [(4, 4)], count=-1))
    refused(lib, -1, "dtype", quantize(lib, [(4, 4)], dtype=9))
    refused(lib, -1, "come together", quantize(lib, [(4, 4)], row=(Y, None)))
    refused(lib, -1, "no form", quantize(lib, [(4, 4)], row=(None, None)))
    refused(lib, -2, "shape", quantize(lib, [(-1, 4)]))
    refused(lib, -2, "shape", quantize(lib, [(4, (1 << 30) + 1)]))
    refused(lib, -2, "stride", quantize(lib, [(4, 40)], strides=39))
    refused(lib, -1, "x is NULL", quantize(lib, [(4, 4)], x=0))
    refused(lib, -1, "aligned", quantize(lib, [(4, 4)], x=X + 1))
    refused(lib, -1, "aligned", quantize(lib, [(4, 4)], row=(Y + 8, Z)))
    refused(lib, -1, "aligned", quantize(lib, [(4, 4)], row=(Y, Z + 8)))
    refused(lib, -1, "overlap", quantize(lib, [(4, 64)], row=(X, Z)))
    assert quantize(lib, [(4, 4)], count=0) == 0


def test_mx_dequantize_arguments(lib):
    def call(shapes=((4, 64),), data=X, scales=Z, y=Y, dtype=0, count=1):
        return lib.muon_mx_dequantize(count, _lib.ptr_array([data]), _lib.ptr_array([scales]), _lib.shape_array(shapes),
                                      _lib.ptr_array([y]), dtype, NULL)
    refused(lib, -1, "count", call(count=-3))
    refused(lib, -1, "dtype", call(dtype=4))
    refused(lib, -2, "shape", call(shapes=((4, -64),)))
    refused(lib, -1, "data is NULL", call(data=0))
    refused(lib, -1, "scales", call(scales=Z + 4))
    refused(lib, -1, "y is not", call(y=Y + 1))
    refused(lib, -1, "overlap", call(y=X))
    assert call(count=0) == 0


def test_mx_product_arguments(lib):
    def call(m=4, n=8, k=64, a=X, sa=Z, b=X + 4096, sb=Z + 4096, out=Y, ldo=8, dtype=0):
        return lib.muon_mx_product(m, n, k, a, sa, b, sb, out, ldo, dtype, NULL)
    refused(lib, -2, "m ", call(m=-1))
    refused(lib, -2, "n ", call(n=1 << 31))
    refused(lib, -2, "k ", call(k=-1))
    refused(lib, -1, "dtype", call(dtype=3))
    refused(lib, -2, "stride", call(ldo=7))
    refused(lib, -1, "out is NULL", call(out=None))
    refused(lib, -1, "a_data is NULL", call(a=None))
    refused(lib, -1, "b_scales", call(sb=Z + 1))
    refused(lib, -1, "b_data", call(b=X + 8))
    refused(lib, -1, "overlap", call(out=X))
    refused(lib, -1, "overlap", call(out=X + 4096 + 32))
    refused(lib, -2, "tiles", call(m=1 << 30, n=1 << 30, ldo=1 << 30))
    assert call(m=0) == 0 and call(n=0) == 0


def test_binding_refuses():
    x = torch.zeros(4, 64)
    for call in (lambda: nsb.muon_layer_norm(x), lambda: nsb.muon_layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: nsb.muon_mx_quantize(x), lambda: nsb.muon_mx_quantize([x]), lambda: nsb.muon_mx_dequantize([x]),
                 lambda: nsb.muon_mx_product(x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="form"):
        nsb.muon_mx_quantize(x, rows=False)
    assert nsb.muon_mx_quantize([]) == [] and nsb.muon_mx_dequantize([]) == []


def test_mx_matrix_checks_its_tensors():
    u8 = torch.uint8
    q = nsb.MxMatrix(torch.zeros(5, 48, dtype=u8), torch.zeros(1, 1, 32, 16, dtype=u8), 5, 70)
    assert q.shape == (5, 70)
    for data, scales in ((torch.zeros(5, 47, dtype=u8), torch.zeros(1, 1, 32, 16, dtype=u8)),
                         (torch.zeros(5, 48), torch.zeros(1, 1, 32, 16, dtype=u8)),
                         (torch.zeros(48, 5, dtype=u8).t(), torch.zeros(1, 1, 32, 16, dtype=u8)),
                         (torch.zeros(5, 48, dtype=u8), torch.zeros(1, 2, 32, 16, dtype=u8))):
        with pytest.raises(ValueError):
            nsb.MxMatrix(data, scales, 5, 70)
    e = nsb.MxMatrix.empty(130, 129, device="cpu")
    assert e.data.shape == (130, 80) and e.scales.shape == (2, 2, 32, 16)
    with pytest.raises(ValueError, match="CUDA"):
        nsb.muon_mx_product(e, e)
    with pytest.raises(ValueError):
        nsb.muon_mx_dequantize(e)


def test_one_device_for_all_tensors():
    from newton_schulz_12_b200 import layers

    class Fake:
        def __init__(self, index):
            self.index = index

        def get_device(self):
            return self.index

    with pytest.raises(ValueError, match="one device"):
        layers._on_stream(lambda s: pytest.fail("called"), [Fake(0), Fake(1)], None)


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """The call runs with the tensors' device current, on that device's current stream."""
    import contextlib

    from newton_schulz_12_b200 import layers
    seen = []

    class Fake:
        def get_device(self):
            return 1

        def record_stream(self, s):
            seen.append("recorded")

    class Stream:
        cuda_stream = 77

    @contextlib.contextmanager
    def device(index):
        seen.append(("device", index))
        yield

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: Stream())
    assert layers._on_stream(lambda s: s, [Fake()], None) == 77
    assert seen == [("device", 1)]
