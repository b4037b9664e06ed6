"""What a layer operator writes shares no byte with anything else of the call: refused by the C ABI before any device work."""
import pytest

from newton_schulz_12_b200 import _lib
from test_layer_refusals import NULL, S1, S2, V, X, Y, Z, backward, forward, lib, refused  # noqa: F401


@pytest.mark.parametrize("names,over", [
    ("y x", dict(y=X + 510)), ("y weight", dict(y=V - 256)), ("y bias", dict(y=V + 512)),
    ("mean x", dict(mean=X + 508)), ("rstd bias", dict(rstd=V + 764)),
    ("y rstd", dict(rstd=Y)), ("mean rstd", dict(mean=S2 + 12)), ("mean rstd", dict(mean=S1, rstd=S1)),
])
def test_layer_norm(lib, names, over):  # noqa: F811
    refused(lib, -1, "must not overlap", forward(lib, **over))
    assert sorted(lib.muon_last_error().decode().split(" must not overlap ")) == sorted(names.split())


@pytest.mark.parametrize("over", [dict(dx=Z + 510), dict(dx=X - 510), dict(dx=V), dict(mean=Y), dict(rstd=Y + 508), dict(dw=X), dict(db=Z + 4),
                                  dict(dw=V + 252), dict(dw=S1 + 12), dict(db=Y), dict(dw=V + 1024, db=V + 1276)])
def test_layer_norm_backward(lib, over):  # noqa: F811
    refused(lib, -1, "overlap", backward(lib, **over))


def quantize(lib, xs, shapes, row=None, col=None):  # noqa: F811
    arr = lambda p: None if p is None else _lib.ptr_array(p)  # noqa: E731
    row, col = row or (None, None), col or (None, None)
    return lib.muon_mx_quantize(len(xs), arr(xs), _lib.shape_array(shapes), None, 0, arr(row[0]), arr(row[1]), arr(col[0]),
                                arr(col[1]), NULL)


def test_mx_quantize(lib):  # noqa: F811
    two = [(4, 64), (4, 64)]  # 512 bytes, forms of 128 (rows) and 1024 (columns), scales of 512
    ok = dict(row=([Y, Y + 4096], [Z, Z + 4096]), col=([V, V + 4096], [S1, S1 + 4096]))
    for form, part, i in (("row", 0, 0), ("row", 1, 0), ("row", 0, 1), ("row", 1, 1), ("col", 0, 1), ("col", 1, 0)):
        for at in (X + 496, X + 4096 + 496, Z + 4096 + 496, V + 1008, S1 + 496):  # the ends of both x, a scale tile, a column form
            if 0 <= at - ok[form][part][i] < 512:
                continue  # itself
            over = {k: tuple(list(p) for p in v) for k, v in ok.items()}
            over[form][part][i] = at
            refused(lib, -1, "overlap", quantize(lib, [X, X + 4096], two, **over))
    # the same form for two matrices
    refused(lib, -1, "overlap", quantize(lib, [X, X + 4096], two, row=([Y, Y], [Z, Z + 4096])))


def test_mx_dequantize(lib):  # noqa: F811
    def call(y, data=(X, X + 4096), scales=(Z, Z + 4096)):
        return lib.muon_mx_dequantize(2, _lib.ptr_array(data), _lib.ptr_array(scales), _lib.shape_array([(4, 64), (4, 64)]),
                                      _lib.ptr_array(y), 0, NULL)
    for y in ((Z + 510, Y), (Z + 4096, Y), (Y, X + 126), (X + 4096 + 126, Y), (Y, Y), (Y, Y + 510)):
        refused(lib, -1, "overlap", call(y))


def test_mx_product(lib):  # noqa: F811
    def call(out, a=X, sa=Z, b=X + 4096, sb=Z + 4096):
        return lib.muon_mx_product(4, 8, 64, a, sa, b, sb, out, 8, 0, NULL)
    for out in (X + 126, X + 4096 + 254, Z, Z + 510, Z - 62, Z + 4096 + 510):
        refused(lib, -1, "overlap", call(out))
