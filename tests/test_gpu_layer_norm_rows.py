"""Layer norm and its gradient on many rows: the kernels that keep the next rows on their way.

A launch takes them from 4 rows a group of threads on (592 rows times the groups of a block on 148 SMs:
16 groups forwards and 12 backwards for rows of one warp, 1 for the widest), so every shape here has more rows
than that, and a count that leaves rows over.  Bounds as in test_gpu_layer_norm.
"""
import pytest
import torch

import newton_schulz_12_b200 as nsb
from test_gpu_layer_norm import EPS, check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu

B, H, F = torch.bfloat16, torch.float16, torch.float32

#: rows, cols, type, parameters' type, columns beside the row.  Threads a row, values a thread (forwards):
CASES = [
    (38001, 64, B, F, 0), (38001, 61, F, F, 0),       # 8, 8; the second value by value
    (19001, 128, H, F, 0), (19001, 96, F, F, 4),      # 16, 8
    (9601, 200, B, B, 0), (9601, 512, F, F, 0),       # 32, 8 and 16
    (9601, 768, B, F, 0), (9601, 768, H, H, 8), (9601, 768, F, F, 0),  # 32, 24
    (9601, 1000, H, F, 0),                            # 32, 32
    (4801, 1021, F, F, 3),                            # 64, 16, value by value
    (2501, 4096, B, B, 16), (2501, 4104, F, F, 0),    # 128 and 160, 32: barriers between a row's warps
    (1301, 8192, B, F, 0), (1301, 8192, F, F, 0),     # 256, 32: two rows at a time, and one
    (2047, 5003, F, F, 7),                            # 320, 16, value by value
    (701, 9001, F, F, 0), (701, 13001, F, F, 0),      # 384, 24 and 416, 32, value by value
    (701, 16384, B, F, 0), (701, 16384, H, H, 0), (701, 16384, F, F, 0),  # 512, 32; backwards read twice
    (4501, 9304, B, B, 0), (331, 9300, B, F, 1),      # 320, 32; 64 and 6 runs of rows for the column sums
    (9601, 1021, B, F, 0), (2501, 5003, H, F, 0),     # value by value, straight into registers
    (601, 16390, B, F, 0), (601, 20000, F, F, 0),     # wider than a block holds
]


@pytest.mark.parametrize("rows,cols,dtype,params,pad", CASES)
def test_forward_and_backward(rows, cols, dtype, params, pad):
    x, dy, w, b = inputs(rows, cols, dtype, params, seed=rows + cols, pad=pad)
    y, mean, rstd = nsb.muon_layer_norm(x, w, b, eps=EPS)
    check_forward(x, w, b, y, mean, rstd)
    del y
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    again = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rows,cols,dtype", [(9601, 768, H), (1301, 8192, B), (701, 9304, F), (4801, 1021, F)])
def test_without_parameters(rows, cols, dtype, weight, bias):
    x, dy, w, b = inputs(rows, cols, dtype, F, seed=5)
    w, b = w if weight else None, b if bias else None
    y, mean, rstd = nsb.muon_layer_norm(x, w, b)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=bias)
    assert (dw is not None) == weight and (db is not None) == bias
    check_backward(dy, x, mean, rstd, w, dx, dw, db)


@pytest.mark.parametrize("cols,dtype", [(768, B), (1024, H), (8192, B), (8192, F), (5003, F), (9304, B), (16384, F)])
def test_a_row_does_not_depend_on_how_many_there_are(cols, dtype):
    """A row's bits in a call of many rows are those of a call of few."""
    rows = 9601 if cols <= 1024 else 1301
    x, dy, w, b = inputs(rows, cols, dtype, F, seed=9)
    y, mean, rstd = nsb.muon_layer_norm(x, w, b)
    dx, _, _ = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    for part in (slice(0, 1), slice(100, 117), slice(rows - 40, rows)):
        got = nsb.muon_layer_norm(x[part], w, b)
        assert all(torch.equal(p, q[part]) for p, q in zip(got, (y, mean, rstd)))
        few, _, _ = nsb.muon_layer_norm_backward(dy[part], x[part], mean[part], rstd[part], w, bias=True)
        assert torch.equal(few, dx[part])


@pytest.mark.parametrize("cols", [1032, 1027])
def test_values_behind_32_bits_of_offsets(cols):
    """The last rows of more than 2^31 values; the others are zeros, which add nothing to any sum."""
    rows, n = (1 << 21) + 77, 300
    x = torch.zeros(rows, cols, dtype=B, device="cuda")
    dy = torch.zeros(rows, cols, dtype=B, device="cuda")
    tx, tdy, w, b = inputs(n, cols, B, F, seed=11)
    x[-n:], dy[-n:] = tx, tdy
    y, mean, rstd = nsb.muon_layer_norm(x, w, b)
    check_forward(tx, w, b, y[-n:], mean[-n:], rstd[-n:])
    assert (mean[:-n] == 0).all() and (y[:-n] == b.bfloat16()).all()
    del y
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert not dx[:-n].any()
    check_backward(tdy, tx, mean[-n:], rstd[-n:], w, dx[-n:], dw, db)
