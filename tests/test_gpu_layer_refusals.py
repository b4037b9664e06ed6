"""Refusals of the layer operators that need CUDA tensors to get as far; nothing is launched by any of them."""
import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu


def test_quantize_out_of_the_wrong_structure():
    x = torch.zeros(40, 70, device="cuda")
    row, col = nsb.MxMatrix.empty(40, 70), nsb.MxMatrix.empty(70, 40)
    for args, out in ((dict(cols=True), row), (dict(cols=True), (row,)), (dict(cols=True), (col, row)), (dict(cols=True), (row, x)),
                      (dict(), (row,)), (dict(), col), (dict(rows=False, cols=True), row)):
        with pytest.raises(ValueError, match="out"):
            nsb.muon_mx_quantize(x, out=out, **args)
    with pytest.raises(ValueError, match="one out"):
        nsb.muon_mx_quantize([x, x], out=[row])
    with pytest.raises(ValueError, match="out"):
        nsb.muon_mx_quantize([x], cols=True, out=[row])


def test_what_is_written_twice_or_read():
    x = torch.zeros(2, 40, 64, device="cuda")
    q = nsb.MxMatrix.empty(40, 64)
    with pytest.raises(nsb.MuonError, match="overlap"):
        nsb.muon_mx_quantize([x[0], x[1]], out=[q, q])
    with pytest.raises(nsb.MuonError, match="overlap"):
        nsb.muon_layer_norm(x[0], out=x[0])
    with pytest.raises(nsb.MuonError, match="overlap"):
        nsb.muon_layer_norm(x[0], bias=x[1, 0], out=x[1])
    buffer = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    held = nsb.MxMatrix(buffer[:128].view(4, 32), buffer[512:1024].view(1, 1, 32, 16), 4, 64)
    with pytest.raises(nsb.MuonError, match="overlap"):
        nsb.muon_mx_product(held, held, out=buffer[992:1024].view(torch.bfloat16).view(4, 4))
    y = nsb.muon_mx_product(held, held, out=buffer[1024:1056].view(torch.bfloat16).view(4, 4))
    assert (y == 0).all() and nsb.muon_get_status() == 0


@pytest.mark.parametrize("call", ["norm", "grad", "quantize", "product"])
def test_strides(call):
    t = torch.zeros(64, 64, device="cuda")
    q = nsb.muon_mx_quantize(t)
    m = torch.zeros(64, device="cuda")
    for bad in (t.t(), t[:1].expand(64, 64), t[:, ::2]):
        with pytest.raises(ValueError, match="rows"):
            if call == "norm":
                nsb.muon_layer_norm(bad)
            elif call == "grad":
                nsb.muon_layer_norm_backward(bad, torch.zeros(bad.shape, device="cuda"), m, m)
            elif call == "quantize":
                nsb.muon_mx_quantize(bad)
            else:
                nsb.muon_mx_product(q, q, out=bad)
