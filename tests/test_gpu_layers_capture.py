"""Layer operators beside another stream's capture."""
import ctypes

import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu


def test_first_product_on_a_stream_while_another_one_captures():
    """It allocates its stream's status word, which must neither fail nor end the capture (torch's default
    mode forbids allocations to every thread)."""
    g = torch.Generator().manual_seed(0)
    a, b = nsb.muon_mx_quantize([torch.randn(300, 600, generator=g).cuda(), torch.randn(200, 600, generator=g).cuda()])
    want = nsb.muon_mx_product(a, b)
    captured, direct = torch.zeros_like(want), torch.zeros_like(want)
    torch.cuda.synchronize()
    nsb.muon_release()  # no stream has a word now
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        nsb.muon_mx_product(a, b, out=captured)
        nsb.muon_mx_product(a, b, out=direct, stream=other)
    other.synchronize()
    assert torch.equal(direct, want) and not captured.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want)
    assert nsb.muon_get_status() == 0 and nsb.muon_get_status(other) == 0


def test_memory_of_the_layer_operators():
    """A status word of 256 bytes a stream with products, nothing else, and nothing after a release."""
    from newton_schulz_12_b200 import _lib

    def held(stream):
        n = ctypes.c_longlong(-1)
        assert _lib.lib().muon_workspace_bytes(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(n)) == 0
        return n.value

    nsb.muon_release()
    s = torch.cuda.Stream()
    x = torch.randn(40, 96).cuda()
    torch.cuda.synchronize()
    y, mean, rstd = nsb.muon_layer_norm(x, stream=s)
    nsb.muon_layer_norm_backward(x, x, mean, rstd, bias=True, stream=s)
    q = nsb.muon_mx_quantize(x, stream=s)
    nsb.muon_mx_dequantize(q, stream=s)
    assert held(s) == 0
    nsb.muon_mx_product(q, q, stream=s)
    assert held(s) == 256
    s.synchronize()
    nsb.muon_release()
    assert held(s) == 0


def test_a_captured_wait_that_runs_out_is_reported_once_whoever_asks_meanwhile():
    g = torch.Generator().manual_seed(1)
    a, b = nsb.muon_mx_quantize([torch.randn(300, 200, generator=g).cuda(), torch.randn(200, 200, generator=g).cuda()])
    want = nsb.muon_mx_product(a, b)
    s, asking = torch.cuda.Stream(), torch.cuda.Stream()
    graphs = []
    nsb.muon_set_wait_timeout_ms(50)
    try:
        for _ in range(2):
            nsb.muon_set_fault_injection(1)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                nsb.muon_mx_product(a, b)
    finally:
        nsb.muon_set_fault_injection(0)
        nsb.muon_set_wait_timeout_ms(2000)
    assert nsb.muon_get_status(asking) == 0
    for graph in graphs:
        reports = 0
        with torch.cuda.stream(s):
            graph.replay()
            done = torch.cuda.Event()
            done.record()
        while not done.query():
            reports += nsb.muon_get_status(asking) == -5
        reports += nsb.muon_get_status(asking) == -5
        assert reports == 1
        assert nsb.muon_get_status(s) == 0
    assert torch.equal(nsb.muon_mx_product(a, b), want)
