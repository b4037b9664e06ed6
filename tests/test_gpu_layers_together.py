"""The layer operators as a training step uses them: together, captured, on streams, at large offsets.

The step of one hidden layer: h = layer_norm(x), y = Q(h) Q(W)^T, then from dy the gradients dh, dW (which
muon_step takes), dx, dw, db, and the new weight's 4-bit forms.  Each stage is checked against its plain
form on the values that the stage before it really gave.
"""
import functools
import threading

import numpy as np
import pytest
import torch

import mxref
import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@functools.lru_cache(maxsize=None)
def streams():
    """Three streams for all tests here (torch hands out the same 32 in turn)."""
    return [torch.cuda.Stream() for _ in range(3)]


def host(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def make(m, n, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(m, k, generator=g) * 2 + 0.5).bfloat16().cuda()
    dy = (torch.randn(m, n, generator=g) * 1e-3).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(k, generator=g)).cuda()
    b = (0.1 * torch.randn(k, generator=g)).cuda()
    W = (0.02 * torch.randn(n, k, generator=g)).cuda()
    return x, dy, w, b, W


def step(x, dy, w, b, Wr, Wc, stream=None):
    """Forward and backward pass of the layer; all that it computes."""
    h, mean, rstd = nsb.muon_layer_norm(x, w, b, stream=stream)
    hr, hc = nsb.muon_mx_quantize(h, rows=True, cols=True, stream=stream)
    y = nsb.muon_mx_product(hr, Wr, stream=stream)
    dyr, dyc = nsb.muon_mx_quantize(dy, rows=True, cols=True, stream=stream)
    dh = nsb.muon_mx_product(dyr, Wc, stream=stream)
    dW = nsb.muon_mx_product(dyc, hc, stream=stream)
    dx, dw, db = nsb.muon_layer_norm_backward(dh, x, mean, rstd, w, bias=True, stream=stream)
    return h, mean, rstd, y, dh, dW, dx, dw, db


def q64(x):
    """The values of Q(x) along the rows, in fp64."""
    return mxref.values(*mxref.quantize(x), x.shape[1])


def near(got, a, b):
    """got = round(a b^T): the sums as in test_gpu_mx.check_product, then one rounding to bf16."""
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2 * (-(-a.shape[1] // 32) + 1) * 2.0 ** -23 * mag
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(host(got) - want) <= tol).all()


@pytest.mark.parametrize("m,n,k", [(1, 96, 64), (50, 256, 128), (333, 520, 264)])
def test_training_step_of_a_layer(m, n, k):
    x, dy, w, b, W = make(m, n, k)
    Wr, Wc = nsb.muon_mx_quantize(W, rows=True, cols=True)
    h, mean, rstd, y, dh, dW, dx, dw, db = step(x, dy, w, b, Wr, Wc)
    H, DY, W64 = host(h), host(dy), host(W)
    near(y, q64(H), q64(W64))
    near(dh, q64(DY), q64(W64.T))
    near(dW, q64(DY.T), q64(H.T))
    # the norm and its gradient on what they were given (their own tests hold them tighter)
    X = x.double()
    mu = X.mean(1, keepdim=True)
    r = (((X - mu) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
    xhat = (X - mu) * r
    ref = xhat * w.double() + b.double()
    assert ((h.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 400 * U * (1 + ref.abs())).all()
    G = dh.double() * w.double()
    rdx = r * (G - G.mean(1, keepdim=True) - xhat * (G * xhat).mean(1, keepdim=True))
    size = r * (G.abs() + G.abs().mean(1, keepdim=True) + xhat.abs() * (G * xhat).abs().mean(1, keepdim=True))
    assert ((dx.double() - rdx).abs() <= 2.0 ** -8 * rdx.abs() + 400 * U * size).all()
    assert ((db.double() - dh.double().sum(0)).abs() <= 400 * U * dh.double().abs().sum(0)).all()
    assert ((dw.double() - (dh.double() * xhat).sum(0)).abs() <= 400 * U * (dh.double() * xhat).abs().sum(0)).all()
    # the gradient goes to the step as it is, and the plan leaves the new weight's forms
    V, M = W.clone(), torch.zeros_like(W)
    plan = nsb.MuonStepPlan([V], [dW], [M], mx_forms=True)
    assert torch.equal(plan.mx_forms[0][0].data, Wr.data) and torch.equal(plan.mx_forms[0][1].scales, Wc.scales)
    plan()
    W2, M2 = W.clone(), torch.zeros_like(W)
    nsb.muon_step([W2], [dW], [M2])
    assert torch.equal(V, W2) and not torch.equal(V, W)
    for got, want in zip(plan.mx_forms[0], nsb.muon_mx_quantize(V, rows=True, cols=True)):
        assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)
    assert nsb.muon_get_status() == 0


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_from_the_first_call_on_a_stream():
    """A graph recorded on a stream that the library has not seen, replayed on new values."""
    x, dy, w, b, W = make(300, 256, 384, seed=1)
    Wr, Wc = nsb.muon_mx_quantize(W, rows=True, cols=True)
    want = step(x, dy, w, b, Wr, Wc)
    x2, dy2, *_ = make(300, 256, 384, seed=2)
    want2 = step(x2, dy2, w, b, Wr, Wc)
    xs, ds = x.clone(), dy.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step(xs, ds, w, b, Wr, Wc)
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)
    xs.copy_(x2), ds.copy_(dy2)
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want2)
    assert nsb.muon_get_status() == 0 and nsb.muon_get_status(s) == 0


def test_two_graphs_replayed_side_by_side():
    """Two captures on one stream share no scratch: replayed at once on two streams they give what each gives alone."""
    sets = [make(700, 384, 512, seed=s) for s in (3, 4)]
    forms = [nsb.muon_mx_quantize(W, rows=True, cols=True) for *_, W in sets]
    want = [step(*p[:4], *f) for p, f in zip(sets, forms)]
    torch.cuda.synchronize()
    s, graphs, got = streams()[0], [], []
    for p, f in zip(sets, forms):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(step(*p[:4], *f))
        graphs.append(g)
    for _ in range(20):
        for g, st in zip(graphs, streams()[1:]):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_plan_with_forms_captured():
    g = torch.Generator().manual_seed(5)
    shapes = [(256, 256), (128, 384), (384, 128)]
    W = [(0.02 * torch.randn(s, generator=g)).cuda() for s in shapes]
    G = [(1e-2 * torch.randn(s, generator=g)).bfloat16().cuda() for s in shapes]
    M = [torch.zeros(s, device="cuda") for s in shapes]
    W2, M2 = [w.clone() for w in W], [m.clone() for m in M]
    plan = nsb.MuonStepPlan(W, G, M, mx_forms=True)
    plan.capture(streams()[0])
    plan.replay()
    for _ in range(2):
        nsb.muon_step(W2, G, M2)
    torch.cuda.synchronize()
    for w, v, pair in zip(W, W2, plan.mx_forms):
        assert torch.equal(w, v)
        for got, want in zip(pair, nsb.muon_mx_quantize(v, rows=True, cols=True)):
            assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)


def test_given_streams_and_threads():
    """Calls on given streams, from several threads at once, give what they give alone."""
    sets = [make(400 + 37 * i, 256, 512, seed=10 + i) for i in range(4)]
    forms = [nsb.muon_mx_quantize(W, rows=True, cols=True) for *_, W in sets]
    want = [step(*p[:4], *f) for p, f in zip(sets, forms)]
    torch.cuda.synchronize()
    got, wrong = [None] * 4, []
    streams()

    def work(i):
        try:
            s = streams()[i % 3]
            for _ in range(10):
                got[i] = step(*sets[i][:4], *forms[i], stream=s if i % 2 else s.cuda_stream)
            s.synchronize()
        except Exception as e:  # pragma: no cover
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not wrong
    for i in range(4):
        assert same(got[i], want[i])


def test_the_default_stream_by_its_handle():
    x, dy, w, b, W = make(100, 128, 256, seed=20)
    Wr, Wc = nsb.muon_mx_quantize(W, rows=True, cols=True)
    want = step(x, dy, w, b, Wr, Wc)
    torch.cuda.synchronize()
    with torch.cuda.stream(streams()[0]):
        got = step(x, dy, w, b, Wr, Wc, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert same(got, want)


def test_more_than_32_bits_of_offsets():
    """Matrices of more than 2^31 values: the last rows as by themselves."""
    rows, cols = (1 << 21) + 77, 1032
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(300, cols, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x.zero_()
    x[-300:] = tail
    w = torch.linspace(0.5, 1.5, cols, device="cuda")
    y, mean, rstd = nsb.muon_layer_norm(x, w)
    ty, tm, tr = nsb.muon_layer_norm(tail, w)
    # (the tail alone takes another kernel: sums in another order, one bf16 step)
    assert ((y[-300:].double() - ty.double()).abs() <= 2.0 ** -7 * ty.double().abs() + 1e-6).all()
    assert ((mean[-300:] - tm).abs() <= 1e-6).all() and (y[:-300] == 0).all()
    del y
    dx, dw, db = nsb.muon_layer_norm_backward(x, x, mean, rstd, w, bias=True)
    td = tail.double()
    rdb = td.sum(0)
    assert ((db.double() - rdb).abs() <= (rows / 64 + 128) * U * td.abs().sum(0)).all()
    assert (dx[:-300] == 0).all() and dx[-300:].abs().max() > 0
    del dx
    row, col = nsb.muon_mx_quantize(x, rows=True, cols=True)
    trow = nsb.muon_mx_quantize(tail)
    assert torch.equal(row.data[-300:], trow.data)
    assert not row.data[:-300].any()
    first = (rows - 300) // 32 * 32  # the columns' blocks of 32 rows from here on
    tcol = nsb.muon_mx_quantize(x[first:].contiguous(), rows=False, cols=True)
    assert torch.equal(col.data[:, first // 2:], tcol.data)
    back = nsb.muon_mx_dequantize(row)
    assert torch.equal(back[-300:], nsb.muon_mx_dequantize(trow)) and not back[:-300].any()


def test_product_of_more_than_32_bits():
    m, n, k = 70000, 31000, 64  # 2.17e9 results
    a, b = nsb.muon_mx_quantize([torch.zeros(m, k, device="cuda").index_fill_(0, torch.tensor([0, m - 1], device="cuda"), 1.0),
                                 torch.ones(n, k, device="cuda")])
    c = nsb.muon_mx_product(a, b)
    assert (c[0] == k).all() and (c[-1] == k).all() and c[1:-1].count_nonzero() == 0


@pytest.mark.parametrize("m,n,k", [(2100, 2300, 1000), (300, 200, 600), (100, 60, 600)])
def test_a_wait_that_runs_out_is_reported(m, n, k):
    """A withheld operand copy: the status word tells, the next call is right (pairs of CTAs, and one CTA)."""
    a, b = nsb.muon_mx_quantize([torch.randn(m, k).cuda(), torch.randn(n, k).cuda()])
    want = nsb.muon_mx_product(a, b)
    assert nsb.muon_get_status() == 0
    nsb.muon_set_wait_timeout_ms(200)
    try:
        nsb.muon_set_fault_injection(1)
        nsb.muon_mx_product(a, b)
        assert nsb.muon_get_status() == -5
        assert nsb.muon_get_status() == 0
    finally:
        nsb.muon_set_fault_injection(0)
        nsb.muon_set_wait_timeout_ms(2000)
    assert torch.equal(nsb.muon_mx_product(a, b), want)
    assert nsb.muon_get_status() == 0


def test_a_wait_that_runs_out_in_a_graph_is_reported():
    """The graph outlives the stream's own status word; any stream reports it, once."""
    a, b = nsb.muon_mx_quantize([torch.randn(300, 600).cuda(), torch.randn(200, 600).cuda()])
    want = nsb.muon_mx_product(a, b)
    torch.cuda.synchronize()
    nsb.muon_set_wait_timeout_ms(200)
    graph = torch.cuda.CUDAGraph()
    try:
        nsb.muon_set_fault_injection(1)
        with torch.cuda.graph(graph, stream=streams()[1]):
            nsb.muon_mx_product(a, b)
    finally:
        nsb.muon_set_fault_injection(0)
        nsb.muon_set_wait_timeout_ms(2000)
    nsb.muon_release()
    assert nsb.muon_get_status() == 0
    graph.replay()
    assert nsb.muon_get_status() == -5
    assert nsb.muon_get_status(streams()[1]) == 0 and nsb.muon_get_status() == 0
    assert torch.equal(nsb.muon_mx_product(a, b), want)
    assert nsb.muon_get_status() == 0


def test_kernels_are_timed():
    x, dy, w, b, W = make(64, 128, 256)
    Wr, Wc = nsb.muon_mx_quantize(W, rows=True, cols=True)
    nsb.muon_profile_begin()
    step(x, dy, w, b, Wr, Wc)
    nsb.muon_mx_dequantize(Wr)
    got = nsb.muon_profile_end()
    counts = {k: got[k][1] for k in ("layer_norm", "layer_norm_grad", "mx_quantize", "mx_dequantize", "mx_product")}
    assert counts == {"layer_norm": 1, "layer_norm_grad": 1, "mx_quantize": 2, "mx_dequantize": 1, "mx_product": 3}
