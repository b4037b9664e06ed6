"""Layer norm and its gradient against the formulas in 64 bits.

Tolerances: u = 2^-24 is the fp32 rounding.  A sum of n terms in fp32 is off by
at most d u sum|terms|, d the longest chain of additions that a term goes
through: n / 512 + 40 covers a chain within one of at least 512 threads and the
steps across them, for narrow rows (fewer threads) n <= 32 * 40.  What follows
from that is written at each check; results are then rounded once to their type
(half a step, eps / 2, relative; 2^-25 at least in fp16's subnormals).
"""
import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
TYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (1, 768), (3, 2), (7, 33), (5, 96), (130, 768), (64, 1021), (33, 1024), (19, 1280), (9, 4096),
          (11, 5003), (6, 8192), (3, 16384), (4, 16390), (2, 40000), (3000, 64), (1500, 200)]


def inputs(rows, cols, dtype, params, seed, pad=0, offset=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g) * torch.exp(0.3 * torch.randn(rows, 1, generator=g)) + offset
    dy = torch.randn(rows, cols + pad, generator=g) * 0.1
    w = 1 + 0.2 * torch.randn(cols, generator=g)
    b = 0.1 * torch.randn(cols, generator=g)
    return x.to(dtype).cuda()[:, :cols], dy.to(dtype).cuda()[:, :cols], w.to(params).cuda(), b.to(params).cuda()


def half_step(ref, dtype):
    if dtype == torch.float32:
        return U * ref.abs()
    return torch.finfo(dtype).eps / 2 * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def within(got, ref, tol):
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


def check_forward(x, w, b, y, mean, rstd, eps=EPS):
    n = x.shape[-1]
    X = x.double()
    m = X.mean(-1, keepdim=True)
    var = ((X - m) ** 2).mean(-1, keepdim=True)
    r = (var + eps) ** -0.5
    d = n / 512 + 40
    dm = (d + 1) * U * X.abs().mean(-1, keepdim=True)         # of the mean
    within(mean.unsqueeze(-1), m, dm + 1e-300)
    # centred values are off by dm and a rounding; their squares' mean by dm^2 (the rest cancels
    # in exact arithmetic: the mean of x - m is 0), the roundings, and 2 dm u |x - m| sums
    spread = (X - m).abs().mean(-1, keepdim=True)
    dvar = dm ** 2 + (d + 6) * U * var + 4 * dm * U * spread * d
    dr = r * (0.5 * dvar * r ** 2 * 1.01 + 4 * U)
    within(rstd.unsqueeze(-1), r, dr)
    xhat = (X - m) * r
    W = w.double() if w is not None else torch.ones(n, dtype=torch.float64, device=x.device)
    B = b.double() if b is not None else torch.zeros(n, dtype=torch.float64, device=x.device)
    ref = xhat * W + B
    tol = W.abs() * ((X - m).abs() * dr + r * dm * 1.01 + 4 * U * xhat.abs()) + 2 * U * (ref.abs() + B.abs())
    within(y, ref, tol + half_step(ref, x.dtype) * 1.001 + 1e-300)


def check_backward(dy, x, mean, rstd, w, dx, dw, db):
    rows, n = x.shape
    G, X = dy.double(), x.double()
    R = rstd.double()[:, None]
    xhat = (X - mean.double()[:, None]) * R
    W = w.double() if w is not None else torch.ones(n, dtype=torch.float64, device=x.device)
    g = G * W
    s, q = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    ref = R * (g - s - xhat * q)
    d = n / 512 + 40
    ds = (d + 4) * U * g.abs().mean(1, keepdim=True)
    dq = (d + 8) * U * (g * xhat).abs().mean(1, keepdim=True)
    tol = R * (ds + xhat.abs() * dq + 6 * U * (g.abs() + s.abs() + (xhat * q).abs()))
    within(dx, ref, tol + half_step(ref, x.dtype) * 1.001 + 1e-300)
    D = rows / 64 + 128  # chains over the rows: runs of at most rows / 64 rows, then the partial sums
    if dw is not None:
        within(dw, (G * xhat).sum(0), (D + 4) * U * (G * xhat).abs().sum(0) + half_step((G * xhat).sum(0), dw.dtype) * 1.001)
    if db is not None:
        within(db, G.sum(0), D * U * G.abs().sum(0) + half_step(G.sum(0), db.dtype) * 1.001)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,params", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                          (torch.float16, torch.float32), (torch.float16, torch.float16),
                                          (torch.float32, torch.float32)])
def test_forward_and_backward(shape, dtype, params):
    x, dy, w, b = inputs(*shape, dtype, params, seed=shape[0] + shape[1])
    y, mean, rstd = nsb.muon_layer_norm(x, w, b, eps=EPS)
    assert y.dtype == dtype and y.shape == x.shape
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert dw.dtype == params and db.dtype == params
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    again = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("cols", [96, 1021, 9000])
def test_without_parameters(weight, bias, cols):
    x, dy, w, b = inputs(50, cols, torch.bfloat16, torch.float32, seed=3)
    w, b = w if weight else None, b if bias else None
    y, mean, rstd = nsb.muon_layer_norm(x, w, b)
    check_forward(x, w, b, y, mean, rstd)
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=bias)
    assert (dw is not None) == weight and (db is not None) == bias
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    only, none, nil = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=bias, params=False)
    assert torch.equal(only, dx) and none is None and nil is None


@pytest.mark.parametrize("pad", [1, 7, 8, 16])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [64, 768, 2000])
def test_strided(pad, dtype, cols):
    x, dy, w, b = inputs(70, cols, dtype, torch.float32, seed=4, pad=pad)
    wide = torch.full((70, cols + pad), 7.0, dtype=dtype, device="cuda")
    y, mean, rstd = nsb.muon_layer_norm(x, w, b, out=wide[:, :cols])
    check_forward(x, w, b, y, mean, rstd)
    assert (wide[:, cols:] == 7.0).all()
    wide = torch.full((70, cols + pad), 7.0, dtype=dtype, device="cuda")
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True, out=wide[:, :cols])
    check_backward(dy, x, mean, rstd, w, dx, dw, db)
    assert (wide[:, cols:] == 7.0).all()


def test_many_dimensions_and_no_rows():
    x, dy, w, b = inputs(24, 768, torch.bfloat16, torch.float32, seed=5)
    y, mean, rstd = nsb.muon_layer_norm(x, w, b)
    y3, m3, r3 = nsb.muon_layer_norm(x.contiguous().view(2, 3, 4, 768), w, b)
    assert y3.shape == (2, 3, 4, 768) and m3.shape == (2, 3, 4)
    assert torch.equal(y3.view(24, 768), y) and torch.equal(m3.view(24), mean) and torch.equal(r3.view(24), rstd)
    one, m1, r1 = nsb.muon_layer_norm(x[0], w, b)
    assert one.shape == (768,) and m1.shape == () and torch.equal(one, y[0])
    none = x[:0]
    y0, m0, r0 = nsb.muon_layer_norm(none, w, b)
    assert y0.shape == (0, 768) and m0.shape == (0,)
    dx, dw, db = nsb.muon_layer_norm_backward(none, none, m0, r0, w, bias=True)
    assert dx.shape == (0, 768) and (dw == 0).all() and (db == 0).all()


def test_large_offset_and_constant_rows():
    """An offset of 4096 spreads leaves the variance its digits; a constant row is 0 times 1/sqrt(eps)."""
    x, _, w, b = inputs(40, 768, torch.float32, torch.float32, seed=6, offset=4096.0)
    check_forward(x, w, b, *nsb.muon_layer_norm(x, w, b))
    flat = torch.full((5, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = nsb.muon_layer_norm(flat)
    assert (y == 0).all() and (mean == 3).all()
    within(rstd, torch.full_like(rstd, EPS).double() ** -0.5, torch.full_like(rstd, 4 * U * EPS ** -0.5).double())


def test_nan_and_infinity_stay_in_their_row():
    x, _, w, b = inputs(30, 500, torch.float32, torch.float32, seed=7)
    x = x.contiguous()
    clean = nsb.muon_layer_norm(x, w, b)[0]
    x[3, 7], x[11, 0] = float("nan"), float("inf")
    y = nsb.muon_layer_norm(x, w, b)[0]
    assert y[3].isnan().all() and y[11].isnan().all()
    keep = [r for r in range(30) if r not in (3, 11)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("cols", [5, 40])
def test_gradient_against_differences(cols):
    """Central differences of the forward formula in 64 bits against the kernel's gradient."""
    x, dy, w, b = inputs(4, cols, torch.float32, torch.float32, seed=8, offset=0.3)
    _, mean, rstd = nsb.muon_layer_norm(x, w, b)
    dx, dw, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, w, bias=True)

    def loss(X, W, B):
        m = X.mean(1, keepdim=True)
        v = ((X - m) ** 2).mean(1, keepdim=True)
        return (((X - m) / torch.sqrt(v + EPS) * W + B) * dy.double()).sum()

    args = [t.double() for t in (x, w, b)]
    h = 1e-5
    for k, got in enumerate((dx, dw, db)):
        flat = args[k].reshape(-1)
        for i in range(flat.numel()):
            sides = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[i] += sign * h
                sides.append(loss(*[moved.view(args[k].shape) if j == k else args[j] for j in range(3)]))
            diff = (sides[0] - sides[1]) / (2 * h)
            # truncation h^2 times a third derivative of order 10 at most; fp32 of the kernel
            assert abs(float(diff) - float(got.reshape(-1)[i])) <= 1e-8 + 2e-5 * float(got.abs().max())
