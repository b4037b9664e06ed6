"""4-bit microscaled quantisation and products against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

import newton_schulz_12_b200 as nsb
import mxref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (1, 31), (2, 32), (33, 65), (31, 300), (128, 128), (129, 257), (257, 129), (300, 96), (513, 640)]


def normal(shape, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(shape[0], 1, generator=g))
    return x.to(dtype)


def host(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def check_form(q, x):
    """q holds exactly the 4-bit form of the fp64 matrix x, zeros beyond it."""
    rows, cols = x.shape
    assert q.shape == (rows, cols)
    data, scales = q.data.cpu().numpy(), q.scales.cpu().numpy()
    code, byte = mxref.unpack(data, scales, rows, cols)
    want_code, want_byte = mxref.quantize(x)
    assert np.array_equal(byte, want_byte)
    ok = want_byte != 255
    assert mxref.same_codes(code[ok], want_code[ok])
    pad = code.reshape(rows, -1)[:, cols:]
    assert not pad[np.repeat(ok[:, -1:], pad.shape[1], 1)].any() if pad.size else True
    used = np.zeros(scales.shape, dtype=bool)
    r, b = np.meshgrid(np.arange(rows), np.arange(byte.shape[1]), indexing="ij")
    used[r // 128, b // 4, r % 32, (r % 128) // 32 * 4 + b % 4] = True
    assert not scales[~used].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_both_forms(shape, dtype):
    x = normal(shape, 1 + shape[0] + shape[1], dtype).cuda()
    row, col = nsb.muon_mx_quantize(x, rows=True, cols=True)
    check_form(row, host(x))
    check_form(col, host(x).T)
    # each form alone is the same
    only = nsb.muon_mx_quantize(x, rows=False, cols=True)
    assert torch.equal(only.data, col.data) and torch.equal(only.scales, col.scales)
    alone = nsb.muon_mx_quantize(x)
    assert torch.equal(alone.data, row.data) and torch.equal(alone.scales, row.scales)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 8, 13])
def test_quantize_strided(pad, dtype):
    wide = normal((200, 150 + pad), 5, dtype).cuda()
    x = wide[:, pad:] if pad != 8 else wide[:, :150]
    row, col = nsb.muon_mx_quantize(x, rows=True, cols=True)
    check_form(row, host(x))
    check_form(col, host(x).T)


def test_quantize_special_values():
    x = torch.zeros(40, 96)
    x[1] = torch.arange(96) - 48.0
    x[2, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)     # ties, scale 1
    x[3, :32] = -x[2, :32]
    x[4, 3], x[4, 40] = float("inf"), 1.0
    x[5, 70] = float("nan")
    x[6] = 1e-45 * (1 + torch.arange(96) % 3)                                       # subnormals
    x[7] = 3.4e38
    x[8, ::2], x[8, 1::2] = 1.17549435e-38, -2.0e-39
    x[9, 0], x[9, 1:32] = 7.99, 5.01                                                # held at 6
    x[10, :32] = -0.0
    x[11, 0], x[11, 1:32] = 2.0 ** -125, 2.0 ** -128
    x = x.cuda()
    row, col = nsb.muon_mx_quantize(x, rows=True, cols=True)
    check_form(row, host(x))
    check_form(col, host(x).T)
    v = host(nsb.muon_mx_dequantize(row, torch.float32))
    want = mxref.values(*mxref.quantize(host(x)), 96)
    assert np.array_equal(np.isnan(v), np.isnan(want))
    assert np.isnan(v[4, :32]).all() and not np.isnan(v[4, 32:]).any()
    assert np.array_equal(v[~np.isnan(v)], want[~np.isnan(want)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_special_values_of_16_bits(dtype):
    """Subnormals, ties, the largest values, infinities and NaNs in blocks of every alignment."""
    info = torch.finfo(dtype)
    sub = info.smallest_normal * info.eps  # the smallest subnormal
    x = torch.zeros(64, 96, dtype=torch.float64)
    x[0] = sub * (torch.arange(96) % 7)
    x[1] = info.smallest_normal * (1 + (torch.arange(96) % 5) * info.eps)
    x[2, ::2], x[2, 1::2] = info.max, -info.max / 3
    x[3] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 12) * info.smallest_normal * 4
    x[4] = -x[3]
    x[5, 40], x[6, 41], x[7, 0] = float("inf"), float("nan"), -float("inf")
    x[8, 3], x[8, 4:32] = 1.0, sub
    x[40:] = torch.randn(24, 96, generator=torch.Generator().manual_seed(1)) * sub * 100
    x = x.to(dtype).cuda()
    row, col = nsb.muon_mx_quantize(x, rows=True, cols=True)
    check_form(row, host(x))
    check_form(col, host(x).T)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize(dtype):
    xs = [normal(s, 40 + i, torch.float32, 1.0).cuda() for i, s in enumerate(SHAPES)]
    qs = nsb.muon_mx_quantize(xs)
    ys = nsb.muon_mx_dequantize(qs, dtype)
    for q, x, y in zip(qs, xs, ys):
        want = torch.from_numpy(mxref.values(*mxref.quantize(host(x)), x.shape[1]))
        assert y.dtype == dtype and torch.equal(y.cpu(), want.to(dtype))
        assert torch.equal(nsb.muon_mx_dequantize(q, dtype), y)


def test_quantize_list_more_than_a_launch_holds():
    xs = [normal((1 + 7 * i % 150, 1 + 11 * i % 140), i).cuda() for i in range(150)] + [torch.empty(0, 5).cuda(), torch.empty(4, 0).cuda()]
    pairs = nsb.muon_mx_quantize(xs, rows=True, cols=True)
    for x, (row, col) in zip(xs, pairs):
        assert row.shape == tuple(x.shape) and col.shape == tuple(x.shape)[::-1]
        if x.numel():
            check_form(row, host(x))
            check_form(col, host(x).T)


def test_quantize_into_given_forms():
    x = normal((70, 200), 3).cuda()
    out = (nsb.MxMatrix.empty(70, 200), nsb.MxMatrix.empty(200, 70))
    for q in out:
        q.data.fill_(255), q.scales.fill_(255)
    assert nsb.muon_mx_quantize(x, rows=True, cols=True, out=out) is out
    check_form(out[0], host(x))
    check_form(out[1], host(x).T)


@pytest.mark.parametrize("shape", [(1, 1), (33, 65), (130, 257), (256, 128)])
def test_nothing_beside_the_forms_is_written(shape):
    """Forms and values between guard bytes."""
    def guarded(count, dtype=torch.uint8):
        wide = torch.full((count + 2 * 256,), 77, dtype=torch.uint8, device="cuda")
        return wide, wide[256:256 + count].view(dtype)
    r, c = shape
    x = normal(shape, 6, torch.bfloat16).cuda()
    wides, forms = [], []
    for a, b in ((r, c), (c, r)):
        d, s = nsb.MxMatrix._data_shape(a, b), nsb.MxMatrix._scales_shape(a, b)
        wd, vd = guarded(d[0] * d[1])
        ws, vs = guarded(s[0] * s[1] * 512)
        wides += [wd, ws]
        forms.append(nsb.MxMatrix(vd.view(d), vs.view(s), a, b))
    nsb.muon_mx_quantize(x, rows=True, cols=True, out=tuple(forms))
    check_form(forms[0], host(x))
    check_form(forms[1], host(x).T)
    for w in wides:
        assert (w[:256] == 77).all() and (w[-256:] == 77).all()


def exact_product(a, b):
    """C and sum |a||b| in fp64 from what the forms hold."""
    def val(q):
        return mxref.values(*mxref.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), *q.shape), q.cols)
    x, y = val(a), val(b)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def check_product(c, a, b, dtype):
    """Products of two codes are exact in fp32 (6 bits, and a power of two); the sums round or
    truncate at most twice a block of 32, each time by at most one fp32 unit, 2^-23, of what is
    summed so far, which sum |a||b| bounds.  The result is then rounded once to its type."""
    want, mag = exact_product(a, b)
    tol = 2 * (-(-a.cols // 32) + 1) * 2.0 ** -23 * mag
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol) + 2.0 ** -25 * (dtype == torch.float16)
    got = host(c)
    assert c.dtype == dtype and got.shape == want.shape
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / np.maximum(tol, 1e-300))


PRODUCTS = [(1, 1, 1), (1, 128, 32), (1, 130, 777), (3, 500, 96), (17, 300, 256), (32, 32, 64), (33, 513, 320),
            (64, 1000, 128), (65, 64, 96), (100, 7, 513), (128, 128, 128), (129, 257, 288), (300, 200, 1000),
            (512, 384, 2048), (1000, 777, 333), (257, 1500, 64), (700, 33, 4000), (2000, 1900, 256)]
# tiles of 256 x 256: several a pair of CTAs, every remainder of k within a stage, ragged edges
PRODUCTS += [(4100, 4200, k) for k in (32, 40, 96, 130, 192, 224, 256)] + [(4100, 4201, 300), (2100, 2300, 1111), (16, 4096, 4096), (40, 300, 5000), (300, 20, 3000), (130, 50, 700), (256, 300, 5000), (5000, 1025, 96)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    a, b = nsb.muon_mx_quantize([normal((m, k), 11 + m, spread=1.0).cuda(), normal((n, k), 12 + n, spread=1.0).cuda()])
    for dtype in TYPES:
        c = nsb.muon_mx_product(a, b, dtype=dtype)
        check_product(c, a, b, dtype)
        assert torch.equal(c, nsb.muon_mx_product(a, b, dtype=dtype))
    assert nsb.muon_get_status() == 0


@pytest.mark.parametrize("m,n", [(200, 150), (20, 300), (300, 60), (4100, 4200)])
def test_product_scales_far_apart(m, n):
    """Each block its own scale, over many powers of two: every scale byte reaches its own block."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(m, 640, generator=g).view(m, 20, 32) * 2.0 ** torch.randint(-12, 12, (m, 20, 1), generator=g)
    y = torch.randn(n, 640, generator=g).view(n, 20, 32) * 2.0 ** torch.randint(-12, 12, (n, 20, 1), generator=g)
    a, b = nsb.muon_mx_quantize([x.reshape(m, 640).cuda(), y.reshape(n, 640).cuda()])
    check_product(nsb.muon_mx_product(a, b, torch.float32), a, b, torch.float32)


@pytest.mark.parametrize("m", [5, 200])
def test_product_nan_blocks_and_zeros(m):
    x, y = normal((m, 300), 21), normal((140, 300), 22)
    x[1, 290] = float("nan")
    x[2] = 0
    y[130, 0] = float("inf")
    a, b = nsb.muon_mx_quantize([x.cuda(), y.cuda()])
    c = nsb.muon_mx_product(a, b, torch.float32).cpu()
    assert c[1].isnan().all() and c[:, 130].isnan().all()
    rest = torch.ones(m, 140, dtype=torch.bool)
    rest[1], rest[:, 130] = False, False
    assert c[rest].isfinite().all() and (c[2][rest[2]] == 0).all()


@pytest.mark.parametrize("m,n", [(40, 300), (300, 40), (300, 300)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_into_a_strided_out(m, n, dtype):
    a, b = nsb.muon_mx_quantize([normal((m, 200), 31).cuda(), normal((n, 200), 32).cuda()])
    for left, right in ((0, 0), (3, 5), (8, 16)):
        wide = torch.full((m + 2, left + n + right), 7.0, dtype=dtype, device="cuda")
        out = wide[1:-1, left:left + n]
        assert nsb.muon_mx_product(a, b, out=out) is out
        assert torch.equal(out, nsb.muon_mx_product(a, b, dtype=dtype))
        wide[1:-1, left:left + n] = 7.0
        assert (wide == 7.0).all()  # nothing beside it was written


def test_product_of_nothing():
    a, b = nsb.muon_mx_quantize([torch.empty(5, 0).cuda(), torch.empty(7, 0).cuda()])
    assert torch.equal(nsb.muon_mx_product(a, b), torch.zeros(5, 7, dtype=torch.bfloat16, device="cuda"))
    a, b = nsb.muon_mx_quantize([torch.empty(0, 64).cuda(), torch.ones(7, 64).cuda()])
    assert nsb.muon_mx_product(a, b).shape == (0, 7) and nsb.muon_mx_product(b, a).shape == (7, 0)
