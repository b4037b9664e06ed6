"""The operators around a Muon-trained linear layer, as work to be measured: layer norm with its gradient,
and 4-bit microscaled (MX) quantisation with the products of the forward and the backward pass.

A block of the models whose hidden matrices ``muon_step`` updates runs, for each of them,

    h  = layer_norm(x) * w + b                      (forward)          dx, dw, db            (backward)
    y  = Q(h) . Q(W)^T                              (forward)
    dh = Q(dy) . Q(W^T)^T,  dW = Q(dy^T) . Q(h^T)^T (backward; dW is the bf16 gradient that ``muon_step`` takes)

where Q(.) is E2M1 with one power-of-two scale for each 32 values along the dimension that the product sums over:
the scale's byte is max(0, E - 2) for the biased fp32 exponent E of the block's largest magnitude (255, a NaN, when
the block holds an infinity or a NaN), and each value is divided by 2^(byte - 127), rounded to the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) and held at 6.

A 4-bit matrix (rows x cols) is held as
    data    uint8 [rows, 16 * ceil(cols / 32)]   two values a byte, the even column in the low half, code = sign * 8 + index
    scales  uint8 [ceil(rows / 128), ceil(cols / 128), 32, 16]
            the byte of block 4 C + b of row 128 R + 32 j + r is scales[R, C, r, 4 j + b]
with zeros beyond the matrix.

``own`` false: the plain forms, in elementary torch operations.  ``own`` true: the framework's calls.
"""
import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token of a decoding loop through a norm of GPT-2 small's width: only latency counts
        dict(name="norm_token", op="norm", rows=1, cols=768, type="bf16", params="fp32", bias=True, pad=0),
        # one micro-batch of 32 sequences of 1024 tokens, GPT-2 small
        dict(name="norm_tokens", op="norm", rows=32768, cols=768, type="bf16", params="fp32", bias=True, pad=0),
        # odd sizes: rows that start on no 16-byte boundary, a slice of a wider tensor, fp32, no bias
        dict(name="norm_ragged", op="norm", rows=2047, cols=5003, type="fp32", params="fp32", bias=False, pad=7),
        # the gradient for a short sequence of the 1024-wide set, fp16 throughout
        dict(name="norm_grad_short", op="norm_grad", rows=331, cols=1024, type="fp16", params="fp16", bias=True, pad=0),
        # the gradient of the micro-batch above
        dict(name="norm_grad_tokens", op="norm_grad", rows=32768, cols=768, type="bf16", params="fp32", bias=True, pad=0),
        # the gradient at a large model's width
        dict(name="norm_grad_wide", op="norm_grad", rows=8192, cols=8192, type="bf16", params="bf16", bias=True, pad=0),
        # four layers of GPT-2 small's hidden matrices (fp32 weights) after a Muon step: both forms of each, in one call
        dict(name="quantize_weights", op="quantize", layers=4, rows=0, cols=768, type="fp32", both=True, pad=0),
        # activations kept for the backward pass, both forms; a token count that ends inside a block
        dict(name="quantize_tokens", op="quantize", layers=0, rows=16381, cols=4096, type="bf16", both=True, pad=0),
        # one token through GPT-2 small's MLP-in weight: quantise it, then the product
        dict(name="linear_token", op="linear", m=1, n=3072, k=768, type="bf16"),
        # a ragged prompt through the 1024-wide set's MLP-in weight
        dict(name="linear_prompt", op="linear", m=777, n=4096, k=1024, type="bf16"),
        # both products of a layer's backward pass: the gradient for its input, and the weight gradient for muon_step
        dict(name="linear_grad", op="linear_grad", m=16384, n=4096, k=1024, type="bf16"),
        # a large product of two matrices that are held in 4 bits
        dict(name="product_large", op="product", m=8192, n=8192, k=8192, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _odd(rng, v, step):
    """Half the sizes are multiples of `step`, as models have them; the others are what they are."""
    return max(step, v // step * step) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "linear", "linear_grad", "product"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        cols = _odd(rng, _log(rng, 64, 16384), 64)
        rows = _log(rng, 1, min(65536, (1 << 26) // cols))
        return dict(op=op, rows=rows, cols=cols, type=kind, params=rng.choice(["fp32", kind]), bias=rng.random() < 0.7,
                    pad=rng.choice([0, 0, 8, 13]))
    if op == "quantize":
        if rng.random() < 0.3:
            return dict(op=op, layers=rng.randint(1, 4), rows=0, cols=rng.choice([256, 384, 640, 768]), type="fp32",
                        both=rng.random() < 0.7, pad=0)
        cols = _odd(rng, _log(rng, 64, 16384), 64)
        rows = _log(rng, 1, min(65536, (1 << 26) // cols))
        return dict(op=op, layers=0, rows=rows, cols=cols, type=kind, both=rng.random() < 0.7, pad=rng.choice([0, 0, 8, 13]))
    n, k = (_odd(rng, _log(rng, 128, 8192), 128) for _ in range(2))
    m = _log(rng, 1, min(16384, (1 << 36) // (n * k)))
    return dict(op=op, m=m, n=n, k=k, type=rng.choice(["bf16", "bf16", "fp16"]))


# ------------------------------------------------------------------------------------------------ inputs

def _shapes(case):
    """The matrices of a quantize case: a set of layers (4 square, MLP-in, MLP-out), or one matrix."""
    if case["layers"]:
        w = case["cols"]
        return ([(w, w)] * 4 + [(w, 4 * w), (4 * w, w)]) * case["layers"]
    return [(case["rows"], case["cols"])]


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _activations(g, rows, cols, kind, pad=0):
    """A residual stream: an offset and a spread for each token, and a few channels that are far larger."""
    x = _normal(g, rows, cols + pad)
    x *= torch.exp(0.5 * _normal(g, 1, cols + pad)) * torch.exp(0.3 * _normal(g, rows, 1))
    x += 0.5 * _normal(g, rows, 1)
    return x.to(TYPES[kind])[:, :cols]


def _gradients(g, rows, cols, kind, pad=0):
    """Gradients: small, of very different size from token to token."""
    x = _normal(g, rows, cols + pad) * torch.exp(_normal(g, rows, 1))
    return (x * (1e-2 if kind == "fp16" else 1e-4)).to(TYPES[kind])[:, :cols]


def _packed(values, state, name):
    """The 4-bit form of a matrix along its rows, in the layout of the module's heading."""
    rows, cols = values.shape
    code, byte = _codes(values.float())
    code = code.reshape(rows, -1)
    state[name + "_data"] = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    r, c = -(-rows // 128), -(-cols // 128)
    full = torch.zeros(r * 128, c * 4, dtype=torch.uint8, device=DEVICE)
    full[:rows, : byte.shape[1]] = byte.to(torch.uint8)
    state[name + "_scales"] = full.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).reshape(r, c, 32, 16).contiguous()
    state[name + "_shape"] = (rows, cols)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = {"case": case}
    op, kind = case["op"], case["type"]
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols, kind, case["pad"])
        s["weight"] = (1 + 0.2 * _normal(g, cols)).to(TYPES[case["params"]])
        s["bias"] = (0.1 * _normal(g, cols)).to(TYPES[case["params"]]) if case["bias"] else None
        if op == "norm_grad":
            s["dy"] = _gradients(g, rows, cols, kind, case["pad"])
            x = s["x"].double()  # what the forward pass kept
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (((x - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
    elif op == "quantize":
        if case["layers"]:
            s["x"] = [0.02 * _normal(g, r, c) for r, c in _shapes(case)]
        else:
            s["x"] = [_activations(g, case["rows"], case["cols"], kind, case["pad"])]
    elif op == "linear":
        s["x"] = _activations(g, case["m"], case["k"], kind)
        _packed(0.02 * _normal(g, case["n"], case["k"]), s, "w")
    elif op == "linear_grad":
        s["dy"] = _gradients(g, case["m"], case["n"], kind)
        _packed(0.02 * _normal(g, case["k"], case["n"]), s, "wt")
        _packed(_activations(g, case["k"], case["m"], "fp32"), s, "xt")
    else:
        _packed(_activations(g, case["m"], case["k"], "fp32"), s, "a")
        _packed(0.02 * _normal(g, case["n"], case["k"]), s, "b")
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _pow2(byte):
    """2^(byte - 127) as fp32; 255 is a NaN."""
    bits = torch.where(byte > 0, byte << 23, torch.full_like(byte, 1 << 22))
    return torch.where(byte == 255, torch.full_like(byte, 0x7FC00000), bits).to(torch.int32).view(torch.float32)


def _codes(x):
    """E2M1 codes [rows, blocks, 32] and scale bytes [rows, blocks] of an fp32 matrix, in blocks along its rows."""
    rows, cols = x.shape
    x = torch.cat([x, x.new_zeros(rows, -cols % 32)], 1).reshape(rows, -1, 32)
    amax = x.abs().amax(2)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
    byte = torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255))
    a = (x * ((254 - byte.clamp(max=252)) << 23).view(torch.float32)[:, :, None]).abs()
    code = (a > 0.25).to(torch.uint8)
    for limit, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= limit) if even else (a > limit)
    return code | (x < 0).to(torch.uint8) << 3, byte


def _grid():
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device=DEVICE)
    return torch.cat([half, -half])


def _rounded(x):
    """The values that the 4-bit form of x stands for, in fp32."""
    rows, cols = x.shape
    code, byte = _codes(x.float())
    return (_grid()[code.long()] * _pow2(byte)[:, :, None]).reshape(rows, -1)[:, :cols]


def _values(s, name):
    """The values that a packed matrix of the state stands for, in fp32."""
    rows, cols = s[name + "_shape"]
    data, scales = s[name + "_data"], s[name + "_scales"]
    code = torch.stack((data & 15, data >> 4), 2).reshape(rows, -1, 32)
    r, c = scales.shape[:2]
    byte = scales.view(r, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, c * 4)[:rows, : code.shape[1]]
    return (_grid()[code.long()] * _pow2(byte.to(torch.int32))[:, :, None]).reshape(rows, -1)[:, :cols]


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _norm_grad(s):
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    out = [dx.to(s["x"].dtype), (dy * xhat).sum(0).to(s["weight"].dtype)]
    return out + [dy.sum(0).to(s["bias"].dtype)] if s["bias"] is not None else out


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, op, case)
    if op == "norm":
        return _norm(s)
    if op == "norm_grad":
        return _norm_grad(s)
    kind = TYPES[case["type"]]
    if op == "quantize":
        out = []
        for x in s["x"]:
            out.append(_rounded(x).bfloat16())
            if case["both"]:
                out.append(_rounded(x.t()).bfloat16())
        return out
    if op == "linear":
        return (_rounded(s["x"]) @ _values(s, "w").t()).to(kind)
    if op == "linear_grad":
        dx = _rounded(s["dy"]) @ _values(s, "wt").t()
        dw = _rounded(s["dy"].t()) @ _values(s, "xt").t()
        return [dx.to(kind), dw.to(kind)]
    return (_values(s, "a") @ _values(s, "b").t()).to(kind)


# ------------------------------------------------------------------------------------------------ the framework's calls

def _own(s, op, case):
    import newton_schulz_12_b200 as nsb

    def held(name):
        return nsb.MxMatrix(s[name + "_data"], s[name + "_scales"], *s[name + "_shape"])

    if op == "norm":
        return nsb.muon_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_grad":
        dx, dw, db = nsb.muon_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], bias=s["bias"] is not None)
        return [dx, dw] if db is None else [dx, dw, db]
    kind = TYPES[case["type"]]
    if op == "quantize":
        forms = nsb.muon_mx_quantize(s["x"], rows=True, cols=case["both"])
        return nsb.muon_mx_dequantize([f for pair in forms for f in pair] if case["both"] else forms)
    if op == "linear":
        return nsb.muon_mx_product(nsb.muon_mx_quantize(s["x"]), held("w"), dtype=kind)
    if op == "linear_grad":
        dyr, dyc = nsb.muon_mx_quantize(s["dy"], rows=True, cols=True)
        return [nsb.muon_mx_product(dyr, held("wt"), dtype=kind), nsb.muon_mx_product(dyc, held("xt"), dtype=kind)]
    return nsb.muon_mx_product(held("a"), held("b"), dtype=kind)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    e = size[case["type"]]

    def held(rows, cols):
        return rows * -(-cols // 32) * 17

    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        p = size[case["params"]] * cols * (2 if case["bias"] else 1)
        if op == "norm":
            return {"bytes": 2 * rows * cols * e + p + 8 * rows, "flops": 8 * rows * cols}
        return {"bytes": 3 * rows * cols * e + p + size[case["params"]] * cols + 8 * rows, "flops": 14 * rows * cols}
    if op == "quantize":
        total = 0
        for r, c in _shapes(case):  # read, then each form written, and read and written as values
            total += r * c * e + 2 * held(r, c) + 2 * r * c
            if case["both"]:
                total += 2 * held(c, r) + 2 * r * c
        return {"bytes": total, "flops": 4 * total}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        return {"bytes": m * k * e + held(n, k) + m * n * e, "flops": 2 * m * n * k}
    if op == "linear_grad":
        return {"bytes": m * n * e + held(k, n) + held(k, m) + (m + n) * k * e, "flops": 4 * m * n * k}
    return {"bytes": held(m, k) + held(n, k) + m * n * e, "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _e2m1(x):
    """Q(x) along the rows of a matrix, in fp64: each value to the nearest multiple of its own step."""
    x = x.double()
    rows, cols = x.shape
    wide = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    wide[:, :cols] = x
    blocks = wide.view(rows, -1, 32)
    top = blocks.abs().max(2, keepdim=True).values
    exponent = torch.frexp(top).exponent.double() - 1  # top = f * 2^exponent, 1 <= f < 2
    scale = torch.exp2((torch.where(top > 0, exponent, -127.0) - 2).clamp(min=-127))
    v = blocks / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((torch.round(v / step) * step).clamp(-6, 6) * scale).reshape(rows, -1)[:, :cols]


def _held_exactly(s, name):
    """A packed matrix of the state in fp64, one bit field at a time."""
    rows, cols = s[name + "_shape"]
    data = s[name + "_data"].to(torch.int16)
    wide = torch.empty(rows, 2 * data.shape[1], dtype=torch.float64, device=data.device)
    for half in (0, 1):
        c = data >> 4 * half & 15
        mant, exp = (c & 1).double(), (c >> 1 & 3).double()
        mag = torch.where(exp > 0, (1 + mant / 2) * torch.exp2(exp - 1), mant / 2)
        wide[:, half::2] = torch.where(c > 7, -mag, mag)
    row = torch.arange(rows, device=data.device)[:, None]
    block = torch.arange(data.shape[1] // 16, device=data.device)[None, :]
    byte = s[name + "_scales"][row // 128, block // 4, row % 32, row % 128 // 32 * 4 + block % 4]
    return (wide.view(rows, -1, 32) * torch.exp2(byte.double() - 127)[:, :, None]).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        y = (x - mean) * rstd * s["weight"].double()
        if s["bias"] is not None:
            y += s["bias"].double()
        return y, mean[:, 0], rstd[:, 0]
    if op == "norm_grad":
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        centred = (s["x"].double() - s["mean"].double()[:, None])
        n = case["cols"]
        wdy = dy * s["weight"].double()
        along = (wdy * centred).sum(1, keepdim=True) * rstd ** 2 / n
        out = [rstd * (wdy - wdy.sum(1, keepdim=True) / n - centred * along),
               torch.einsum("rc,rc->c", dy, centred * rstd)]
        return out + [dy.sum(0)] if s["bias"] is not None else out
    if op == "quantize":
        out = []
        for x in s["x"]:
            out.append(_e2m1(x))
            if case["both"]:
                out.append(_e2m1(x.t()))
        return out
    if op == "linear":
        return _e2m1(s["x"]) @ _held_exactly(s, "w").t()
    if op == "linear_grad":
        return [_e2m1(s["dy"]) @ _held_exactly(s, "wt").t(), _e2m1(s["dy"].t()) @ _held_exactly(s, "xt").t()]
    return _held_exactly(s, "a") @ _held_exactly(s, "b").t()
