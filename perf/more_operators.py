"""The operators of a layer whose product is taken in 8 bits: the product itself, with a scale for each block of 128; the
root-mean-square norm that feeds it, with the residual's addition, and its gradient; activations and gradients turned into 8
bits by rows and by columns; and the 8-bit copies of many weights that an optimizer's step leaves behind.

An 8-bit matrix of `rows` x `cols` values holds them as e4m3 or e5m2 codes, rows padded with zeros to whole blocks of 128, and
one power of two for each block of 128 along a row: the least 2^e, e >= -127, with which the block's largest finite value fits
the format.  The exponents are bytes e + 127, those of four neighbouring blocks together: scales[group, row, 4].  Weights share
one scale over 128 x 128 values, so that a matrix and its transpose hold the same values.

  norm      z = x + residual, rounded to the residual's type;  r = 1 / sqrt(mean(z^2) + eps);  h = (z r) w, in 8 bits by rows
  normback  a = w g;  dz = r (a - z r mean(a z r)) + add;  dw = sum over the rows of g z r
  quantize  a matrix in 8 bits by its rows, by its columns (the transpose, by rows), or both
  flip      an 8-bit matrix's transpose, its values scaled anew along the other side
  weights   8-bit copies of many matrices and of their transposes
  product   C = A B^T, or C + A B^T: y = x W^T, dx = dy W (from W's transpose), dW = dy^T x (from both transposes)
"""
import math
import random

import torch

own = False

BLOCK = 128
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}          # the exponent of the format's largest value, 1.75 * 2^TOP
LEAST = {"e4m3": -9, "e5m2": -16}      # of its smallest
DIGITS = {"e4m3": 3, "e5m2": 2}        # bits behind the point


# ------------------------------------------------------------------ cases
def _matrices(case):
    """The weight matrices of a case: (rows, columns)."""
    which = case["set"]
    if which == "ctr":
        return [(1024, 1024), (1024, 512), (512, 256)]
    if which == "bert":
        return ([(1024, 1024)] * 4 + [(1024, 4096), (4096, 1024)]) * 24
    r = random.Random(case["tseed"])
    return [(int(2 ** r.uniform(3, 12)), int(2 ** r.uniform(3, 12))) for _ in range(case["tensors"])]


def listed():
    def norm(name, rows, dim, x="bf16", res="bf16", pad=0):
        return {"name": name, "op": "norm", "rows": rows, "dim": dim, "x": x, "res": res, "pad": pad}

    def back(name, rows, dim, g="bf16", z="bf16", pad=0):
        return {"name": name, "op": "normback", "rows": rows, "dim": dim, "g": g, "z": z, "pad": pad}

    def product(name, m, n, k, a="e4m3", b="e4m3", out="bf16", add=False, pad=0):
        return {"name": name, "op": "product", "m": m, "n": n, "k": k, "a": a, "b": b, "out": out, "add": add, "pad": pad}

    return [
        # one token through a norm: the latency of a call
        norm("norm-token", 1, 1024),
        # the tokens of a training step at BERT-large's width, residual stream in 32 bits
        norm("norm-16384x1024", 16384, 1024, "bf16", "f32"),
        # rows of no pattern cut out of a wider buffer, everything in 32 bits
        back("normback-1501x1000", 1501, 1000, "f32", "f32", 3),
        # a wide model's step
        back("normback-8192x4096", 8192, 4096),
        # gradients of odd sizes, for both of the products that read them
        {"name": "quantize-3001x1530", "op": "quantize", "rows": 3001, "cols": 1530, "x": "f32", "fmt": "e5m2", "by": "both", "pad": 1},
        # what the forward pass left in 8 bits, transposed for the weight's gradient
        {"name": "flip-16384x4096", "op": "flip", "rows": 16384, "cols": 4096, "fmt": "e4m3"},
        # the weights of a click model's MLP after a step
        {"name": "weights-ctr", "op": "weights", "set": "ctr", "x": "f32"},
        # all the matrices of a BERT-large-shaped model after a step
        {"name": "weights-bert", "op": "weights", "set": "bert", "x": "bf16"},
        # one token through a feed-forward matrix: the pace of reading the weight
        product("product-token", 1, 4096, 1024),
        # a ragged batch into a classifier's 1000 classes, logits in 32 bits
        product("product-777x1000", 777, 1000, 2048, out="f32", pad=1),
        # a weight's gradient added over micro-batches: a long sum into a small matrix, gradients in e5m2
        product("product-dw", 1024, 4096, 16384, "e5m2", "e4m3", "f32", True),
        # the largest forward product
        product("product-8192", 8192, 8192, 8192),
    ]


def draw(rng):
    size = lambda low, high: max(1, int(2 ** rng.uniform(low, high)))  # noqa: E731
    kind = lambda: rng.choice(("bf16", "f32", "f16"))  # noqa: E731
    op = rng.choice(("norm", "norm", "normback", "normback", "quantize", "flip", "weights", "product", "product", "product", "product"))
    if op in ("norm", "normback"):
        dim = size(5, 14)
        case = {"op": op, "rows": min(size(0, 15), 33_000_000 // dim), "dim": dim, "pad": rng.choice((0, 0, 1, 8))}
        return {**case, "x": kind(), "res": rng.choice(("none", "bf16", "f32", "f16"))} if op == "norm" else {**case, "g": kind(), "z": kind()}
    if op in ("quantize", "flip"):
        cols = size(3, 13)
        case = {"op": op, "rows": min(size(0, 14.5), 33_000_000 // cols), "cols": cols, "fmt": rng.choice(("e4m3", "e5m2"))}
        return {**case, "x": kind(), "by": rng.choice(("rows", "cols", "both")), "pad": rng.choice((0, 0, 1, 8))} if op == "quantize" else case
    if op == "weights":
        return {"op": op, "set": "ragged", "x": rng.choice(("bf16", "f32")), "tseed": rng.randrange(1 << 30), "tensors": size(0, 5)}
    most = 8192 ** 3
    n, k = size(5, 13), size(5, 13)
    m = min(size(0, 14.5), most // (n * k))
    out = rng.choice(("bf16", "f32", "f16"))
    return {"op": op, "m": m, "n": n, "k": k, "a": rng.choice(("e4m3", "e4m3", "e5m2")), "b": rng.choice(("e4m3", "e4m3", "e5m2")), "out": out,
            "add": out == "f32" and rng.random() < 0.4, "pad": rng.choice((0, 0, 1, 8))}


# ------------------------------------------------------------------ 8-bit matrices in elementary operations
def _up(n, unit=BLOCK):
    return -(-n // unit) * unit


def _blocks(x):
    """Rows cut into blocks of 128, with zeros behind their end."""
    return torch.nn.functional.pad(x, (0, _up(x.shape[1]) - x.shape[1])).view(x.shape[0], -1, BLOCK)


def _coded(blocks, largest, fmt):
    """Codes and exponent bytes of blocks by their largest finite values."""
    byte = (((largest.view(torch.int32) + 0x1FFFFF) >> 23) - TOP[fmt]).clamp_min(0)
    inverse = ((254 - byte) << 23).view(torch.float32)
    codes = (blocks * inverse).to(CODES[fmt])
    return codes.view(blocks.shape[0], -1), _grouped(byte[..., 0])


def _grouped(byte):
    """Bytes of (row, block) as [group, row, 4]."""
    rows, n = byte.shape
    byte = torch.nn.functional.pad(byte, (0, _up(n, 4) - n)).view(rows, -1, 4)
    return byte.transpose(0, 1).contiguous().to(torch.uint8)


def _largest(x, dims):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dims, keepdim=True)


def _encode(x, fmt):
    blocks = _blocks(x)
    return _coded(blocks, _largest(blocks, -1), fmt)


def _encode_weight(x):
    """A matrix and its transpose, one scale for each 128 x 128 values."""
    rows, cols = x.shape
    tiles = torch.nn.functional.pad(x, (0, _up(cols) - cols, 0, _up(rows) - rows)).view(_up(rows) // BLOCK, BLOCK, -1, BLOCK)
    largest = _largest(tiles, (1, 3))
    side = lambda t, m, n: _coded(_blocks(t), m.expand(-1, BLOCK, -1, -1).reshape(-1, m.shape[2], 1)[:n], "e4m3")  # noqa: E731
    return *side(x, largest, rows), *side(x.t().contiguous(), largest.permute(2, 1, 0, 3), cols)


def _decode(codes, scales, cols):
    """The values, in fp32."""
    rows, pitch = codes.shape
    byte = scales.transpose(0, 1).reshape(rows, -1)[:, :pitch // BLOCK].to(torch.int32)
    scale = torch.where(byte == 0, torch.full_like(byte, 1 << 22), byte << 23).view(torch.float32)
    return (codes.float().view(rows, -1, BLOCK) * scale[..., None]).view(rows, pitch)[:, :cols]


# ------------------------------------------------------------------ inputs
def _sections(shapes):
    """Places of the codes and of the scales of matrices and their transposes, one after another in whole 256 bytes."""
    codes = scales = 0
    found = []
    for r, c in shapes:
        for rows, cols in ((r, c), (c, r)):
            n, s = rows * _up(cols), rows * _up(cols // BLOCK + (cols % BLOCK > 0), 4)
            found.append((codes, n, scales, s))
            codes, scales = codes + _up(n, 256), scales + _up(s, 256)
    return found, codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)

    def wide(rows, cols, dtype, spread, pad=0, level=1.0):
        """Rows of a buffer `pad` elements wider.  Values of a network: most of one size, `spread` sets how far rows (tokens)
        or columns (channels) are from each other."""
        x = torch.empty(rows, cols + pad, dtype=DTYPES[dtype], device=dev)[:, :cols]
        v = torch.randn(rows, cols, generator=gen, device=dev)
        if spread == "rows":
            v *= torch.exp(torch.randn(rows, 1, generator=gen, device=dev))
        else:
            v *= torch.where(torch.rand(1, cols, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        x.copy_(v * level)
        return x

    s = dict(case)
    op = case["op"]
    if op == "norm":
        rows, dim = case["rows"], case["dim"]
        s["x"] = wide(rows, dim, case["x"], "cols", case["pad"])
        s["w"] = 1 + 0.1 * torch.randn(dim, generator=gen, device=dev)
        s["residual"] = wide(rows, dim, case["res"], "cols", case["pad"], 3.0) if case["res"] != "none" else None
    elif op == "normback":
        rows, dim = case["rows"], case["dim"]
        s["grad"] = wide(rows, dim, case["g"], "rows", case["pad"], 1e-3)
        s["z"] = wide(rows, dim, case["z"], "cols", case["pad"], 3.0)
        s["add"] = wide(rows, dim, case["z"], "rows", case["pad"], 1e-3)
        s["w"] = 1 + 0.1 * torch.randn(dim, generator=gen, device=dev)
        s["rstd"] = 1 / (s["z"].double().square().mean(1) + EPS).sqrt().float()
    elif op == "quantize":
        s["x"] = wide(case["rows"], case["cols"], case["x"], "rows", case["pad"], 1e-4)
    elif op == "flip":
        s["codes"], s["scales"] = _encode(wide(case["rows"], case["cols"], "bf16", "cols").float(), case["fmt"])
    elif op == "weights":
        s["shapes"] = _matrices(case)
        s["params"] = [wide(r, c, case["x"], "cols", 0, 0.02) for r, c in s["shapes"]]
        s["places"], s["ncodes"], s["nscales"] = _sections(s["shapes"])
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["a_codes"], s["a_scales"] = _encode(wide(m, k, "f32", "rows"), case["a"])
        s["b_codes"], s["b_scales"] = _encode(wide(n, k, "f32", "cols", 0, 0.02), case["b"])
        s["c"] = wide(m, n, case["out"], "rows", case["pad"])
    if own:
        _own_objects(s, dev)
    return s


def _own_objects(s, dev):
    """What a program that uses the framework's operators keeps beside its data."""
    from second_order_optimizer_amd import fp8 as F
    s["F"], op = F, s["op"]
    seen = lambda m: [m.codes, m.scales.view(torch.float8_e8m0fnu)]  # noqa: E731
    if op == "norm":
        s["out8"] = F.Matrix8(s["rows"], s["dim"], device=dev)
        s["total"] = torch.empty_like(s["residual"]) if s["residual"] is not None else None
        s["rstd"] = torch.empty(s["rows"], device=dev)
        s["seen"] = [s["total"], s["rstd"], *seen(s["out8"])]
    elif op == "normback":
        s["dz"], s["dw"] = torch.empty_like(s["z"]), torch.empty(s["dim"], device=dev)
        s["seen"] = [s["dz"], s["dw"]]
    elif op == "quantize":
        s["by_rows"] = F.Matrix8(s["rows"], s["cols"], s["fmt"], device=dev) if s["by"] != "cols" else None
        s["by_cols"] = F.Matrix8(s["cols"], s["rows"], s["fmt"], device=dev) if s["by"] != "rows" else None
        s["seen"] = [v for m in (s["by_rows"], s["by_cols"]) if m is not None for v in seen(m)]
    elif op == "flip":
        s["m"] = F.Matrix8(s["rows"], s["cols"], s["fmt"], device=dev, codes=s["codes"], scales=s["scales"])
        s["by_cols"] = F.Matrix8(s["cols"], s["rows"], s["fmt"], device=dev)
        s["seen"] = seen(s["by_cols"])
    elif op == "weights":
        s["copies"] = F.Weights8(s["shapes"], param=s["x"], device=dev)
        s["copies"].bind(s["params"])
        s["seen"] = [s["copies"].codes, s["copies"].scales.view(torch.float8_e8m0fnu)]
    else:
        s["a8"] = F.Matrix8(s["m"], s["k"], s["a"], device=dev, codes=s["a_codes"], scales=s["a_scales"])
        s["b8"] = F.Matrix8(s["n"], s["k"], s["b"], device=dev, codes=s["b_codes"], scales=s["b_scales"])


# ------------------------------------------------------------------ plain forms
def _plain(s):
    op = s["op"]
    shown = lambda codes, scales: [codes, scales.view(torch.float8_e8m0fnu)]  # noqa: E731
    if op == "norm":
        z = s["x"].float()
        total = None
        if s["residual"] is not None:
            total = (z + s["residual"].float()).to(s["residual"].dtype)
            z = total.float()
        r = 1 / ((z * z).mean(1) + EPS).sqrt()
        return [total, r, *shown(*_encode((z * r[:, None]) * s["w"], "e4m3"))]
    if op == "normback":
        g, z, r = s["grad"].float(), s["z"].float(), s["rstd"][:, None]
        a, unit = g * s["w"], z * r
        dz = r * (a - unit * (a * unit).mean(1, keepdim=True)) + s["add"].float()
        return [dz.to(s["z"].dtype), (g * unit).sum(0)]
    if op == "quantize":
        x = s["x"].float()
        return (shown(*_encode(x, s["fmt"])) if s["by"] != "cols" else []) + (shown(*_encode(x.t().contiguous(), s["fmt"])) if s["by"] != "rows" else [])
    if op == "flip":
        return shown(*_encode(_decode(s["codes"], s["scales"], s["cols"]).t().contiguous(), s["fmt"]))
    if op == "weights":
        codes = torch.zeros(s["ncodes"], dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.zeros(s["nscales"], dtype=torch.uint8, device="cuda")
        made = [_encode_weight(p.float()) for p in s["params"]]
        pairs = [pair for four in made for pair in (four[:2], four[2:])]
        torch._foreach_copy_([codes[at:at + n].view(torch.uint8) for at, n, _, _ in s["places"]], [c.view(torch.uint8).view(-1) for c, _ in pairs])
        torch._foreach_copy_([scales[at:at + n] for _, _, at, n in s["places"]], [b.view(-1) for _, b in pairs])
        return shown(codes, scales)
    c = _decode(s["a_codes"], s["a_scales"], s["k"]) @ _decode(s["b_codes"], s["b_scales"], s["k"]).t()
    s["c"].copy_(s["c"] + c if s["add"] else c)
    return [s["c"]]


# ------------------------------------------------------------------ a pass
def run(s):
    if not own:
        return _plain(s)
    F, op = s["F"], s["op"]
    if op == "norm":
        F.rms_norm(s["x"], s["w"], EPS, residual=s["residual"], total=s["total"], out8=s["out8"], rstd=s["rstd"])
    elif op == "normback":
        F.rms_norm_backward(s["grad"], s["z"], s["rstd"], s["w"], add=s["add"], dz=s["dz"], dw=s["dw"])
    elif op == "quantize":
        F.quantize(s["x"], rows=s["by_rows"], cols=s["by_cols"])
    elif op == "flip":
        F.transpose(s["m"], s["by_cols"])
    elif op == "weights":
        s["copies"].refresh()
    else:
        F.matmul(s["a8"], s["b8"], s["c"], accumulate=s["add"])
        return [s["c"]]
    return s["seen"]


def work(case):
    size = lambda name: 4 if case[name] == "f32" else 2  # noqa: E731
    op = case["op"]
    if op == "norm":
        n = float(case["rows"] * case["dim"])
        wide = size("x") + (2 * size("res") if case["res"] != "none" else 0)
        return {"bytes": n * (wide + 1 + 1 / BLOCK) + 4 * case["rows"] + 4 * case["dim"], "flops": 7 * n}
    if op == "normback":
        n = float(case["rows"] * case["dim"])
        return {"bytes": n * (size("g") + 3 * size("z")) + 4 * case["rows"] + 8 * case["dim"], "flops": 11 * n}
    if op in ("quantize", "flip"):
        n = float(case["rows"] * case["cols"])
        read = 1 + 1 / BLOCK if op == "flip" else size("x")
        return {"bytes": n * (read + (1 + 1 / BLOCK) * (2 if case.get("by") == "both" else 1)), "flops": 3 * n}
    if op == "weights":
        n = float(sum(r * c for r, c in _matrices(case)))
        return {"bytes": n * (size("x") + 2 + 2 / BLOCK), "flops": 3 * n}
    m, n, k = float(case["m"]), float(case["n"]), float(case["k"])
    return {"bytes": (m + n) * k * (1 + 1 / BLOCK) + m * n * size("out") * (2 if case["add"] else 1), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definition in 64 bits
def _power(largest, fmt):
    """The least e >= -127 with largest <= 1.75 * 2^(TOP + e), for fp64 values of 24 bits."""
    fraction, e = torch.frexp(largest)                                   # fraction in [0.5, 1)
    e = e.double() - 1 - TOP[fmt] + (2 * fraction > 1.75).double()
    return torch.where(largest > 0, e, torch.full_like(e, -127.0)).clamp_min(-127.0)


def _nearest(y, fmt):
    """The format's nearest values, halves to the even one."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -200)))
    e = e + (y.abs() >= torch.exp2(e + 1)).double() - (y.abs() < torch.exp2(e)).double()
    step = torch.exp2(torch.maximum(e - DIGITS[fmt], torch.full_like(e, float(LEAST[fmt]))))
    return torch.round(y / step) * step


def _defined(x, fmt, power=None):
    """Codes and scales as values, laid out as they are held.  power: (rows, blocks) exponents, by default each block's own."""
    rows, cols = x.shape
    blocks = torch.zeros(rows, _up(cols), dtype=torch.float64, device=x.device)
    blocks[:, :cols] = x
    blocks = blocks.reshape(rows, -1, BLOCK)
    e = _power(blocks.abs().max(2)[0], fmt) if power is None else power
    scales = torch.full((-(-e.shape[1] // 4), rows, 4), 2.0 ** -127, dtype=torch.float64, device=x.device)
    for b in range(e.shape[1]):
        scales[b // 4, :, b % 4] = torch.exp2(e[:, b])
    return [_nearest(blocks * torch.exp2(-e)[..., None], fmt).reshape(rows, -1), scales]


def _values(codes, scales, cols):
    rows, pitch = codes.shape
    out = codes.double()
    for b in range(pitch // BLOCK):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= torch.exp2(scales[b // 4, :, b % 4].double() - 127)[:, None]
    return out[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        z, total = s["x"].double(), None
        if s["residual"] is not None:
            z = z + s["residual"].double()
            total = z
            z = z.to(s["residual"].dtype).double()      # the norm is that of the values that are stored
        r = torch.rsqrt(torch.linalg.vector_norm(z, dim=1).square() / z.shape[1] + EPS)
        return [total, r, *_defined(z * s["w"].double() * r[:, None], "e4m3")]
    if op == "normback":
        g, z, w, r = (s[name].double() for name in ("grad", "z", "w", "rstd"))
        inner = torch.einsum("mj,mj,j->m", g, z, w)
        dz = r[:, None] * g * w - z * (inner * r ** 3 / z.shape[1])[:, None] + s["add"].double()
        return [dz, torch.mv((g * z).t(), r)]
    if op == "quantize":
        x = s["x"].double()
        return (_defined(x, s["fmt"]) if s["by"] != "cols" else []) + (_defined(x.t(), s["fmt"]) if s["by"] != "rows" else [])
    if op == "flip":
        return _defined(_values(s["codes"], s["scales"], s["cols"]).t(), s["fmt"])
    if op == "weights":
        codes = torch.zeros(s["ncodes"], dtype=torch.float64, device="cuda")
        scales = torch.full((s["nscales"],), 2.0 ** -127, dtype=torch.float64, device="cuda")
        for i, p in enumerate(s["params"]):
            r, c = p.shape
            whole = torch.zeros(_up(r), _up(c), dtype=torch.float64, device="cuda")
            whole[:r, :c] = p
            e = _power(whole.abs().reshape(_up(r) // BLOCK, BLOCK, -1, BLOCK).amax((1, 3)), "e4m3")
            for k, (x, power) in enumerate(((p.double(), e), (p.double().t(), e.t()))):
                at, n, sat, sn = s["places"][2 * i + k]
                got = _defined(x, "e4m3", power.repeat_interleave(BLOCK, 0)[:x.shape[0]])
                codes[at:at + n], scales[sat:sat + sn] = got[0].reshape(-1), got[1].reshape(-1)
        return [codes, scales]
    c = _values(s["a_codes"], s["a_scales"], s["k"]) @ _values(s["b_codes"], s["b_scales"], s["k"]).t()
    return [c + s["c"].double() if case["add"] else c]
