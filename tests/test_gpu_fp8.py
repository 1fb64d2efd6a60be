"""The operators of a layer in 8 bits on the GPU against the fp64 oracle:
codes and scales bit for bit, products of whole numbers exactly, and elsewhere
bounds that count the roundings along the formula."""
import numpy as np
import pytest

from oracle import fp8_oracle as O
from second_order_optimizer_amd import adamw as A
from second_order_optimizer_amd import shampoo as S

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from second_order_optimizer_amd import fp8 as F  # noqa: E402

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {t: torch.finfo(TORCH[t]).eps / 2 for t in TORCH}
U = 2.0 ** -24                       # half a step of fp32
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SENTINEL = 0x5A


def np64(t):
    return t.detach().double().cpu().numpy()


class Held:
    """A Matrix8 between guard bytes: rows `pitch` bytes apart, scales `apart`
    words from group to group, all of it first filled with a sentinel."""

    def __init__(self, rows, cols, fmt="e4m3", more=0, apart=0):
        blocks = -(-cols // 128)
        self.groups, self.pitch, self.apart = -(-blocks // 4), blocks * 128 + 16 * more, rows + apart
        self.rows, self.cols, self.width, self.fmt = rows, cols, blocks * 128, fmt
        self.craw = torch.full((64 + rows * self.pitch + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.sraw = torch.full((64 + self.groups * self.apart * 4 + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
        codes = self.craw[64:64 + rows * self.pitch].view(rows, self.pitch)[:, :self.width].view(CODES[fmt])
        scales = self.sraw[64:64 + self.groups * self.apart * 4].view(self.groups, self.apart, 4)[:, :rows]
        self.m = F.Matrix8(rows, cols, fmt, codes=codes, scales=scales)

    def codes(self):
        return self.m.codes.view(torch.uint8).cpu().numpy()

    def scales(self):
        return self.m.scales.cpu().numpy()

    def values(self):
        return O.values(self.codes(), self.scales(), self.cols, self.fmt)

    def untouched(self):
        """Everything but the codes and the scales that rows have."""
        c, s = self.craw.cpu().numpy().copy(), self.sraw.cpu().numpy().copy()
        if self.rows and self.cols:
            c[64:64 + self.rows * self.pitch].reshape(self.rows, self.pitch)[:, :self.width] = SENTINEL
            has = O.grouped(np.zeros((self.rows, -(-self.cols // 128)), np.int64))[1]
            s[64:64 + self.groups * self.apart * 4].reshape(self.groups, self.apart, 4)[:, :self.rows][has] = SENTINEL
        assert np.all(c == SENTINEL) and np.all(s == SENTINEL)

    def check(self, codes, e):
        got = self.codes()
        v = O.code_values(self.fmt)
        nan = np.isnan(v[codes])
        np.testing.assert_array_equal(np.isnan(v[got]), nan)      # the sign of a NaN says nothing
        np.testing.assert_array_equal(got[~nan], codes[~nan])
        want, has = O.grouped(e)
        np.testing.assert_array_equal(self.scales()[has], want[has])
        self.untouched()


def wide(values, dtype, pad=0, offset=0):
    """Rows in a buffer of NaNs, `pad` elements wider, from element `offset` on."""
    rows, cols = values.shape
    buf = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=TORCH[dtype], device="cuda")
    t = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(np.ascontiguousarray(values)))
    return t, buf


def beside(t, buf):
    """That nothing but t's elements was written: the rest are NaN still."""
    rest = buf.clone()
    rest.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(float("nan"))
    assert bool(torch.isnan(rest).all())


def spread(rng, rows, cols, decades=2.0):
    return rng.standard_normal((rows, cols)) * 10 ** rng.uniform(-decades, decades, (rows, 1)) * 10 ** rng.uniform(-decades, decades, (1, cols))


SHAPES = [(1, 1), (1, 128), (1, 1000), (3, 7), (127, 129), (128, 128), (129, 127), (130, 640), (257, 513), (1000, 30)]


# ------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(dtype, shape):
    rng = np.random.default_rng(sum(shape))
    rows, cols = shape
    for n, (fr, fc, pad, offset) in enumerate((("e4m3", "e4m3", 0, 0), ("e5m2", "e4m3", 3, 1), ("e4m3", "e5m2", 8, 5), ("e5m2", "e5m2", 1, 0))):
        x, buf = wide(spread(rng, rows, cols), dtype, pad, offset)
        v = np64(x)
        a, b = Held(rows, cols, fr, n, n), Held(cols, rows, fc, n, 2 * n)
        F.quantize(x, rows=a.m, cols=b.m)
        a.check(*O.encode(v, fr))
        b.check(*O.encode(v.T, fc))
        a2, b2 = Held(rows, cols, fr), Held(cols, rows, fc)
        F.quantize(x, rows=a2.m)
        F.quantize(x, cols=b2.m)
        a2.check(*O.encode(v, fr))
        b2.check(*O.encode(v.T, fc))
        beside(x, buf)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_border(fmt):
    """Each code's value, the middles between codes, and their fp32 neighbours,
    in blocks whose largest value leaves the scale at 2^e."""
    v = O.code_values(fmt)[:128]
    v = v[np.isfinite(v)]
    mid = (v[1:] + v[:-1]) / 2
    y = np.concatenate([v, mid]).astype(np.float32)
    y = np.concatenate([y, np.nextafter(y, np.float32(np.inf)), np.nextafter(y, np.float32(0))])
    y = y[y <= v[-1]]
    y = np.concatenate([y, -y])
    y = np.concatenate([y, np.zeros(-len(y) % 127, np.float32)]).reshape(-1, 127)
    x = np.concatenate([np.full((len(y), 1), v[-1], np.float32), y], 1)     # the largest, then 127 of them
    for e in (-100, 0, 60):
        z = np.ldexp(x, e)
        t, _ = wide(z, "f32")
        a, b = Held(len(x), 128, fmt), Held(128, len(x), fmt)
        F.quantize(t, rows=a.m, cols=b.m)
        codes, exps = O.encode(z, fmt)
        assert np.all(exps == e)
        a.check(codes, exps)
        b.check(*O.encode(z.T, fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_at_their_borders(fmt):
    """Blocks of one size, from the smallest fp32 number to the largest, at and
    next to the size where the scale steps; and a block of zeros."""
    top = 1.75
    sizes = [0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 2.0 ** -120, 2.0 ** -100, 3.4028234663852886e38]
    for e in (-119, -118, -117, -112, -111, -20, 0, 20, 127):
        s = np.float32(np.ldexp(top, e))
        sizes += [s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(np.inf))]
    x = np.outer(np.array(sizes), np.r_[1.0, -0.5, np.linspace(-1, 1, 126)]).astype(np.float32)
    t, _ = wide(x, "f32")
    a, b = Held(len(x), 128, fmt), Held(128, len(x), fmt)
    F.quantize(t, rows=a.m, cols=b.m)
    a.check(*O.encode(x.astype(np.float64), fmt))
    b.check(*O.encode(x.T.astype(np.float64), fmt))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_not_finite(dtype, fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 300))
    x[0, 0], x[0, 200], x[5, 17], x[199, 299], x[130] = np.inf, np.nan, -np.inf, np.nan, np.nan
    x[:, 40] = -np.inf
    t, _ = wide(x, dtype)
    v = np64(t)
    a, b = Held(200, 300, fmt), Held(300, 200, fmt)
    F.quantize(t, rows=a.m, cols=b.m)
    a.check(*O.encode(v, fmt))
    b.check(*O.encode(v.T, fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", SHAPES)
def test_transpose(shape, fmt):
    rng = np.random.default_rng(7)
    rows, cols = shape
    x, _ = wide(spread(rng, rows, cols, 3.0), "f32")
    a = Held(rows, cols, fmt, 2, 3)
    F.quantize(x, rows=a.m)
    for to in ("e4m3", "e5m2"):
        b = Held(cols, rows, to, 1, 1)
        F.transpose(a.m, b.m)
        b.check(*O.encode(a.values().T, to))
        a.untouched()


def test_transpose_of_what_is_not_finite_and_of_part():
    x, _ = wide(np.random.default_rng(2).standard_normal((300, 500)), "f32")
    x[3, 4], x[200, 499], x[299] = float("nan"), float("inf"), float("nan")
    for fmt in ("e4m3", "e5m2"):
        a, b = Held(300, 500, fmt), Held(500, 155, fmt)
        F.quantize(x, rows=a.m)
        F.transpose(a.m.between(145, 300), b.m)
        b.check(*O.encode(a.values()[145:300].T, fmt))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_weights(dtype):
    rng = np.random.default_rng(4)
    shapes = [(128, 128), (1, 1), (0, 5), (130, 700), (7, 3), (5, 0), (257, 100), (1, 1000), (640, 1)]
    vals = [spread(rng, r, c, 1.0) for r, c in shapes]
    vals[3][0, 0], vals[3][129, 699], vals[6][3, :] = np.nan, np.inf, 0.0
    ts = [torch.from_numpy(v).to(TORCH[dtype]).cuda() for v in vals]
    w = F.Weights8(shapes, param=dtype)
    w.bind(ts)
    for _ in range(2):
        w.refresh()
        for t, a, b, (r, c) in zip(ts, w.rows, w.cols, shapes):
            (ca, ea), (cb, eb) = O.encode_weight(np64(t)) if r and c else ((np.zeros((r, -(-c // 128) * 128)), None), (np.zeros((c, -(-r // 128) * 128)), None))
            for m, codes, e in ((a, ca, ea), (b, cb, eb)):
                got = m.codes.view(torch.uint8).cpu().numpy()
                nan = np.isnan(O.code_values("e4m3")[codes.astype(np.uint8)])
                np.testing.assert_array_equal(np.isnan(O.code_values("e4m3")[got]), nan)
                np.testing.assert_array_equal(got[~nan], codes[~nan])
                if e is not None:
                    np.testing.assert_array_equal(m.scales.cpu().numpy(), np.where(O.grouped(e)[1], O.grouped(e)[0], 0))
        for t in ts:
            t.mul_(-3.7)


def test_weights_past_one_binding_launch():
    n = 900
    ts = [torch.full((3, 5), float(i + 1), device="cuda") for i in range(n)]
    w = F.Weights8([(3, 5)] * n)
    w.bind(ts)
    w.refresh()
    first = np.array([O.values(m.codes.view(torch.uint8).cpu().numpy(), m.scales.cpu().numpy(), 5, "e4m3")[2, 4] for m in w.rows[::37]])
    want = np.arange(1, n + 1)[::37].astype(np.float64)
    assert np.all(np.abs(first - want) <= O.HALF["e4m3"] * want)
    assert first[0] == 1.0


# ------------------------------------------------------------ norm
def depth(dim):
    """Roundings of a row's sum: a thread's own terms one after another (16 of
    them, or what a thread of 1024 meets in a longer row), six steps across the
    wave, and at most sixteen waves."""
    return 8 * max(2, -(-dim // 8192)) + 6 + 16


def check8(h8, h, rel):
    """An 8-bit matrix against exact values, of which the kernel rounded ones
    within `rel` of them."""
    got = h8.values()
    codes, e = O.encode(h, "e4m3")
    byte, has = O.grouped(e)
    sc = h8.scales()
    rows, nb = e.shape
    for b in range(nb):
        s = sc[b // 4, :, b % 4].astype(int) - 127
        big = np.abs(h[:, b * 128:(b + 1) * 128]).max(1)
        fits = lambda x: O.exponents(x, "e4m3")  # noqa: E731
        assert np.all((s >= fits(big * (1 - rel))) & (s <= fits(big * (1 + rel))))
        part = slice(b * 128, min((b + 1) * 128, h.shape[1]))
        a = np.abs(h[:, part])
        tol = np.maximum(O.HALF["e4m3"] * a * (1 + rel), O.HALF_LOW["e4m3"] * np.ldexp(1.0, s)[:, None]) + rel * a
        assert np.all(np.abs(got[:, part] - h[:, part]) <= tol)
    padded = h8.codes().reshape(rows, -1)[:, h.shape[1]:]
    assert np.all(padded == 0)
    h8.untouched()


NORM_DIMS = [1, 7, 128, 500, 512, 513, 1000, 1025, 2048, 2050, 4096, 4100, 8192, 8193, 16384, 16391, 40000]


@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("x_type,res_type", [("bf16", "bf16"), ("f32", None), ("f16", "f32"), ("f32", "f16"), ("bf16", None)])
def test_norm(dim, x_type, res_type):
    rng = np.random.default_rng(dim)
    eps = 1e-5
    for rows, pad, offset, w_type in ((1, 0, 0, "f32"), (5, 3, 1, "bf16"), (9, 8, 0, "f16")):
        x, xb = wide(2 * rng.standard_normal((rows, dim)), x_type, pad, offset)
        w = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).to(TORCH[w_type]).cuda()
        res = total = tb = None
        if res_type:
            res, rb = wide(rng.standard_normal((rows, dim)), res_type, pad, offset)
            total, tb = wide(np.zeros((rows, dim)), res_type, pad + 1, offset)
        out, ob = wide(np.zeros((rows, dim)), "f32", pad, 1)
        rstd = torch.full((rows + 2,), -1.0, device="cuda")
        h8 = Held(rows, dim, "e4m3", 1, 1)
        F.rms_norm(x, w, eps, residual=res, total=total, out8=h8.m, out=out, rstd=rstd[1:1 + rows])
        z = np64(x)
        if res_type:
            s = z + np64(res)
            z = np64(total)
            assert np.all(np.abs(z - s) <= (HALF[res_type] + 2 * U) * np.abs(s) + 2.0 ** -25 * (res_type == "f16"))
            beside(total, tb)
            beside(res, rb)
        r, h = O.rms_norm(z, np64(w), eps)
        rel_r = U * (depth(dim) / 2 + 1 + 3)     # the sum's roundings count half in a root; mean and eps; root, quotient
        got_r = np64(rstd)
        assert got_r[0] == got_r[-1] == -1.0
        assert np.all(np.abs(got_r[1:-1] - r) <= rel_r * r)
        rel = rel_r + 3 * U
        assert np.all(np.abs(np64(out) - h) <= rel * np.abs(h))
        check8(h8, h, rel)
        beside(x, xb)
        beside(out, ob)


@pytest.mark.parametrize("out_type", ["bf16", "f16"])
def test_norm_wide_alone(out_type):
    rng = np.random.default_rng(0)
    x, _ = wide(rng.standard_normal((33, 1003)), "bf16")
    w = torch.ones(1003, device="cuda")
    out, ob = wide(np.zeros((33, 1003)), out_type, 5, 3)
    F.rms_norm(x, w, 1e-6, out=out)
    h = O.rms_norm(np64(x), np.ones(1003), 1e-6)[1]
    tol = HALF[out_type] * (1 + 2.0 ** -10) + U * (depth(1003) / 2 + 7)
    assert np.all(np.abs(np64(out) - h) <= tol * np.abs(h) + 2.0 ** -25 * (out_type == "f16"))
    beside(out, ob)


@pytest.mark.parametrize("dim", [96, 1000, 5000, 20000])
def test_norm_in_place(dim):
    """The sum over the residual, or over x: as into memory of its own."""
    rng = np.random.default_rng(dim)
    x, _ = wide(rng.standard_normal((6, dim)), "f32", 2)
    res, _ = wide(rng.standard_normal((6, dim)), "f32", 4)
    w = torch.from_numpy(rng.standard_normal(dim)).float().cuda()
    z, h = torch.empty_like(res), Held(6, dim)
    F.rms_norm(x, w, 1e-6, residual=res, total=z, out8=h.m)
    for over in ("res", "x"):
        x2, xb = wide(np64(x), "f32", 2)
        r2, rb = wide(np64(res), "f32", 4)
        g = Held(6, dim)
        F.rms_norm(x2, w, 1e-6, residual=r2, total=r2 if over == "res" else x2, out8=g.m)
        assert torch.equal(r2 if over == "res" else x2, z)
        assert torch.equal(x2 if over == "res" else r2, x if over == "res" else res)
        np.testing.assert_array_equal(g.codes(), h.codes())
        beside(x2, xb)
        beside(r2, rb)


def test_norm_of_odd_rows():
    """Rows of zeros, of NaN, with an infinity, of the largest and of tiny values."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 300)).astype(np.float32)
    x[1] = 0
    x[2, 7] = np.nan
    x[3, 299] = np.inf
    x[4] = 3e38          # the squares' sum leaves fp32, not 64 bits
    x[5] = 1e-30         # eps is all that is left
    t, _ = wide(x, "f32")
    w = torch.ones(300, device="cuda")
    h8, r = Held(7, 300), torch.empty(7, device="cuda")
    F.rms_norm(t, w, 1e-6, out8=h8.m, rstd=r)
    v = h8.values()
    rr = np64(r)
    assert np.all(v[1] == 0) and np.all(np.isnan(v[2])) and np.isnan(rr[2]) and rr[3] == 0
    assert np.isnan(v[3, 299]) and np.all(v[3, :299] == 0)
    assert np.all(v[4] == 1.0) and abs(rr[4] * 3e38 - 1) < 1e-6      # fp32 holds 1 / 3e38 in 21 bits
    assert abs(rr[1] - 1e3) <= 1e3 * 4 * U and abs(rr[5] - 1e3) <= 1e3 * 4 * U
    assert np.all(np.abs(v[5] - 1e-27) <= O.HALF["e4m3"] * 1.01e-27)
    assert np.all(np.isfinite(v[[0, 6]]))
    assert np.all(h8.codes()[:, 300:] == 0)      # behind the last column, in every row


@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("g_type,z_type,add", [("bf16", "bf16", True), ("f32", "f32", False), ("f16", "f32", True), ("f32", "f16", True), ("bf16", "f32", True)])
def test_norm_backward(dim, g_type, z_type, add):
    rng = np.random.default_rng(dim + 1)
    for rows, pad, offset, w_type in ((1, 0, 0, "f32"), (6, 3, 1, "bf16"), (4097 if dim < 600 else 1100 if dim < 3000 else 40, 0, 0, "f32")):
        g, gb = wide(rng.standard_normal((rows, dim)) * 10 ** rng.uniform(-1, 1, (rows, 1)), g_type, pad, offset)
        z, zb = wide(rng.standard_normal((rows, dim)), z_type, pad, offset)
        q = wide(rng.standard_normal((rows, dim)), z_type, pad + 2, offset)[0] if add else None
        w = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).to(TORCH[w_type]).cuda()
        r = torch.from_numpy(O.rms_norm(np64(z), np64(w), 1e-5)[0]).float().cuda()
        dz, db = wide(np.zeros((rows, dim)), z_type, pad + 1, offset)
        dw = torch.full((dim + 2,), 7.0, device="cuda")
        F.rms_norm_backward(g, z, r, w, dz=dz, add=q, dw=dw[1:1 + dim])
        g64, z64, r64, w64 = np64(g), np64(z), np64(r), np64(w)
        want, want_dw = O.rms_norm_backward(g64, z64, r64, w64, None if q is None else np64(q))
        a, unit = np.abs(g64 * w64), np.abs(z64) * r64[:, None]
        # a, unit: a rounding each; their products' mean: the sum's, two of the terms, two of the mean; then four
        mean = (a * unit).mean(1, keepdims=True)
        tol = U * (r64[:, None] * (4 * a + unit * mean * (depth(dim) + 10)) + 4 * np.abs(want) + (0 if q is None else np.abs(np64(q))))
        tol = tol + HALF[z_type] * (np.abs(want) + tol) + 2.0 ** -25 * (z_type == "f16")
        assert np.all(np.abs(np64(dz) - want) <= tol)
        # dw: a rounding of each term, one for each further row of a slot, 31 + 31 and more in the slots' sum
        turns = -(-rows // 64) + 130
        assert np.all(np.abs(np64(dw)[1:-1] - want_dw) <= U * (2 + turns) * (np.abs(g64) * unit).sum(0))
        assert float(dw[0]) == float(dw[-1]) == 7.0
        beside(dz, db)
        beside(g, gb)
        beside(z, zb)
        before = dw.clone()
        dz2 = torch.empty_like(dz)
        F.rms_norm_backward(g, z, r, w, dz=dz2, add=q, dw=dw[1:1 + dim], accumulate=True)
        assert torch.equal(dz2, dz)
        assert torch.equal(dw[1:-1], before[1:-1] + before[1:-1])     # doubling rounds nothing
        dz2.zero_()
        F.rms_norm_backward(g, z, r, w, dz=dz2, add=q)
        assert torch.equal(dz2, dz)


@pytest.mark.parametrize("dim", [96, 1000, 5000, 20000])
def test_norm_backward_in_place(dim):
    rng = np.random.default_rng(dim)
    mk = lambda pad: wide(rng.standard_normal((5, dim)), "f32", pad)[0]  # noqa: E731
    g, z, q, w = mk(1), mk(2), mk(3), torch.ones(dim, device="cuda")
    r = torch.rand(5, device="cuda") + 0.5
    dz, dw = torch.empty_like(z), torch.empty(dim, device="cuda")
    F.rms_norm_backward(g, z, r, w, dz=dz, add=q, dw=dw)
    for name in ("g", "z", "q"):
        t = {"g": g.clone(), "z": z.clone(), "q": q.clone()}
        dw2 = torch.empty_like(dw)
        F.rms_norm_backward(t["g"], t["z"], r, w, dz=t[name], add=t["q"], dw=dw2)
        assert torch.equal(t[name], dz) and torch.equal(dw2, dw)


def test_norm_backward_without_rows():
    e = torch.empty(0, 5, device="cuda")
    dw = torch.full((5,), 3.0, device="cuda")
    F.rms_norm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(5, device="cuda"), dz=e, dw=dw, accumulate=True)
    assert torch.all(dw == 3)
    F.rms_norm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(5, device="cuda"), dz=e, dw=dw)
    assert torch.all(dw == 0)


# ------------------------------------------------------------ product
def whole(rng, rows, cols, fmt, more=0, apart=0, powers=3):
    """An 8-bit matrix of whole numbers up to 7 times 1 to 2^powers by block."""
    m = Held(rows, cols, fmt, more, apart)
    top = 7 if fmt == "e4m3" else 4
    v = np.zeros((rows, m.width))
    v[:, :cols] = rng.integers(-top, top + 1, (rows, cols))
    e = rng.integers(0, powers + 1, (rows, m.width // 128))
    m.m.codes.view(torch.uint8).copy_(torch.from_numpy(O.nearest(v, fmt)).view(rows, -1))
    byte, has = O.grouped(e)
    s = m.m.scales
    s.copy_(torch.from_numpy(np.where(has, byte, SENTINEL)))
    return m


def random8(rng, rows, cols, fmt, decades=0.5):
    x, _ = wide(spread(rng, rows, cols, decades), "f32")
    m = Held(rows, cols, fmt)
    F.quantize(x, rows=m.m)
    return m


PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 1000, 1000), (2, 300, 129), (15, 17, 640), (16, 256, 512), (17, 257, 300), (33, 64, 2000),
            (64, 4096, 130), (65, 1, 1025), (100, 3, 5000), (128, 128, 128), (129, 255, 384), (200, 777, 1030), (256, 256, 256),
            (257, 513, 640), (300, 500, 0), (511, 1, 77), (600, 1300, 1500), (1, 5, 20000), (48, 96, 30000), (1024, 512, 8200),
            # every size of tile, whole and with ragged ends, and sums in parts
            (2048, 2048, 256), (2049, 2100, 300), (4100, 4001, 129), (4096, 4096, 128), (4099, 4103, 1152), (2300, 4600, 1400), (4000, 4090, 1930), (513, 520, 33000)]


@pytest.mark.parametrize("mnk", PRODUCTS)
def test_product_of_whole_numbers(mnk):
    """Terms and sums that fp32 holds exactly: the result is exact, rounded once
    where the output's type needs it."""
    m, n, k = mnk
    rng = np.random.default_rng(m + n + k)
    for i, (fa, fb, out, pad, offset, add) in enumerate((("e4m3", "e4m3", "f32", 0, 0, False), ("e5m2", "e4m3", "bf16", 3, 1, False),
                                                         ("e4m3", "e5m2", "f32", 1, 3, True), ("e5m2", "e5m2", "bf16", 8, 0, True),
                                                         ("e4m3", "e4m3", "f16", 2, 2, False))):
        powers = 3 if k < 8000 and out != "f16" else 0
        a, b = whole(rng, m, k, fa, i, i, powers), whole(rng, n, k, fb, 2 * i, i, powers)
        va, vb = a.values(), b.values()
        assert np.all(np.abs(va) @ np.abs(vb).T < 2 ** 24 - 4096)
        want = va @ vb.T
        old = rng.integers(-50, 50, (m, n)).astype(np.float64)
        c, buf = wide(old, out, pad, offset)
        F.matmul(a.m, b.m, c, accumulate=add)
        want = torch.from_numpy(want + old if add else want).to(TORCH[out])
        assert torch.equal(c.cpu(), want)
        beside(c, buf)


@pytest.mark.parametrize("mnk", [(1, 700, 1000), (5, 64, 4096), (40, 500, 3000), (130, 300, 700), (512, 512, 2048), (300, 200, 9000)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_product(mnk, fa, fb):
    """fp32: every addition is off by at most 2^-23 of the sum of magnitudes (a
    step, should the matrix unit cut off rather than round), K of them and the
    joining of parts.  16 bits: the 8-bit instructions also cut each product of
    eight below 2^-13 of the largest of them, seven of them 7 * 2^-13 of the
    largest and so of the eight's magnitudes; then the output's rounding."""
    m, n, k = mnk
    rng = np.random.default_rng(k)
    a, b = random8(rng, m, k, fa), random8(rng, n, k, fb)
    va, vb = a.values(), b.values()
    want, most = va @ vb.T, np.abs(va) @ np.abs(vb).T
    for out in ("f32", "bf16"):
        c = torch.full((m, n), float("nan"), dtype=TORCH[out], device="cuda")
        F.matmul(a.m, b.m, c)
        tol = ((k + 64) * 2 * U + (0 if out == "f32" else 7 * 2.0 ** -13)) * most
        assert np.all(np.abs(np64(c) - want) <= tol + HALF[out] * (np.abs(want) + tol))
        # and as sums of that many terms go, not as the worst could
        assert np.sqrt(np.mean((np64(c) - want) ** 2)) <= (HALF[out] + 8 * U) * np.sqrt(np.mean(most ** 2))


def test_product_range_and_not_finite():
    """Scales at both ends, zeros against them, NaN and infinities to where they belong."""
    for fmt in ("e4m3", "e5m2"):
        a, b = Held(4, 256, fmt), Held(3, 256, fmt)
        for h in (a, b):
            h.m.codes.view(torch.uint8).fill_(int(O.nearest(1.0, fmt)))
            h.m.scales.fill_(127)
        a.m.scales[0, 1, :2], b.m.scales[0, 1, :2] = 127 + 60, 127 - 60
        a.m.scales[0, 2, :2] = 254
        a.m.codes.view(torch.uint8)[2].fill_(0)
        a.m.codes.view(torch.uint8)[3, 77] = 0x7F
        c = torch.empty(4, 3, device="cuda")
        F.matmul(a.m, b.m, c)
        c = np64(c)
        assert c[0].tolist() == [256, 256 * 2.0 ** -60, 256] and c[1].tolist() == [256 * 2.0 ** 60, 256, 256 * 2.0 ** 60]
        assert c[2].tolist() == [0, 0, 0] and np.all(np.isnan(c[3]))
        if fmt == "e5m2":
            a.m.codes.view(torch.uint8)[3, 77] = 0xFC
            d = torch.empty(4, 3, device="cuda")
            F.matmul(a.m, b.m, d)
            assert np.all(np.isneginf(np64(d)[3])) and np.array_equal(np64(d)[:3], c[:3])


def test_product_of_parts_and_of_itself():
    rng = np.random.default_rng(5)
    a = whole(rng, 300, 1000, "e4m3", 1, 5, 1)
    b = whole(rng, 200, 1000, "e4m3", 0, 0, 1)
    va, vb = a.values(), b.values()
    c = torch.zeros(70, 50, device="cuda")
    F.matmul(a.m.between(131, 201), b.m.between(7, 57), c)
    assert np.array_equal(np64(c), va[131:201] @ vb[7:57].T)
    d = torch.zeros(300, 300, device="cuda")
    F.matmul(a.m, a.m, d)
    assert np.array_equal(np64(d), va @ va.T)


def test_product_without_terms():
    a, b = F.Matrix8(5, 0), F.Matrix8(7, 0)
    c = torch.full((5, 7), 3.0, device="cuda")
    F.matmul(a, b, c, accumulate=True)
    assert torch.all(c == 3)
    F.matmul(a, b, c)
    assert torch.all(c == 0)
    F.matmul(F.Matrix8(0, 9), F.Matrix8(7, 9), torch.empty(0, 7, device="cuda"))


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes and elements: what lies at their ends."""
    rows, cols = 33000, 131200
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, cols, device="cuda").bfloat16()
    x[:, -5:] = torch.randn(rows, 5, device="cuda").bfloat16()
    a, b = F.Matrix8(rows, cols), F.Matrix8(cols, rows)
    F.quantize(x, rows=a, cols=b)
    v = np64(x[-130:])
    codes, e = O.encode(v, "e4m3")
    np.testing.assert_array_equal(a.codes[-130:].view(torch.uint8).cpu().numpy(), codes)
    byte, has = O.grouped(e)
    np.testing.assert_array_equal(a.scales[:, -130:].cpu().numpy()[has], byte[has])
    codes, e = O.encode(np64(x[:, -140:]).T, "e4m3")
    np.testing.assert_array_equal(b.codes[-140:].view(torch.uint8).cpu().numpy(), codes)
    t = F.Matrix8(cols, rows)
    F.transpose(a, t)
    held = O.values(a.codes.view(torch.uint8)[:, -128:].cpu().numpy(), a.scales[-1:, :, cols // 128 % 4 - 1:].cpu().numpy(), 128, "e4m3")
    codes, _ = O.encode(held.T, "e4m3")
    np.testing.assert_array_equal(t.codes[-128:].view(torch.uint8).cpu().numpy(), codes)
    del t
    # products of the last rows, each kind of kernel by the number of rows
    va = O.values(a.codes[-2:].view(torch.uint8).cpu().numpy(), a.scales[:, -2:].cpu().numpy(), cols, "e4m3")
    want, most = va @ va.T, np.abs(va) @ np.abs(va).T
    for many in (2, 100, 700):
        c = torch.empty(many, many, device="cuda")
        F.matmul(a.between(rows - many, rows), a.between(rows - many, rows), c)
        assert np.all(np.abs(np64(c)[-2:, -2:] - want) <= (cols + 64) * 2 * U * most)
    out, w = torch.empty_like(x), torch.ones(cols, device="cuda")
    F.rms_norm(x, w, 1e-6, out8=a, out=out)
    h = O.rms_norm(v[-3:], np.ones(cols), 1e-6)[1]
    assert np.all(np.abs(np64(out[-3:]) - h) <= HALF["bf16"] * (1 + 2.0 ** -10) * np.abs(h))
    big = torch.empty(66000, 66000, dtype=torch.bfloat16, device="cuda")       # 2^32 elements of C
    m = F.Matrix8(66000, 130)
    m.codes.view(torch.uint8)[-1, :130] = int(O.nearest(1.0, "e4m3"))
    m.scales[0, -1, :2] = 127
    F.matmul(m, m, big)
    assert float(big[-1, -1]) == 130.0 and float(big[-1, -2]) == 0.0 and float(big[0, 0]) == 0.0


# ------------------------------------------------------------ together
class Layer:
    """A norm and a linear layer in 8 bits with everything that its step needs."""

    def __init__(self, tokens, width, out, seed=0, dtype="bf16"):
        rng = np.random.default_rng(seed)
        t = lambda *s, dt=dtype: torch.from_numpy(rng.standard_normal(s)).to(TORCH[dt]).cuda()  # noqa: E731
        self.x, self.res, self.dy = t(tokens, width), t(tokens, width, dt="f32"), t(tokens, out)
        self.gain = 1 + 0.1 * t(width, dt="f32")
        self.w = 0.05 * t(out, width, dt="f32")
        self.more = t(tokens, width, dt="f32")
        self.w8 = F.Weights8([(out, width)])
        self.w8.bind([self.w])
        self.h8, self.ht8 = F.Matrix8(tokens, width), F.Matrix8(width, tokens)
        self.d8, self.dt8 = F.Matrix8(tokens, out, "e5m2"), F.Matrix8(out, tokens, "e5m2")
        self.z, self.r = torch.empty_like(self.res), torch.empty(tokens, device="cuda")
        self.y, self.dh = torch.empty(tokens, out, dtype=TORCH[dtype], device="cuda"), torch.empty(tokens, width, dtype=TORCH[dtype], device="cuda")
        self.dz, self.dw, self.dgain = torch.empty_like(self.res), torch.zeros(out, width, device="cuda"), torch.empty(width, device="cuda")

    def run(self):
        self.w8.refresh()
        F.rms_norm(self.x, self.gain, 1e-6, residual=self.res, total=self.z, out8=self.h8, rstd=self.r)
        F.matmul(self.h8, self.w8.rows[0], self.y)
        F.quantize(self.dy, rows=self.d8, cols=self.dt8)
        F.matmul(self.d8, self.w8.cols[0], self.dh)
        F.transpose(self.h8, self.ht8)
        F.matmul(self.dt8, self.ht8, self.dw)
        F.rms_norm_backward(self.dh, self.z, self.r, self.gain, add=self.more, dz=self.dz, dw=self.dgain)
        return [self.y, self.dh, self.dw, self.dz, self.dgain, self.z, self.r]


@pytest.mark.parametrize("tokens,width,out", [(1, 128, 64), (77, 300, 200), (600, 1024, 512)])
def test_layer_against_the_formulas(tokens, width, out):
    """The whole chain in fp64 from the inputs; each rounding to 8 bits is off by
    half a step of its block's values at most, so a sum of them is, too."""
    s = Layer(tokens, width, out)
    y, dh, dw, dz, dgain, z, r = (np64(v) for v in s.run())
    z64 = np64(s.x) + np64(s.res)
    r64, h = O.rms_norm(z64, np64(s.gain), 1e-6)
    w, dy = np64(s.w), np64(s.dy)
    rel4, rel5 = O.HALF["e4m3"] * 1.01, O.HALF["e5m2"] * 1.01
    low4 = lambda v: np.abs(v).max() * 2.0 ** -17  # noqa: E731  below 2^-6 of the scale: half of 2^-9 of 2^e <= max / 224
    ah, aw, ad = np.abs(h) + low4(h), np.abs(w) + low4(w), np.abs(dy)
    far = lambda p, q, a, b: a + b + a * b  # noqa: E731
    e = far(0, 0, rel4, rel4)
    assert np.all(np.abs(y - h @ w.T) <= (e + 2.0 ** -8) * 1.01 * (ah @ aw.T))
    e = far(0, 0, rel5, rel4)
    bound_dh = (e + 2.0 ** -8) * 1.01 * (ad @ aw)
    assert np.all(np.abs(dh - dy @ w) <= bound_dh)
    e4 = far(0, 0, rel4, 2 * rel4)                     # transposed: below the normal range rounded twice
    assert np.all(np.abs(dw - dy.T @ h) <= far(0, 0, rel5, e4) * 1.01 * (ad.T @ ah))
    want_dz, want_dg = O.rms_norm_backward(dy @ w, z64, r64, np64(s.gain), np64(s.more))
    unit = np.abs(z64) * r64[:, None]
    a = bound_dh * np.abs(np64(s.gain))
    assert np.all(np.abs(dz - want_dz) <= 1.01 * r64[:, None] * (a + unit * (a * unit).mean(1, keepdims=True)) + 1e-4 * (1 + np.abs(want_dz)))
    assert np.all(np.abs(dgain - want_dg) <= 1.01 * (bound_dh * unit).sum(0) + 1e-4)


def test_repeatable():
    s = Layer(333, 1000, 700)
    first = [v.clone() for v in s.run()]
    for _ in range(3):
        for a, b in zip(first, s.run()):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """Two graphs of the same layer objects' kind, replayed in turn with eager
    work between them, against eager runs of the same inputs."""
    layers = [Layer(200, 512, 384, seed=1), Layer(70, 1000, 130, seed=2)]
    for s in layers:
        s.run()
    torch.cuda.synchronize()
    graphs = []
    for s in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(4):
        for s in layers:
            s.x.mul_(-1.25 if turn % 2 else 0.8).add_(0.01)
            s.w.mul_(0.97)
        want = [[v.clone() for v in s.run()] for s in layers]
        for s in layers:
            for v in (s.y, s.dh, s.dw, s.dz, s.dgain, s.z, s.r):
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        busy = torch.randn(500, 500, device="cuda") @ torch.randn(500, 500, device="cuda")
        torch.cuda.synchronize()
        assert busy.shape == (500, 500)
        for s, w in zip(layers, want):
            for a, b in zip((s.y, s.dh, s.dw, s.dz, s.dgain, s.z, s.r), w):
                assert torch.equal(a, b)


def test_two_streams():
    """Two layers at once on streams of their own, and as alone."""
    layers = [Layer(900, 2000, 1000, seed=k) for k in range(2)]
    want = [[v.clone() for v in s.run()] for s in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(layers, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(layers, want):
        for a, b in zip((s.y, s.dh, s.dw, s.dz, s.dgain, s.z, s.r), w):
            assert torch.equal(a, b)


def test_steps_refresh_their_copies():
    """Shampoo and AdamW steps leave the copies those of the stepped weights."""
    s = Layer(64, 256, 128)
    s.run()
    opt = S.Shampoo([(128, 256, S.DENSE)], S.make_config(128, root_mode="auto"))
    vec = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    wide_w = torch.randn(300, 200, device="cuda").bfloat16()
    copies = F.Weights8([(300, 200)], param="bf16")
    copies.bind([wide_w])
    aopt = A.AdamW([A.tensor(256, param="bf16"), A.tensor(300 * 200, param="bf16")])
    aopt.bind([vec, wide_w.view(-1)], [torch.ones_like(vec), torch.randn(300 * 200, device="cuda").bfloat16()])
    for t in range(3):
        before = s.w.clone()
        s.run()
        opt.step([s.w], [s.dw], t, 2, copies8=s.w8)
        aopt.step(1e-2, copies8=copies)
        assert not torch.equal(before, s.w)
        for w, c in ((s.w, s.w8), (wide_w, copies)):
            fresh = F.Weights8([tuple(w.shape)], param="f32" if w.dtype == torch.float32 else "bf16")
            fresh.bind([w])
            fresh.refresh()
            assert torch.equal(fresh.codes.view(torch.uint8), c.codes.view(torch.uint8)) and torch.equal(fresh.scales, c.scales)
