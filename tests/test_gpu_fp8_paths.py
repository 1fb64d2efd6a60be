"""The 8-bit operators on the paths that only some sizes take: the norm and its
gradient over several turns of their workgroups, every kernel of the product
with random values, scales that differ by block, sums in parts, and values at
the ends of the range."""
import ctypes

import numpy as np
import pytest

from oracle import fp8_oracle as O
from second_order_optimizer_amd import shampoo as S
from test_gpu_fp8 import HALF, SENTINEL, TORCH, U, Held, beside, depth, np64, random8, wide

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from second_order_optimizer_amd import fp8 as F  # noqa: E402


# ------------------------------------------------------------ norm
@pytest.mark.parametrize("dim", [1, 7, 128, 500, 513, 1000, 1025, 2050, 4100, 8193, 16391, 40000])
@pytest.mark.parametrize("x_type,res_type", [("bf16", "bf16"), ("f32", None), ("f16", "f32")])
def test_norm_is_one_rounding_from_the_formula(dim, x_type, res_type):
    """Sum, root and products in 64 bits: a thread's chain of at most 40 terms,
    6 + 16 joins, eps, mean, root, quotient and two products, each off by 2^-53,
    are less than 2^-44 of the result, so r and h are off by one rounding to fp32
    and that; and the codes are those of h as it was rounded, bit for bit."""
    rng = np.random.default_rng(dim)
    one = U * (1 + 2.0 ** -20)
    for rows, w_type in ((1, "f32"), (37, "bf16")):
        x, _ = wide(rng.standard_normal((rows, dim)) * 10 ** rng.uniform(-4, 4, (rows, 1)), x_type, 1, 1)
        w = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).to(TORCH[w_type]).cuda()
        res = total = None
        if res_type:
            res, _ = wide(rng.standard_normal((rows, dim)), res_type, 2)
            total, _ = wide(np.zeros((rows, dim)), res_type, 3)
        out, r, h8 = torch.empty(rows, dim, device="cuda"), torch.empty(rows, device="cuda"), Held(rows, dim, "e4m3", 1, 1)
        F.rms_norm(x, w, 1e-6, residual=res, total=total, out8=h8.m, out=out, rstd=r)
        want_r, want = O.rms_norm(np64(x if total is None else total), np64(w), 1e-6)
        assert np.all(np.abs(np64(r) - want_r) <= one * want_r)
        assert np.all(np.abs(np64(out) - want) <= one * np.abs(want))
        h8.check(*O.encode(np64(out), "e4m3"))


# rows of as many waves as there are, so many that every workgroup takes at least
# three turns, the last one not in full
TURNS = [(300, 12300), (1000, 12299), (1500, 6200), (2048, 4500), (3000, 2100), (4096, 2101), (4100, 1300), (8192, 1301), (8193, 1299), (16384, 1030), (16391, 1300)]


@pytest.mark.parametrize("dim,rows", TURNS)
@pytest.mark.parametrize("g_type,z_type", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_norm_backward_over_turns(dim, rows, g_type, z_type):
    rng = np.random.default_rng(dim + rows)
    g, _ = wide(rng.standard_normal((rows, dim)) * 10 ** rng.uniform(-1, 1, (rows, 1)), g_type)
    z, _ = wide(rng.standard_normal((rows, dim)), z_type, 1)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).float().cuda()
    r = torch.from_numpy(O.rms_norm(np64(z), np64(w), 1e-5)[0]).float().cuda()
    dz, db = wide(np.zeros((rows, dim)), z_type, 2)
    dw = torch.empty(dim, device="cuda")
    F.rms_norm_backward(g, z, r, w, dz=dz, dw=dw)
    g64, z64, r64, w64 = np64(g), np64(z), np64(r), np64(w)
    want, want_dw = O.rms_norm_backward(g64, z64, r64, w64, None)
    a, unit = np.abs(g64 * w64), np.abs(z64) * r64[:, None]
    mean = (a * unit).mean(1, keepdims=True)
    tol = U * (r64[:, None] * (4 * a + unit * mean * (depth(dim) + 10)) + 4 * np.abs(want))
    assert np.all(np.abs(np64(dz) - want) <= tol + HALF[z_type] * (np.abs(want) + tol))
    # dw: a rounding of z r and one of each term as it is added, by the rows of a
    # group of waves, the 8 groups of a workgroup, a sixteenth of 512 slots, and 31
    assert np.all(np.abs(np64(dw) - want_dw) <= U * (1 + -(-rows // 512) + 8 + 16 + 31) * (1 + 2.0 ** -10) * (np.abs(g64) * unit).sum(0))
    beside(dz, db)
    old, again = dw.clone(), torch.empty_like(z)
    F.rms_norm_backward(g, z, r, w, dz=again, dw=dw, accumulate=True)
    assert torch.equal(again, dz) and torch.equal(dw, old + old)


@pytest.mark.parametrize("dim,rows", [(300, 6001), (2048, 2300), (16391, 600)])
def test_norm_backward_keeps_what_is_not_finite_to_its_row(dim, rows):
    """One infinity in grad, in a row that is not the last turn's: its row of dz
    and its element of dw, and no others."""
    rng = np.random.default_rng(dim)
    g, z = (torch.from_numpy(rng.standard_normal((rows, dim))).float().cuda() for _ in range(2))
    g[17, 5] = float("inf")
    dz, dw = torch.empty_like(z), torch.empty(dim, device="cuda")
    F.rms_norm_backward(g, z, torch.ones(rows, device="cuda"), torch.ones(dim, device="cuda"), dz=dz, dw=dw)
    bad = ~torch.isfinite(dz)
    assert bool(bad[17, 5]) and not bool(bad[:17].any()) and not bool(bad[18:].any())
    assert not bool(torch.isfinite(dw[5])) and int((~torch.isfinite(dw)).sum()) == 1


def test_transpose_of_the_largest_numbers():
    """The largest fp32 number rounds to a code that stands for 2^128, which
    transposes as an infinity: NaN in e4m3, and its neighbours as they were."""
    for fmt in ("e4m3", "e5m2"):
        x = torch.ones(130, 200, device="cuda")
        x[3], x[100, 7], x[129, 199] = 3.4028234663852886e38, -3.4028234663852886e38, 3e38
        a = Held(130, 200, fmt)
        F.quantize(x, rows=a.m)
        v = a.values().T
        assert v[5, 3] == 2.0 ** 128 and v[7, 100] == -2.0 ** 128 and v[199, 129] < 2.0 ** 128
        v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
        for to in ("e4m3", "e5m2"):
            b = Held(200, 130, to)
            F.transpose(a.m, b.m)
            b.check(*O.encode(v, to))


# ------------------------------------------------------------ product
def kind_sizes(k):
    """A product of k <= 300 for each kernel: one row of pieces and three of
    k_mul8_few's, and tiles of 64, 128 and 256."""
    assert 256 < k <= 300
    return [(4, 48, k), (40, 70, k), (100, 100, k), (1000, 2050, k), (2050, 4100, k)]


def parts_of(m, n, k, out):
    """The number of parts that a sum goes in, by the workspace."""
    need = ctypes.c_size_t()
    assert S.lib().shampoo_matmul8_workspace(m, n, k, {"f32": 0, "bf16": 1, "f16": 2}[out], ctypes.byref(need)) == 0
    return max(1, need.value // (4 * m * n))


def small(rng, rows, cols, fmt):
    """-1, 0 and 1 times 1, 2, 4 or 8 by block: sums of 33000 products are exact."""
    m = Held(rows, cols, fmt, 1, 1)
    v = np.zeros((rows, m.width))
    v[:, :cols] = rng.integers(-1, 2, (rows, cols))
    m.m.codes.view(torch.uint8).copy_(torch.from_numpy(O.nearest(v, fmt)).view(rows, -1))
    byte, has = O.grouped(rng.integers(0, 4, (rows, m.width // 128)))
    m.m.scales.copy_(torch.from_numpy(np.where(has, byte, SENTINEL)))
    return m


@pytest.mark.parametrize("mnk,out,tile", [((40, 100, 4200), "f32", 64), ((260, 260, 16500), "bf16", 64), ((260, 260, 16500), "f32", 64),
                                          ((1000, 1030, 8300), "bf16", 128), ((1000, 1030, 8300), "f32", 128), ((1000, 1030, 8300), "f16", 128),
                                          ((1000, 2050, 9000), "bf16", 256), ((1000, 4100, 8300), "bf16", 256), ((997, 2050, 8300), "f32", 256)])
def test_parts_begin_at_their_scales(mnk, out, tile):
    """Sums in parts by every kernel that takes them, with scales that differ from
    block to block: exact."""
    m, n, k = mnk
    assert parts_of(m, n, k, out) > 1
    rng = np.random.default_rng(m + n + k)
    for fa, fb, add in (("e4m3", "e4m3", False), ("e5m2", "e4m3", True)):
        a, b = small(rng, m, k, fa), small(rng, n, k, fb)
        va, vb = a.values(), b.values()
        want = va @ vb.T
        old = rng.integers(-50, 50, (m, n)).astype(np.float64)
        c, buf = wide(old, out, 3, 1)
        F.matmul(a.m, b.m, c, accumulate=add)
        assert torch.equal(c.cpu(), torch.from_numpy(want + old if add else want).to(TORCH[out]))
        beside(c, buf)


@pytest.mark.parametrize("mnk", kind_sizes(300))
def test_fp16_results_added(mnk):
    """c + A B^T in fp16 by each kernel: an exact sum, rounded once."""
    m, n, k = mnk
    rng = np.random.default_rng(m)
    for fa, fb in (("e4m3", "e4m3"), ("e4m3", "e5m2")):
        a, b = small(rng, m, k, fa), small(rng, n, k, fb)
        old = rng.integers(-50, 50, (m, n)).astype(np.float64)
        c, buf = wide(old, "f16", 1, 1)
        F.matmul(a.m, b.m, c, accumulate=True)
        assert torch.equal(c.cpu(), torch.from_numpy(a.values() @ b.values().T + old).to(torch.float16))
        beside(c, buf)


@pytest.mark.parametrize("mnk", [(1000, 2050, 300), (2050, 2100, 1100), (2050, 4100, 300), (2050, 4100, 1100), (1000, 1030, 8300), (1000, 2050, 9000)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_random_values_by_the_large_tiles(mnk, fa, fb):
    """fp32: K additions and the joining of parts, each off by at most 2^-23 of
    the sum of magnitudes; 16 bits: products of eight cut off below 2^-13 of the
    largest as well, at most 7 of them, then the output's rounding.  As they go,
    and not as the worst could, the sum of K such errors is far less."""
    m, n, k = mnk
    rng = np.random.default_rng(k + m)
    a, b = random8(rng, m, k, fa), random8(rng, n, k, fb)
    va, vb = a.values(), b.values()
    want, most = va @ vb.T, np.abs(va) @ np.abs(vb).T
    for out in ("f32", "bf16", "f16"):
        scaled = 1.0 if out != "f16" else 2.0 ** -np.ceil(np.log2(most.max() / 30000))     # into fp16's range, exactly
        if scaled != 1.0:
            a.m.scales.copy_((a.m.scales.to(torch.int32) + int(np.log2(scaled))).clamp_min(1).to(torch.uint8))
        ref, top = want * scaled, most * scaled
        c = torch.full((m, n), float("nan"), dtype=TORCH[out], device="cuda")
        F.matmul(a.m, b.m, c)
        err = np.abs(np64(c) - ref)
        tol = ((k + 64) * 2 * U + (0 if out == "f32" else 7 * 2.0 ** -13)) * top
        assert np.all(err <= tol + HALF[out] * (np.abs(ref) + tol) + (2.0 ** -25 if out == "f16" else 0))
        assert np.sqrt(np.mean(err ** 2)) <= (HALF[out] + 8 * U) * np.sqrt(np.mean(top ** 2)) + (2.0 ** -25 if out == "f16" else 0)


@pytest.mark.parametrize("mnk", kind_sizes(300))
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_ends_of_the_range_by_every_kernel(mnk, fmt, out):
    """Scales of 2^60 against 2^-60 and of 2^-127 against 2^127, zeros under the
    largest scale, NaN and infinities: to their rows and columns alone.  Where 299
    terms of 2^127 meet one of -infinity, two of them are 2^128, infinite in fp32:
    by the order of the additions the sum is -infinity or NaN."""
    m, n, k = mnk
    ones, big = int(O.nearest(1.0, fmt)), int(O.nearest(256.0, fmt))
    a, b = Held(m, k, fmt), Held(n, k, fmt)
    for h in (a, b):
        c8 = h.m.codes.view(torch.uint8)
        c8[:, :k], c8[:, k:] = ones, 0
        h.m.scales.fill_(127)
    ca = a.m.codes.view(torch.uint8)
    a.m.scales[:, m - 1], b.m.scales[:, n - 1] = 127 + 60, 127 - 60
    a.m.scales[:, m // 2], ca[m // 2] = 254, 0
    ca[0, 77] = 0x7F
    ca[1, :k], a.m.scales[:, 1] = big, 0
    b.m.scales[:, n // 2] = 254
    if fmt == "e5m2":
        ca[m - 2, k - 1] = 0xFC
    want = np.full((m, n), 300.0)
    want[m - 1] *= 2.0 ** 60
    want[1] *= 2.0 ** -119
    want[:, n - 1] *= 2.0 ** -60
    want[:, n // 2] *= 2.0 ** 127
    want[m // 2], want[0] = 0, np.nan
    if fmt == "e5m2":
        want[m - 2] = -np.inf
    c, buf = wide(np.zeros((m, n)), out, 1, 1)
    F.matmul(a.m, b.m, c)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(want).float().to(TORCH[out])
    got = c.cpu()
    if fmt == "e5m2" and torch.isnan(got[m - 2, n // 2]):
        ref[m - 2, n // 2] = float("nan")
    torch.testing.assert_close(got, ref, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("mnk", kind_sizes(300))
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_what_cancels_down_to_the_cut(mnk, out):
    """Products of 256 that cancel, and ones of 2^-5, 2^-13 of them, that are left:
    none is cut off, in any order.  At 2^-6 the 16-bit results may lose them, up to
    7 * 2^-13 of 256 in each eight; fp32 does not."""
    m, n, k = mnk
    rng = np.random.default_rng(m + 1)
    b = Held(n, k)
    cb = b.m.codes.view(torch.uint8)
    cb[:, :k], cb[:, k:] = int(O.nearest(1.0, "e4m3")), 0
    b.m.scales.fill_(127)
    for unit in (2.0 ** -5, 2.0 ** -6):
        v = np.zeros((m, k))
        v[:, :100], v[:, 100:200], v[:, 200:] = 256.0, -256.0, unit * rng.integers(-1, 2, (m, k - 200))
        v = rng.permuted(v, axis=1)
        a = Held(m, k)
        code = np.zeros((m, a.width))
        code[:, :k] = v
        a.m.codes.view(torch.uint8).copy_(torch.from_numpy(O.nearest(code, "e4m3")).view(m, -1))
        a.m.scales.fill_(127)
        c = torch.empty(m, n, dtype=TORCH[out], device="cuda")
        F.matmul(a.m, b.m, c)
        want = np.repeat(v.sum(1, keepdims=True), n, 1)
        if out == "f32" or unit == 2.0 ** -5:
            np.testing.assert_array_equal(np64(c), want)
        else:
            assert np.all(np.abs(np64(c) - want) <= -(-k // 8) * 7 * 2.0 ** -5)


def test_nothing_is_recorded_for_autograd():
    """Inputs that require a gradient are values, and outputs carry none."""
    x = torch.randn(5, 200, device="cuda", requires_grad=True)
    gain = torch.ones(200, device="cuda", requires_grad=True)
    out, r, h8, y = torch.empty(5, 200, device="cuda"), torch.empty(5, device="cuda"), F.Matrix8(5, 200), torch.empty(5, 5, device="cuda")
    F.rms_norm(x, gain, 1e-6, out=out, out8=h8, rstd=r)
    F.matmul(h8, h8, y)
    for t in (out, r, y):
        assert not t.requires_grad and t.grad_fn is None
    want = O.rms_norm(np64(x), np64(gain), 1e-6)[1]
    assert np.all(np.abs(np64(out) - want) <= U * (1 + 2.0 ** -20) * np.abs(want))


def test_norm_backward_of_the_longest_row():
    """2^27 elements and a few: more columns than threads that one launch has."""
    dim = (1 << 27) + 37
    gen = torch.Generator("cuda").manual_seed(0)
    mk = lambda: torch.randn(1, dim, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    g, z, w = mk(), mk(), mk().view(-1)
    r = torch.tensor([0.75], device="cuda")
    dz, dw = torch.full_like(z, float("nan")), torch.full((dim,), float("nan"), device="cuda")
    F.rms_norm_backward(g, z, r, w, dz=dz, dw=dw)
    g64, x64 = g[0].double(), z[0].double() * 0.75
    want = g64 * x64
    assert bool(((dw.double() - want).abs() <= 2 * U * want.abs()).all())
    old = dw.clone()
    F.rms_norm_backward(g, z, r, w, dz=dz, dw=dw, accumulate=True)
    assert torch.equal(dw, old + old)
    a = g64 * w.double()
    mean = float((a * x64).mean())
    most = float((a * x64).abs().mean())
    want = 0.75 * (a - x64 * mean)
    tol = U * (0.75 * (4 * a.abs() + x64.abs() * most * (depth(dim) + 10)) + 4 * want.abs())
    assert bool(((dz[0].double() - want).abs() <= tol + HALF["bf16"] * (want.abs() + tol)).all())
