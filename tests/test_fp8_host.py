"""The 8-bit operators without a GPU: struct layouts, refusals, plans, and the
oracle's own pieces against torch's formats and brute force."""
import ctypes

import numpy as np
import pytest

from oracle import fp8_oracle as O
from second_order_optimizer_amd import shampoo as S

torch = pytest.importorskip("torch")

E_ARG, E_STATE, E_UNSUPPORTED = -1, -2, -5
# addresses that no refused call may use
X, C8, S8, D8, T8, OUT, WORK = (0x10000000 * k for k in range(1, 8))


def m8(rows, cols, codes=C8, scales=S8, pitch=None, scale_pitch=None, fmt=0, reserved=0):
    pitch = -(-cols // 128) * 128 if pitch is None else pitch
    return S.Matrix8Desc(codes, scales, rows, cols, pitch, rows if scale_pitch is None else scale_pitch, fmt, reserved)


def at(m):
    return None if m is None else ctypes.addressof(m)


def test_struct_sizes():
    assert ctypes.sizeof(S.Matrix8Desc) == 56
    assert ctypes.sizeof(S.RmsNormArgs) == 128
    assert ctypes.sizeof(S.RmsNormGradArgs) == 120
    assert ctypes.sizeof(S.WeightDesc) == 24
    assert ctypes.sizeof(S.Weights8Layout) == 40


# ------------------------------------------------------------ refusals
def quantize(x=X, type=1, pitch=300, rows=200, cols=300, a=None, b=None):
    return S.lib().shampoo_quantize8(x, type, pitch, rows, cols, at(a), at(b), None)


@pytest.mark.parametrize("kw", [
    dict(a=None), dict(a=m8(200, 299)), dict(a=m8(300, 200)), dict(b=m8(200, 300)), dict(a=m8(200, 300, fmt=2)),
    dict(a=m8(200, 300, fmt=-1)), dict(a=m8(200, 300, reserved=1)), dict(a=m8(200, 300, pitch=256)),
    dict(a=m8(200, 300, pitch=392)), dict(a=m8(200, 300, scale_pitch=199)), dict(a=m8(200, 300, codes=C8 + 8)),
    dict(a=m8(200, 300, scales=S8 + 2)), dict(a=m8(200, 300, codes=None)), dict(a=m8(200, 300, scales=None)),
    dict(a=m8(200, 300), x=None), dict(a=m8(200, 300), x=X + 1), dict(a=m8(200, 300), type=3), dict(a=m8(200, 300), type=-1),
    dict(a=m8(200, 300), pitch=299), dict(a=m8(-1, 300), rows=-1), dict(a=m8(200, -1), cols=-1),
    dict(a=m8(200, 300), rows=1 << 41), dict(a=m8(200, 300, codes=X + 16)), dict(a=m8(200, 300, scales=X)),
    dict(a=m8(200, 300), b=m8(300, 200)), dict(a=m8(200, 300), b=m8(300, 200, codes=D8, scales=S8 + 4)),
    dict(a=m8(200, 300, scales=C8 + 128))])
def test_quantize_refuses(kw):
    assert quantize(**kw) == E_ARG


def test_quantize_past_a_launch_and_empty():
    big = 1 << 31
    assert quantize(rows=big, cols=256, pitch=256, a=m8(big, 256, codes=1 << 45, scales=1 << 50)) == E_UNSUPPORTED
    assert quantize(rows=0, a=m8(0, 300)) == 0
    assert quantize(x=None, rows=5, cols=0, a=m8(5, 0, codes=None, scales=None), b=m8(0, 5)) == 0


def test_transpose_refuses():
    f = S.lib().shampoo_transpose8
    a = m8(200, 300)
    assert f(None, at(a), None) == E_ARG
    assert f(at(a), None, None) == E_ARG
    for o in (m8(200, 300, D8, T8), m8(300, 200, C8, T8), m8(300, 200, D8, S8), m8(300, 200, D8 + 1, T8), m8(300, 200, D8, C8 + 512)):
        assert f(at(a), at(o), None) == E_ARG
    assert f(at(m8(0, 5)), at(m8(5, 0, D8, T8)), None) == 0


def matmul(a=None, b=None, c=OUT, type=0, pitch=100, add=0, work=None, bytes=0):
    a = m8(50, 300) if a is None else a
    b = m8(100, 300, D8, T8) if b is None else b
    return S.lib().shampoo_matmul8(at(a), at(b), c, type, pitch, add, work, bytes, None)


@pytest.mark.parametrize("kw", [
    dict(b=m8(100, 301, D8, T8)), dict(c=None), dict(c=OUT + 2), dict(type=3), dict(pitch=99), dict(add=2), dict(add=-1),
    dict(a=m8(50, 300, fmt=2)), dict(a=m8(50, 300, codes=None)), dict(a=m8(50, 300, pitch=384 + 8)),
    dict(b=m8(100, 300, D8, T8, reserved=3)), dict(c=C8 + 64), dict(c=T8 + 4), dict(a=m8(-50, 300))])
def test_matmul_refuses(kw):
    assert matmul(**kw) == E_ARG


def test_matmul_empty_and_nulls():
    L = S.lib()
    assert matmul(a=m8(0, 300)) == 0
    assert matmul(b=m8(0, 300, D8, T8), c=None, pitch=0) == 0
    assert L.shampoo_matmul8(None, at(m8(1, 1)), OUT, 0, 1, 0, None, 0, None) == E_ARG
    n = ctypes.c_size_t()
    assert L.shampoo_matmul8_workspace(1, 1, 1, 0, None) == E_ARG
    assert L.shampoo_matmul8_workspace(-1, 1, 1, 0, ctypes.byref(n)) == E_ARG
    for m, k in ((0, 0), (1, 1), (7, 100000)):
        assert L.shampoo_matmul8_workspace(m, 5, k, 0, ctypes.byref(n)) == 0
    assert L.shampoo_matmul8_workspace(1, 1, 1, 3, ctypes.byref(n)) == E_ARG
    # a long sum into a small matrix goes in parts, whose sums need memory
    assert L.shampoo_matmul8_workspace(512, 512, 65536, 0, ctypes.byref(n)) == 0 and n.value % (512 * 512 * 4) == 0 and n.value
    far = m8(3, 300, pitch=(1 << 23) + 128)
    assert matmul(a=far) == E_UNSUPPORTED


def norm(**kw):
    a = S.RmsNormArgs(20, 300, X, None, None, OUT, None, None, WORK, 300, 300, 300, 300, 1, 1, 1, 1, 1e-6)
    keep = kw.get("out8")
    for k, v in kw.items():
        setattr(a, k, at(v) if k == "out8" else v)
    rc = S.lib().shampoo_rms_norm8(ctypes.addressof(a), None)
    del keep
    return rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dim=0), E_ARG), (dict(rows=-1), E_ARG), (dict(eps=0.0), E_ARG), (dict(eps=float("nan")), E_ARG),
    (dict(eps=float("inf")), E_ARG), (dict(eps=1e-60), E_ARG), (dict(eps=1e60), E_ARG), (dict(x=None), E_ARG),
    (dict(x=X + 1), E_ARG), (dict(x_type=3), E_ARG), (dict(x_pitch=299), E_ARG), (dict(weight=None), E_ARG),
    (dict(weight_type=5), E_ARG), (dict(residual=C8), E_ARG), (dict(total=C8), E_ARG), (dict(out=None), E_ARG),
    (dict(out_type=7), E_ARG), (dict(rstd=S8 + 2), E_ARG), (dict(rstd=WORK + 64), E_ARG), (dict(out=X), E_ARG),
    (dict(residual=C8, total=C8 + 2), E_ARG), (dict(residual=C8, total=X, x_type=0), E_ARG),
    (dict(residual=C8, total=C8, total_pitch=301), E_ARG), (dict(residual=C8, total=OUT), E_ARG),
    (dict(residual=C8, total=WORK), E_ARG), (dict(out8=m8(20, 299)), E_ARG), (dict(out8=m8(20, 300, codes=X)), E_ARG),
    (dict(out8=m8(20, 300, fmt=1)), E_UNSUPPORTED), (dict(out8=m8(20, 300, codes=WORK)), E_ARG)])
def test_norm_refuses(kw, rc):
    assert norm(**kw) == rc


def test_norm_without_rows_and_past_a_launch():
    assert norm(rows=0) == 0
    assert norm(rows=0, x=None, weight=None, out=None) == 0
    big = 1 << 23
    assert norm(rows=big, dim=10000, x=1 << 45, out=1 << 50, x_pitch=10000, out_pitch=10000) == E_UNSUPPORTED
    assert S.lib().shampoo_rms_norm8(None, None) == E_ARG


def back(work=WORK, bytes=1 << 27, **kw):
    a = S.RmsNormGradArgs(20, 300, X, C8, S8, OUT, None, D8, T8, 300, 300, 300, 300, 1, 1, 1, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return S.lib().shampoo_rms_norm8_backward(ctypes.addressof(a), work, bytes, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dim=0), E_ARG), (dict(rows=-1), E_ARG), (dict(grad=None), E_ARG), (dict(z=None), E_ARG), (dict(rstd=None), E_ARG),
    (dict(rstd=S8 + 1), E_ARG), (dict(weight=None), E_ARG), (dict(dz=None), E_ARG), (dict(grad_type=3), E_ARG),
    (dict(z_type=-1), E_ARG), (dict(weight_type=3), E_ARG), (dict(accumulate=2), E_ARG), (dict(z_pitch=299), E_ARG),
    (dict(dz=C8 + 2), E_ARG), (dict(dz=C8, dz_pitch=301), E_ARG), (dict(dz=X, grad_type=2), E_ARG),
    (dict(add=D8 + 600), E_ARG), (dict(dz=S8), E_ARG), (dict(dw=T8 + 2), E_ARG), (dict(dw=D8), E_ARG), (dict(dw=OUT), E_ARG),
    (dict(work=None), E_STATE), (dict(bytes=10), E_STATE), (dict(work=WORK + 8), E_ARG), (dict(work=X), E_ARG),
    (dict(work=D8), E_ARG)])
def test_norm_backward_refuses(kw, rc):
    assert back(**kw) == rc


def test_norm_backward_workspace():
    L, n = S.lib(), ctypes.c_size_t()
    assert L.shampoo_rms_norm8_backward_workspace(1, 0, ctypes.byref(n)) == E_ARG
    assert L.shampoo_rms_norm8_backward_workspace(1, 1, None) == E_ARG
    for rows, dim in ((0, 5), (1, 1), (100000, 4096), (10, 100000)):
        assert L.shampoo_rms_norm8_backward_workspace(rows, dim, ctypes.byref(n)) == 0
        assert n.value % (4 * dim) == 0 and n.value >= 4 * dim * min(rows, 1) and n.value <= 4 * dim * 4096


def create(descs):
    h = S._P()
    arr = (S.WeightDesc * max(len(descs), 1))(*descs)
    return S.lib().shampoo_weights8_create(len(descs), arr, ctypes.byref(h)), h


def test_weights_refuse():
    L = S.lib()
    assert create([])[0] == E_ARG
    assert L.shampoo_weights8_create(1, None, ctypes.byref(S._P())) == E_ARG
    assert L.shampoo_weights8_create(1, (S.WeightDesc * 1)(S.WeightDesc(1, 1, 0, 0)), None) == E_ARG
    for d, rc in ((S.WeightDesc(-1, 1, 0, 0), E_ARG), (S.WeightDesc(1, 1, 3, 0), E_ARG), (S.WeightDesc(1, 1, 0, 1), E_ARG),
                  (S.WeightDesc(1, 1, 1, 0), E_ARG), (S.WeightDesc(1 << 31, 1, 0, 0), E_UNSUPPORTED),
                  (S.WeightDesc(1 << 20, 1 << 20, 0, 0), E_UNSUPPORTED)):
        assert create([S.WeightDesc(4, 4, 0, 0), d])[0] == rc
    rc, h = create([S.WeightDesc(200, 300, 1, 0), S.WeightDesc(0, 7, 1, 0)])
    assert rc == 0
    lay = S.Weights8Layout()
    assert L.shampoo_weights8_get_layout(h, ctypes.byref(lay)) == 0
    assert lay.code_bytes == 200 * 384 + 300 * 256 and lay.scale_bytes == 4 * 200 + 224 + 4 * 300 + 80   # whole 256 bytes
    assert L.shampoo_weights8_get_layout(h, None) == E_ARG
    m, ptrs = S.Matrix8Desc(), (S._P * 2)(X, X)
    assert L.shampoo_weights8_matrix(h, 0, 0, ctypes.byref(m)) == E_STATE
    assert L.shampoo_weights8_matrix(h, 2, 0, ctypes.byref(m)) == E_ARG
    assert L.shampoo_weights8_matrix(h, 0, 2, ctypes.byref(m)) == E_ARG
    assert L.shampoo_weights8_refresh(h, None) == E_STATE
    assert L.shampoo_weights8_refresh(None, None) == E_ARG
    assert L.shampoo_weights8_bind_weights(h, ptrs, None) == E_STATE
    assert L.shampoo_weights8_bind_weights(h, None, None) == E_ARG
    assert L.shampoo_weights8_bind_state(h, None, 0, None) == E_ARG
    assert L.shampoo_weights8_bind_state(h, 128, 1 << 30, None) == E_ARG
    assert L.shampoo_weights8_bind_state(h, 256, 16, None) == E_STATE
    L.shampoo_weights8_destroy(h)


# ------------------------------------------------------------ the binding, before it reaches the library
def test_binding_refuses():
    from second_order_optimizer_amd import fp8 as F
    cpu = dict(device="cpu")
    a = F.Matrix8(4, 200, **cpu)
    assert a.codes.shape == (4, 256) and a.scales.shape == (1, 4, 4)
    x = torch.zeros(4, 200)
    with pytest.raises(ValueError):
        F.quantize(x)                                            # no output
    with pytest.raises(ValueError):
        F.quantize(x, rows=F.Matrix8(4, 201, **cpu))
    with pytest.raises(ValueError):
        F.quantize(x, cols=a)
    with pytest.raises(ValueError):
        F.quantize(x, rows=a)                                    # no kernels for the CPU
    with pytest.raises(ValueError):
        F.quantize(torch.zeros(200, 4).t(), rows=a)              # rows whose elements are apart
    with pytest.raises(ValueError):
        F.quantize(torch.zeros(1, 200).expand(4, 200), rows=a)   # rows in one place
    with pytest.raises(ValueError):
        F.quantize(x.double(), rows=a)
    with pytest.raises(ValueError):
        F.quantize(x[0], rows=a)
    with pytest.raises(ValueError):
        F.transpose(a, F.Matrix8(4, 200, **cpu))
    with pytest.raises(ValueError):
        F.matmul(a, F.Matrix8(3, 201, **cpu), torch.zeros(4, 3))
    with pytest.raises(ValueError):
        F.matmul(a, F.Matrix8(3, 200, **cpu), torch.zeros(3, 4))
    w = torch.ones(200)
    with pytest.raises(ValueError):
        F.rms_norm(x, w[:199], 1e-6, out8=a)
    with pytest.raises(ValueError):
        F.rms_norm(x, w, 1e-6, out8=a, residual=x)
    with pytest.raises(ValueError):
        F.rms_norm(x, w, 1e-6, out8=a, residual=x, total=x.bfloat16())
    with pytest.raises(ValueError):
        F.rms_norm(x, w, 1e-6, out8=a, rstd=torch.zeros(3))
    with pytest.raises(ValueError):
        F.rms_norm_backward(x, x, torch.ones(4), w, dz=x.bfloat16())
    with pytest.raises(ValueError):
        F.rms_norm_backward(x, x, torch.ones(4), w, dz=torch.zeros(4, 200), dw=w.bfloat16())
    for bad in (dict(codes=torch.zeros(4, 256, dtype=torch.uint8)), dict(codes=a.codes[:, :128], scales=a.scales),
                dict(codes=a.codes, scales=a.scales.transpose(0, 1)), dict(codes=a.codes, scales=a.scales.int())):
        with pytest.raises(ValueError):
            F.Matrix8(4, 200, **bad)
    with pytest.raises(ValueError):
        F.Matrix8(-1, 5, **cpu)
    with pytest.raises(KeyError):
        F.Matrix8(1, 5, "e3m4", **cpu)
    with pytest.raises(ValueError):
        F.Weights8([(4, 4)], device="cpu")


def test_rows_between():
    from second_order_optimizer_amd import fp8 as F
    a = F.Matrix8(10, 700, device="cpu")
    b = a.between(3, 7)
    assert (b.rows, b.cols, b.desc.pitch, b.desc.scale_pitch) == (4, 700, 768, 10)
    assert b.desc.codes == a.desc.codes + 3 * 768 and b.desc.scales == a.desc.scales + 12
    assert a.between(5, 5).rows == 0
    for s in ((-1, 3), (4, 3), (0, 11)):
        with pytest.raises(ValueError):
            a.between(*s)


# ------------------------------------------------------------ the oracle's pieces
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_codes_against_torch(fmt, dtype):
    every = torch.arange(256, dtype=torch.uint8)
    v = every.view(dtype).double().numpy()
    np.testing.assert_array_equal(O.code_values(fmt), v)
    fin = np.sort(v[np.isfinite(v)])
    half = (fin[1:] + fin[:-1]) / 2
    y = np.concatenate([fin, half, half * (1 + 2.0 ** -20), half * (1 - 2.0 ** -20), fin * (1 + 2.0 ** -20)])
    y = y[np.abs(y) <= fin[-1]]
    got = O.nearest(y, fmt)
    want = torch.from_numpy(y).float().to(dtype).view(torch.uint8).numpy()
    np.testing.assert_array_equal(O.code_values(fmt)[got], O.code_values(fmt)[want])
    np.testing.assert_array_equal(got[y != 0], want[y != 0])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponents(fmt):
    top = 448.0 if fmt == "e4m3" else 57344.0
    for e in (-127, -126, -1, 0, 5, 100):
        edge = np.ldexp(top, e)
        assert O.exponents([edge, edge * (1 + 2.0 ** -40)], fmt).tolist() == [e, e + 1]
    assert O.exponents([0.0, 2.0 ** -149], fmt).tolist() == [-127, -127]


def test_weight_and_its_transpose_hold_the_same():
    x = np.random.default_rng(0).standard_normal((200, 300)) * np.exp(np.random.default_rng(1).standard_normal((200, 1)))
    (a, ea), (b, eb) = O.encode_weight(x)
    va, vb = O.values(a, O.grouped(ea)[0], 300, "e4m3"), O.values(b, O.grouped(eb)[0], 200, "e4m3")
    np.testing.assert_array_equal(va, vb.T)
    assert np.all(np.abs(va - x) <= np.maximum(O.HALF["e4m3"] * np.abs(x), 448 * np.abs(x).max() * O.HALF_LOW["e4m3"] / 224))


def test_norm_gradient_against_differences():
    """Central differences of step h in fp64: an error of order h^2 plus 2^-53 / h, some 1e-9 of the values here."""
    rng = np.random.default_rng(3)
    z, w, g = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    f = lambda z, w: float((O.rms_norm(z, w, 1e-3)[1] * g).sum())  # noqa: E731
    dz, dw = O.rms_norm_backward(g, z, O.rms_norm(z, w, 1e-3)[0], w, None)
    h = 1e-5
    for i in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[i] = h
        assert abs((f(z + d, w) - f(z - d, w)) / (2 * h) - dz[i]) < 1e-7
    for i in range(7):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(z, w + d) - f(z, w - d)) / (2 * h) - dw[i]) < 1e-7


# ------------------------------------------------------------ weights as their plan has them
def unbound(shapes, device="cpu"):
    """A Weights8 whose binding can be checked without a GPU: no library, no state."""
    from second_order_optimizer_amd import fp8 as F
    w = F.Weights8.__new__(F.Weights8)
    w.shapes = list(shapes)
    w.want = [(r * c, 0) for r, c in shapes]
    w.device, w._types = torch.device(device), (torch.float32, torch.bfloat16, torch.float16)
    w.calls = []
    w._call = lambda fn, *args: w.calls.append(fn.__name__)
    w._held = None
    return w


@pytest.mark.parametrize("planned,shape", [((4, 6), (6, 4)), ((4, 6), (3, 8)), ((4, 6), (2, 12)), ((4, 6), (6, 2, 2)), ((2, 12), (3, 2, 4)),
                                           ((1, 24), (4, 6, 1)), ((24, 1), (2, 12)), ((4, 0), (0, 7)), ((5, 0), (4, 0))])
def test_bind_refuses_other_shapes(planned, shape):
    """As many elements in other rows would be copied as rows that they are not."""
    w = unbound([(3, 3), planned])
    with pytest.raises(ValueError, match=r"weights\[1\]"):
        w.bind([torch.zeros(3, 3), torch.zeros(shape)])
    assert not w.calls and w._held is None


@pytest.mark.parametrize("planned,shape", [((4, 6), (4, 6)), ((4, 6), (24,)), ((4, 6), (4, 2, 3)), ((4, 6), (2, 2, 6)), ((4, 6), (4, 2, 3, 1)),
                                           ((4, 6), (1, 4, 6)), ((1, 24), (1, 4, 6)), ((24, 1), (4, 6, 1)), ((0, 5), (0, 5)), ((5, 0), (5, 0)), ((1, 1), ())])
def test_bind_takes_the_plans_rows(planned, shape):
    """The plan's shape, its elements in one dimension, and more dimensions that
    are its rows and columns taken apart."""
    w = unbound([planned])
    t = torch.zeros(shape)
    w.bind([t])
    assert w.calls == ["shampoo_weights8_bind_weights"] and w._held[0] is t


# ------------------------------------------------------------ copies behind a step
class Stepped(S.Shampoo):
    """Shampoo's and AdamW's step() around steps that only say that they ran."""

    def __init__(self):
        self.ran = 0

    def _step(self, *args):
        self.ran += 1


def adamw_over(params):
    from second_order_optimizer_amd import adamw as A
    opt = A.AdamW.__new__(A.AdamW)
    opt.torch, opt.device, opt.ran = torch, torch.device("cpu"), 0
    opt._held = [params, None]

    def call(fn, *args):
        opt.ran += 1
    opt._call = call
    return opt


def both_steps(params, copies):
    """The steps that ran, of Shampoo and of AdamW, before either's refusal."""
    out = []
    s = Stepped()
    a = adamw_over(params)
    for opt, step in ((s, lambda: s.step(params, [None] * len(params), 0, 1, copies8=copies)), (a, lambda: a.step(1e-3, copies8=copies))):
        try:
            step()
            out.append(opt.ran)
        except ValueError:
            assert opt.ran == 0, "refused before the step, not behind it"
            out.append(None)
    return out


def test_copies_are_of_the_stepped_weights():
    """Copies of tensors that the step does not change would stay those of old
    values; a part of a stepped tensor is one."""
    a, b, other = torch.zeros(4, 6), torch.zeros(8, 3), torch.zeros(4, 6)
    w = unbound([(4, 6), (8, 3)])
    assert both_steps([a, b], w) == [None, None]               # nothing bound
    w.bind([a, b])
    assert both_steps([a, b], w) == [1, 1]
    assert both_steps([other, b, a], w) == [1, 1]
    assert both_steps([a, b, a[:1], b[:2]], w) == [1, 1]       # views that begin where they do
    assert w.calls.count("shampoo_weights8_refresh") == 6
    assert both_steps([other, b], w) == [None, None]           # another tensor in a's place
    assert both_steps([other, other], w) == [None, None]
    assert both_steps([a.clone(), b.clone()], w) == [None, None]
    w.bind([a.view(-1), b.view(8, 3, 1)])
    assert both_steps([a, b], w) == [1, 1]
    part = unbound([(2, 6), (0, 6)])
    part.bind([a[1:3], torch.zeros(0, 6)])
    assert both_steps([b, a], part) == [1, 1]
    assert both_steps([a[:2], b], part) == [None, None]        # its second row is not stepped
    assert both_steps([a[1:3], b], part) == [1, 1]


@pytest.mark.parametrize("dim,rows", [(8193, 1 << 22), (8192, 1 << 23), (4097, 1 << 23), (4096, 1 << 24), (2049, 1 << 24), (2048, 1 << 25), (1025, 1 << 25), (1024, 1 << 26)])
def test_norm_rows_past_a_launch(dim, rows):
    """The least number of rows whose launch would have 2^32 threads."""
    assert norm(rows=rows, dim=dim, x=1 << 45, out=1 << 50, x_pitch=dim, out_pitch=dim) == E_UNSUPPORTED
