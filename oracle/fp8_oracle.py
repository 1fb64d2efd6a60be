"""fp64 oracle of the operators of a layer in 8 bits: NumPy, no code of the
library.  Codes are found in the table of all the values a format has."""
import numpy as np

BLOCK = 128
TOP = {"e4m3": 8, "e5m2": 15}
#: half a step: relative to a value in the format's normal range, and in units
#: of the scale below it
HALF = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
HALF_LOW = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}


def code_values(fmt):
    """The value of each of the 256 codes (OCP e4m3 without infinities, e5m2)."""
    mant, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    out = np.empty(256)
    for u in range(256):
        e, m = (u & 0x7F) >> mant, u & ((1 << mant) - 1)
        if fmt == "e4m3" and (u & 0x7F) == 0x7F:
            v = np.nan
        elif fmt == "e5m2" and e == 31:
            v = np.inf if m == 0 else np.nan
        elif e == 0:
            v = m * 2.0 ** (1 - bias - mant)
        else:
            v = (1 + m / (1 << mant)) * 2.0 ** (e - bias)
        out[u] = -v if u & 0x80 else v
    return out


_POSITIVE = {}


def _positive(fmt):
    if fmt not in _POSITIVE:
        v = code_values(fmt)[:128]
        _POSITIVE[fmt] = v[np.isfinite(v)]
    return _POSITIVE[fmt]


def nearest(y, fmt):
    """Codes of values whose magnitudes the format reaches: the nearest, halves
    to the even code.  Not finite: NaN, or an infinity where the format has one
    (the sign bit of a NaN is not defined; it is left 0 here)."""
    y = np.asarray(y, np.float64)
    table = _positive(fmt)
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.minimum(np.searchsorted(table, a), len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (up == 0), hi, lo)
    code = np.where(np.signbit(y), code + 128, code)
    if fmt == "e5m2":
        code = np.where(np.isinf(y), np.where(y < 0, 0xFC, 0x7C), code)
        code = np.where(np.isnan(y), 0x7F, code)
    else:
        code = np.where(np.isfinite(y), code, 0x7F)
    return code.astype(np.uint8)


def exponents(largest, fmt):
    """The least e >= -127 with largest <= 1.75 2^(TOP + e)."""
    largest = np.asarray(largest, np.float64)
    e = np.full(largest.shape, -127, np.int64)
    for i in np.ndindex(largest.shape):
        while largest[i] > np.ldexp(1.75, TOP[fmt] + int(e[i])):
            e[i] += 1
    return e


def _padded(x):
    rows, cols = x.shape
    out = np.zeros((rows, -(-cols // BLOCK) * BLOCK))
    out[:, :cols] = x
    return out.reshape(rows, -1, BLOCK)


def finite_abs(x):
    return np.where(np.isfinite(x), np.abs(x), 0.0)


def encode(x, fmt, e=None):
    """(codes (rows, pitch), exponents (rows, blocks)) of an fp64 matrix."""
    b = _padded(np.asarray(x, np.float64))
    if e is None:
        e = exponents(finite_abs(b).max(2), fmt)
    return nearest(np.ldexp(b, -e[..., None]), fmt).reshape(b.shape[0], -1), e


def encode_weight(x):
    """Codes and exponents of a matrix and of its transpose, one exponent for
    each 128 x 128 values."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    big = np.zeros((-(-rows // BLOCK) * BLOCK, -(-cols // BLOCK) * BLOCK))
    big[:rows, :cols] = finite_abs(x)
    e = exponents(big.reshape(big.shape[0] // BLOCK, BLOCK, -1, BLOCK).max((1, 3)), "e4m3")
    er = np.repeat(e, BLOCK, 0)[:rows]
    ec = np.repeat(e.T, BLOCK, 0)[:cols]
    return encode(x, "e4m3", er), encode(x.T, "e4m3", ec)


def grouped(e):
    """Exponent bytes as they are held: (groups, rows, 4), and which of them a
    row has."""
    rows, n = e.shape
    out = np.zeros((-(-n // 4), rows, 4), np.uint8)
    has = np.zeros(out.shape, bool)
    for b in range(n):
        out[b // 4, :, b % 4] = e[:, b] + 127
        has[b // 4, :, b % 4] = True
    return out, has


def values(codes, scales, cols, fmt):
    """What an 8-bit matrix holds, from its codes and grouped scale bytes."""
    rows, pitch = codes.shape
    v = code_values(fmt)[codes]
    for b in range(-(-cols // BLOCK)):
        e = scales[b // 4, :, b % 4].astype(np.int64) - 127
        v[:, b * BLOCK:(b + 1) * BLOCK] = np.ldexp(v[:, b * BLOCK:(b + 1) * BLOCK], e[:, None].astype(np.int32))
    return v[:, :cols]


def rms_norm(z, w, eps):
    r = 1.0 / np.sqrt((z * z).mean(1) + eps)
    return r, z * r[:, None] * w


def rms_norm_backward(g, z, r, w, add):
    a, unit = g * w, z * r[:, None]
    dz = r[:, None] * (a - unit * (a * unit).mean(1, keepdims=True))
    return (dz if add is None else dz + add), (g * unit).sum(0)
