"""fp64 oracle of the first-order operators: the AdamW step, the e4m3 codes of
its 8-bit moments, and the global gradient norm.  NumPy, written from the
formulas; shares no code with the library.  Used by the tests.

Beside each value the oracle gives how far an fp32 evaluation may be from it:
`u = 2^-24` for each rounding to nearest (relative to what is rounded), summed
along the formula."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

U = 2.0 ** -24          # half a unit in the last place of fp32, relative
TINY = 2.0 ** -149      # and the least that a rounding of denormals can be off by
RUN = 256


@dataclass
class Hyper:
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    lr: float = 1e-3
    weight_decay: float = 0.0
    lr_scale: float = 1.0


def step(p, g, m, v, t, h: Hyper, coef=1.0, m_err=0.0, v_err=0.0):
    """One step (the t-th, from 1) of fp64 arrays.  m_err, v_err: how far the
    library's own m and v may be from these before it.  Returns new p, m, root
    = sqrt(v), v and the same number of error bounds."""
    x = coef * g
    x_err = 2 * U * np.abs(x) + TINY            # the coefficient's rounding, the product's
    m1 = h.beta1 * m + (1 - h.beta1) * x
    # each product: its scalar's rounding and its own; then the sum's
    m1_err = (h.beta1 * m_err + 2 * U * np.abs(h.beta1 * m) + (1 - h.beta1) * x_err
              + 2 * U * np.abs((1 - h.beta1) * x) + U * np.abs(m1) + 3 * TINY)
    v1 = h.beta2 * v + (1 - h.beta2) * x * x
    v1_err = (h.beta2 * v_err + 2 * U * h.beta2 * v
              + (1 - h.beta2) * (2 * np.abs(x) * x_err + 3 * U * x * x) + U * v1 + 4 * TINY)
    root = np.sqrt(v1)
    # |sqrt(a) - sqrt(b)| <= |a - b| / sqrt(max), and <= sqrt|a - b|
    with np.errstate(divide="ignore", invalid="ignore"):
        near = np.where(root > 0, v1_err / np.where(root > 0, root, 1), np.inf)
    root_err = np.minimum(near, np.sqrt(v1_err)) + U * root
    c = 1.0 / np.sqrt(1.0 - h.beta2 ** t)
    d = root * c + h.eps
    d_err = c * root_err + 3 * U * c * root + U * h.eps + U * d + TINY
    q = m1 / d
    d_low = np.maximum(d - d_err, h.eps * (1 - 2 * U))
    q_err = m1_err / d_low + np.abs(m1) * d_err / (d * d_low) + U * np.abs(q) + 2 * TINY
    b = h.lr * h.lr_scale / (1.0 - h.beta1 ** t)
    a = h.lr * h.lr_scale * h.weight_decay
    upd = a * p + b * q
    p1 = p - upd
    p1_err = (2 * U * np.abs(a * p) + b * q_err + 3 * U * np.abs(b * q) + U * np.abs(upd)
              + U * np.abs(p1) + 4 * TINY)
    return p1, m1, root, v1, p1_err, m1_err, root_err, v1_err


def _times(x, c):
    return (x.astype(np.uint64) * np.uint64(c) & np.uint64(0xFFFFFFFF)).astype(np.uint64)


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    x = _times(x ^ (x >> np.uint64(16)), 0xFD63ED5B)
    x = _times(x ^ (x >> np.uint64(15)), 0x7BC73A83)
    return x ^ (x >> np.uint64(16))


def random_bits(seed, t, tensor, element):
    """The 16 bits each that round m and sqrt(v) of an element at step t."""
    m32 = np.uint64(0xFFFFFFFF)
    element = np.asarray(element, dtype=np.uint64)
    key = mix((mix(seed) + np.uint64(t)) & m32)
    key = mix((key + np.uint64(tensor)) & m32)
    key = (key + _times(element >> np.uint64(32), 0x85157AF5)) & m32
    h = mix(key ^ (element & m32))
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def e4m3_values():
    """The 127 non-negative values of e4m3, rising."""
    code = np.arange(127)
    e, f = code >> 3, code & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))


def decode(codes):
    """e4m3 codes (uint8) as fp64 values."""
    table = np.concatenate([e4m3_values(), [np.nan]])
    codes = np.asarray(codes, dtype=np.uint8)
    return np.where(codes >> 7, -1.0, 1.0) * table[codes & 127]


def run_scales(x):
    """Scale of every run of 256 values (the last one may be short): 1/448 of
    the largest finite magnitude, at least 2^-110 / 448."""
    n = -(-x.size // RUN) * RUN
    y = np.zeros(n)
    y[:x.size] = np.where(np.isfinite(x), np.abs(x), 0.0)
    return np.maximum(y.reshape(-1, RUN).max(1, initial=0.0), 2.0 ** -110) / 448


def store(y, r, positive):
    """Magnitudes y (in units of the scale) rounded down or up to e4m3 by the
    random r / 65536, as values.  Monotonic in y."""
    y = np.minimum(y, 448.0)
    q = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    z = np.minimum(np.floor(y / q + r / 65536.0) * q, 448.0)
    return np.where((y > 0) & (z == 0), 2.0 ** -9, z) if positive else z


def store_range(x, x_err, scale, r, positive):
    """The least and the largest magnitude that fp32 may store for x, whose own
    fp32 value is within x_err: the scale's two roundings (and the error of the
    value it is taken from), the reciprocal's and the product's come on top."""
    s = np.repeat(scale, RUN)[:x.size]
    top = s * 448
    with np.errstate(invalid="ignore"):
        err = np.repeat(np.maximum.reduceat(np.where(np.isfinite(x_err), x_err, 0.0),
                                            np.arange(0, x.size, RUN)), RUN)[:x.size]
    y = np.abs(x) / s
    dy = x_err / s + y * (err / top + 5 * U) + 2.0 ** -33   # adding 2^-6 rounds at 2^-30 / 2 at most
    lo = store(np.maximum(y - dy, 0.0), r, positive)
    hi = store(y + dy, r, positive)
    if positive:   # a root that is 0 or next to it
        lo = np.where(np.abs(x) - x_err <= 0, 0.0, lo)
    return lo, hi


def bf16_split(w):
    """fp32 weights as the nearest bf16 (ties away from zero) and what is left
    in units of fp32's last place."""
    bits = np.asarray(w, dtype=np.float32).view(np.uint32).astype(np.int64)
    hi = (bits + 0x8000) >> 16
    return hi.astype(np.uint16), (bits - (hi << 16)).astype(np.int16)


def bf16_join(hi, rem):
    bits = (hi.astype(np.int64) << 16) + rem.astype(np.int64)
    return (bits & 0xFFFFFFFF).astype(np.uint32).view(np.float32)


def norm(grads, max_norm, grad_scale=1.0):
    """Global norm and clip coefficient, in fp64 with exact sums of squares."""
    import math
    total = math.fsum(float(np.dot(g, g)) for g in grads)
    n = grad_scale * math.sqrt(total) if math.isfinite(total) else math.inf
    if not math.isfinite(n):
        return n, 0.0
    return n, grad_scale * min(1.0, max_norm / n if n > 0 else 1.0)


# ---------------------------------------------------------------- in fp32
def step32(p, g, m, v, t, h: Hyper, coef=1.0):
    """The step in fp32 (NumPy's operations round to nearest): every operation
    rounded on its own in the order of the formula, scalars formed in fp64 and
    rounded once.  Returns p, m, root, v."""
    f = np.float32
    with np.errstate(all="ignore"):
        x = g * f(coef)
        m = m * f(h.beta1) + x * f(1 - h.beta1)
        v = v * f(h.beta2) + (x * x) * f(1 - h.beta2)
        root = np.sqrt(v)
        a = f(h.lr * h.lr_scale * h.weight_decay)
        b = f(h.lr * h.lr_scale * (1.0 / (1.0 - h.beta1 ** t)))
        d = root * f(1.0 / np.sqrt(1.0 - h.beta2 ** t)) + f(h.eps)
        p = p - (p * a + (m / d) * b)
    return p, m, root, v


def codes32(x, r, positive):
    """Codes and scales of fp32 values (whole runs, finite) in fp32 steps."""
    f = np.float32
    y = np.abs(x).reshape(-1, RUN)
    scale = np.maximum(y.max(1), f(2.0 ** -110)) * f(1 / 448)
    y = y * (f(1) / scale)[:, None]
    small = y < f(2.0 ** -6)
    bits = np.where(small, y + f(2.0 ** -6), y).astype(f).view(np.int32)
    code = ((bits + (r.reshape(-1, RUN).astype(np.int32) << 4)) >> 20) - np.where(small, 968, 960)
    if positive:
        code = np.maximum(code, x.reshape(-1, RUN) > 0)
    else:
        code = code + 128 * np.signbit(x).reshape(-1, RUN)
    return code.astype(np.uint8).reshape(-1), scale
