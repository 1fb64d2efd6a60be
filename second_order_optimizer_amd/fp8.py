"""Layers in 8 bits, operators of libshampoo_mi355x.so (ctypes; argument
marshalling only): the product of a layer whose weights an optimizer here owns,
with a scale for each block of 128, the norm that feeds it, and what turns
activations, gradients and weights into 8 bits.

    w8 = fp8.Weights8([tuple(w.shape) for w in weights], param="f32")
    w8.bind(weights); w8.refresh()
    ...
    fp8.rms_norm(x, gain, 1e-6, residual=res, total=z, out8=h8, rstd=r)   # h8: tokens x width
    fp8.matmul(h8, w8.rows[0], y)                                         # y = h W^T
    ...
    fp8.quantize(dy, rows=dy8, cols=dyt8)                                 # dy and its transpose
    fp8.matmul(dy8, w8.cols[0], dh)                                       # dh = dy W
    fp8.transpose(h8, ht8)
    fp8.matmul(dyt8, ht8, dw, accumulate=True)                            # dW += dy^T h, fp32
    fp8.rms_norm_backward(dh, z, r, gain, add=dz, dz=dz, dw=dgain)
    opt.step(weights, [dw], t, cadence, copies8=w8)                       # Shampoo, or AdamW

A value in 8 bits is an e4m3 or e5m2 code times a power of two that 128
neighbours along a row share (weights: 128 x 128).  The gradients take the
rounding to 8 bits as the identity.  The calls record nothing for autograd: they
take tensors that require a gradient as values, and their outputs carry none; a
backward pass is made of the calls above.

Tensors are 2-D with neighbouring elements in a row (any row pitch, any start);
outputs are given.  Every call runs on the current stream of its tensors'
device, does not wait, and can be captured into a graph.  It raises if the
library has not been built -- there is no fallback.
"""
from __future__ import annotations

import bisect
import ctypes
import functools
import itertools
import operator
import struct
from typing import Optional, Sequence, Tuple

import torch

from .adamw import DTYPES, _Bound
from .shampoo import (Matrix8Desc, RmsNormArgs, RmsNormGradArgs, Weights8Layout, WeightDesc, _check, _P,
                      lib)

FORMATS = {"e4m3": 0, "e5m2": 1}
BLOCK = 128
_CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_F32 = (torch.float32,)

_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                  lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(device, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    index = device.index
    if index is None or device.type != "cuda":
        raise ValueError(f"no kernels for {device}")
    if _current() == index:
        rc = fn(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream(index))
    if rc:
        _check(rc, fn.__name__)


def _wide(t, rows, cols, device, what):
    """(address, type, pitch) of a wide matrix."""
    code = _TYPES.get(t.dtype)
    if code is None or t.shape != (rows, cols) or t.device != device:
        raise ValueError(f"{what} must be an fp32, bf16 or fp16 tensor of {rows} x {cols} on {device}")
    pitch, step = t.stride()
    if step != 1 and cols > 1 or pitch < cols and rows > 1:
        raise ValueError(f"{what}: the elements of a row must be neighbours and rows apart, got strides {t.stride()}")
    return t.data_ptr(), code, pitch if pitch > cols else cols


def _shape(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got {tuple(t.shape)}")
    return t.shape


def _vector(t, numel, device, what, types=_TYPES):
    if t.dtype not in types or t.dim() != 1 or t.numel() != numel or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be a contiguous vector of {numel} elements on {device}")
    return t.data_ptr()


class Matrix8:
    """rows x cols values in 8 bits.

    ``codes``: (rows, pitch) float8 codes, rows padded with zeros to whole blocks
    of 128; ``scales``: (groups, rows, 4) bytes e + 127 of the blocks' scales
    2^e, four neighbouring blocks of a row together (viewed as float8_e8m0fnu
    they are the scales).  Both are allocated unless given."""

    def __init__(self, rows: int, cols: int, fmt: str = "e4m3", device="cuda", codes=None, scales=None):
        rows, cols = int(rows), int(cols)
        if rows < 0 or cols < 0:
            raise ValueError(f"a matrix of {rows} x {cols}")
        blocks = -(-cols // BLOCK)
        groups = -(-blocks // 4)
        if codes is None or scales is None:
            if codes is not None or scales is not None:
                raise ValueError("codes and scales are given together")
            codes = torch.zeros(rows, blocks * BLOCK, dtype=torch.uint8, device=device).view(_CODES[fmt])
            scales = torch.zeros(groups, rows, 4, dtype=torch.uint8, device=device)
        if (codes.dtype != _CODES[fmt] or codes.dim() != 2 or codes.shape[0] != rows
                or codes.shape[1] < blocks * BLOCK
                or (codes.stride(1) != 1 and codes.shape[1] > 1)):
            raise ValueError(f"codes must be {_CODES[fmt]}, {rows} x at least {blocks * BLOCK}, neighbours in a row")
        if (scales.dtype != torch.uint8 or scales.device != codes.device
                or tuple(scales.shape) != (groups, rows, 4)
                or (scales.numel() and (scales.stride(2) != 1 or (rows > 1 and scales.stride(1) != 4)
                                        or (groups > 1 and scales.stride(0) % 4)))):
            raise ValueError(f"scales must be uint8 ({groups}, {rows}, 4) on {codes.device}, bytes of a row together")
        self.rows, self.cols, self.fmt, self.device = rows, cols, fmt, codes.device
        self.codes, self.scales = codes, scales
        pitch = codes.stride(0) if rows > 1 else max(blocks * BLOCK, 16)
        scale_pitch = scales.stride(0) // 4 if groups > 1 else rows
        self.desc = Matrix8Desc(codes.data_ptr(), scales.data_ptr(), rows, cols, pitch, scale_pitch,
                                FORMATS[fmt], 0)
        self.ptr = ctypes.addressof(self.desc)

    def between(self, start: int, stop: int) -> "Matrix8":
        """The rows from start on and before stop, in place."""
        if not 0 <= start <= stop <= self.rows:
            raise ValueError(f"rows {start} to {stop} of {self.rows}")
        return Matrix8(stop - start, self.cols, self.fmt, codes=self.codes[start:stop],
                       scales=self.scales[:, start:stop])


def _at8(m, rows, cols, device, what):
    if type(m) is not Matrix8 or m.rows != rows or m.cols != cols or m.device != device:
        raise ValueError(f"{what} must be a Matrix8 of {rows} x {cols} on {device}")
    return m.ptr


def quantize(x, rows: Optional[Matrix8] = None, cols: Optional[Matrix8] = None):
    """x in 8 bits: by its rows into ``rows`` (x's shape), by its columns into
    ``cols`` (its transpose's shape), or both with one reading of x."""
    dev = x.device
    r, c = _shape(x, "x")
    at, code, pitch = _wide(x, r, c, dev, "x")
    if rows is None and cols is None:
        raise ValueError("quantize: neither rows nor cols")
    _run(dev, lib().shampoo_quantize8, at, code, pitch, r, c,
         None if rows is None else _at8(rows, r, c, dev, "rows"),
         None if cols is None else _at8(cols, c, r, dev, "cols"))


def transpose(m: Matrix8, out: Matrix8):
    """The transpose of an 8-bit matrix, scaled anew along the other side."""
    _run(m.device, lib().shampoo_transpose8, m.ptr, _at8(out, m.cols, m.rows, m.device, "out"))


def matmul(a: Matrix8, b: Matrix8, out, accumulate: bool = False):
    """out (a.rows x b.rows; fp32, bf16 or fp16) = A B^T, or out + A B^T."""
    dev = a.device
    L = lib()
    _at8(b, b.rows, a.cols, dev, "b")
    at, code, pitch = _wide(out, a.rows, b.rows, dev, "out")
    need = _matmul_workspace(a.rows, b.rows, a.cols, code)
    work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _run(dev, L.shampoo_matmul8, a.ptr, b.ptr, at, code, pitch, 1 if accumulate else 0,
         work.data_ptr() if need else None, need)


_size = ctypes.c_size_t


def _workspace(fn, *sizes):
    out = _size()
    _check(fn(*sizes, ctypes.byref(out)), fn.__name__)
    return out.value


@functools.lru_cache(maxsize=4096)
def _matmul_workspace(m, n, k, code):     # by the sizes alone
    return _workspace(lib().shampoo_matmul8_workspace, m, n, k, code)


@functools.lru_cache(maxsize=4096)
def _norm_workspace(rows, dim):
    return _workspace(lib().shampoo_rms_norm8_backward_workspace, rows, dim)


# RmsNormArgs and RmsNormGradArgs as bytes: a third of the time that a ctypes
# structure of twenty fields takes
_pack_norm = struct.Struct("=2q7Q4q4id").pack
_pack_norm_grad = struct.Struct("=2q7Q4q4i").pack
assert struct.calcsize("=2q7Q4q4id") == ctypes.sizeof(RmsNormArgs)
assert struct.calcsize("=2q7Q4q4i") == ctypes.sizeof(RmsNormGradArgs)


def rms_norm(x, weight, eps: float, *, residual=None, total=None, out8: Optional[Matrix8] = None,
             out=None, rstd=None):
    """z = x + residual (into ``total``, in the residual's type; without a
    residual z is x), r = 1 / sqrt(mean(z^2) + eps) over each row (into
    ``rstd``), h = (z r) weight into ``out8`` (e4m3), ``out``, or both.
    total may be the residual or x itself."""
    dev = x.device
    rows, dim = _shape(x, "x")
    xp, xt, xs = _wide(x, rows, dim, dev, "x")
    rp = rt = rs = tp = ts = op = ot = os = 0
    if residual is not None and total is not None:
        rp, rt, rs = _wide(residual, rows, dim, dev, "residual")
        tp, tt, ts = _wide(total, rows, dim, dev, "total")
        if tt != rt:
            raise ValueError(f"total has the residual's type, {residual.dtype}")
    elif residual is not None or total is not None:
        raise ValueError("a residual and total are given together")
    if out is not None:
        op, ot, os = _wide(out, rows, dim, dev, "out")
    a = _pack_norm(rows, dim, xp, rp, tp, _vector(weight, dim, dev, "weight"),
                   0 if rstd is None else _vector(rstd, rows, dev, "rstd", _F32),
                   0 if out8 is None else _at8(out8, rows, dim, dev, "out8"), op,
                   xs, rs, ts, os, xt, rt, _TYPES[weight.dtype], ot, eps)
    _run(dev, lib().shampoo_rms_norm8, a)


def rms_norm_backward(grad, z, rstd, weight, *, dz, add=None, dw=None, accumulate: bool = False):
    """The gradient of rms_norm for grad = dL/dh, with z (its ``total``, or x)
    and rstd from it: into ``dz`` that of x and of the residual, ``add`` (the
    gradient that reaches z otherwise) included, and into ``dw`` (fp32) that of
    the weight, or added to what is there.  dz has z's type and may be add,
    grad or z itself."""
    dev = z.device
    rows, dim = _shape(z, "z")
    gp, gt, gs = _wide(grad, rows, dim, dev, "grad")
    zp, zt, zs = _wide(z, rows, dim, dev, "z")
    dp, dt, ds = _wide(dz, rows, dim, dev, "dz")
    ap = at = as_ = 0
    if add is not None:
        ap, at, as_ = _wide(add, rows, dim, dev, "add")
    if dt != zt or (add is not None and at != zt):
        raise ValueError(f"dz and add have z's type, {z.dtype}")
    wp = need = work = 0
    if dw is not None:
        wp = _vector(dw, dim, dev, "dw", _F32)
        need = _norm_workspace(rows, dim)
        work = torch.empty(need, dtype=torch.uint8, device=dev)
    a = _pack_norm_grad(rows, dim, gp, zp, _vector(rstd, rows, dev, "rstd", _F32),
                        _vector(weight, dim, dev, "weight"), ap, dp, wp,
                        gs, zs, as_, ds, gt, zt, _TYPES[weight.dtype], 1 if accumulate else 0)
    _run(dev, lib().shampoo_rms_norm8_backward, a, work.data_ptr() if need else None, need)


class Weights8(_Bound):
    """8-bit copies of many weights and of their transposes (e4m3, one scale for
    each 128 x 128 values, so that both hold the same values): ``rows[i]`` is
    weight i, ``cols[i]`` its transpose, each a Matrix8 in the handle's state."""

    def __init__(self, shapes: Sequence[Tuple[int, int]], param: str = "f32", device="cuda"):
        L = lib()
        self._destroy = L.shampoo_weights8_destroy
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        self.want = [(r * c, DTYPES[param]) for r, c in self.shapes]
        descs = (WeightDesc * max(len(self.shapes), 1))(*[WeightDesc(r, c, DTYPES[param], 0) for r, c in self.shapes])
        h = _P()
        _check(L.shampoo_weights8_create(len(self.shapes), descs, ctypes.byref(h)), "shampoo_weights8_create")
        self.h = h
        self._open(device)
        lay = Weights8Layout()
        _check(L.shampoo_weights8_get_layout(h, ctypes.byref(lay)), "shampoo_weights8_get_layout")
        self.state = torch.empty(lay.total, dtype=torch.uint8, device=self.device)
        self._call(L.shampoo_weights8_bind_state, self.state.data_ptr(), lay.total)
        #: all codes and all scales, one copy after another
        self.codes = self.state[lay.off_codes:lay.off_codes + lay.code_bytes].view(torch.float8_e4m3fn)
        self.scales = self.state[lay.off_scales:lay.off_scales + lay.scale_bytes]
        self.rows = [self._matrix(i, 0) for i in range(len(self.shapes))]
        self.cols = [self._matrix(i, 1) for i in range(len(self.shapes))]
        self._held = None

    def _matrix(self, i, transposed):
        d = Matrix8Desc()
        _check(lib().shampoo_weights8_matrix(self.h, i, transposed, ctypes.byref(d)), "shampoo_weights8_matrix")
        base = self.state.data_ptr()
        at, groups = d.codes - base, -(-d.cols // (4 * BLOCK))
        codes = self.state[at:at + d.rows * d.pitch].view(torch.float8_e4m3fn).view(d.rows, d.pitch)
        at = d.scales - base
        scales = self.state[at:at + 4 * groups * d.rows].view(groups, d.rows, 4)
        return Matrix8(d.rows, d.cols, "e4m3", codes=codes, scales=scales)

    def bind(self, weights):
        """The weights from now on: contiguous tensors of the plan's shapes, flat
        ones, or ones of more dimensions that are the plan's two taken apart
        (out x in x 3 x 3 for out rows)."""
        weights = list(weights)
        at = self._addresses(weights, self.want, "weights")
        for i, (t, (r, c)) in enumerate(zip(weights, self.shapes)):
            if t is not None and t.dim() > 1 and r not in itertools.accumulate(t.shape[:-1], operator.mul):
                raise ValueError(f"weights[{i}] must have {r} rows of {c} elements, got {tuple(t.shape)}")
        self._call(lib().shampoo_weights8_bind_weights, at)
        self._held = weights
        self._spans = [(i, t.data_ptr(), t.data_ptr() + t.nbytes) for i, t in enumerate(weights)
                       if t is not None and t.nbytes]

    def _stepped(self, params):
        """Refuses params, the tensors of a step, that a bound weight is not one
        or a part of: its copies would stay those of a tensor left behind."""
        if self._held is None:
            raise ValueError("copies8: no weights are bound")
        params = [p for p in params or () if p is not None]
        sizes = {p.data_ptr(): p.nbytes for p in params}
        starts = reach = None
        for i, low, high in self._spans:
            if sizes.get(low, 0) >= high - low:
                continue
            if starts is None:       # parts of tensors: how far memory goes from each start on
                spans = sorted((p.data_ptr(), p.data_ptr() + p.nbytes) for p in params)
                starts = [at for at, _ in spans]
                reach = list(itertools.accumulate((end for _, end in spans), max))
            k = bisect.bisect_right(starts, low) - 1
            if k < 0 or reach[k] < high:
                raise ValueError(f"copies8: weights[{i}] is not of the tensors that this step changes; bind the "
                                 "present ones, or call refresh() where several steps share the copies")

    def refresh(self):
        """Copies of the bound weights as they are now (one launch)."""
        self._call(lib().shampoo_weights8_refresh)
