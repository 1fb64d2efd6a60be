"""First-order operators of libshampoo_mi355x.so (ctypes; argument marshalling
only): one AdamW step over many tensors at once, with moments in 32 or in 8
bits, and the global gradient norm whose clip coefficient it reads.

    specs = [adamw.tensor(p.numel(), param="bf16", grad="bf16", state_bits=8) for p in params]
    opt = adamw.AdamW(specs, adamw.make_config(beta2=0.95))
    norm = adamw.GradNorm([(g.numel(), "bf16") for g in grads])
    opt.bind(params, grads)
    norm.bind(grads)
    for t in range(steps):
        ...                               # gradients into the bound tensors
        norm.compute(max_norm=1.0)
        opt.step(lr=1e-3, clip=norm)

Beside Shampoo, GradNorm takes the gradients of both optimizers and
``clip_into`` writes the fp32 ones that Shampoo.step takes: zeros where the norm
is not finite, with which a Shampoo step still decays its statistics (beta2 < 1)
and moves weights by its momentum; to leave that step out as AdamW does, read
``nonfinite`` first.  ``bind``,
``compute``, ``clip_into`` and ``step`` neither wait for the GPU nor copy to it,
and can be captured into a graph; what is bound or captured stays alive, and is
used by one stream at a time.  It raises if the library has not been built --
there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence, Tuple

from .shampoo import (AdamWConfig, AdamWLayout, AdamWTensor, GradDesc, ShampooError, _check, _P,
                      lib)

DTYPES = {"f32": 0, "bf16": 1, "f16": 2}
RUN = 256          # elements of a run: the unit of a tensor's place in the state


def make_config(*, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                seed: int = 0) -> AdamWConfig:
    """seed (32 bits): of the rounding of 8-bit moments."""
    if not 0 <= seed < 1 << 32:
        raise ValueError("seed must fit 32 bits")
    return AdamWConfig(beta1, beta2, eps, seed, 0)


def tensor(numel: int, *, param: str = "f32", grad: Optional[str] = None, state_bits: int = 32,
           weight_decay: float = 0.0, lr_scale: float = 1.0) -> AdamWTensor:
    """One tensor of a plan.  param: "f32" or "bf16" (whose rounding error the
    state keeps in 16 bits more); grad: "f32", "bf16" or "f16" (default: as
    param)."""
    return AdamWTensor(int(numel), DTYPES[param], DTYPES[grad or param], state_bits, 0,
                       weight_decay, lr_scale)


class _Bound:
    """What both handles share: the device, its stream, and tensors as
    addresses that stay alive while they are bound."""

    def _open(self, device):
        import torch
        self.torch = torch
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        if dev.type != "cuda":
            raise ValueError(f"no kernels for {dev}")
        self.device = dev
        self._types = (torch.float32, torch.bfloat16, torch.float16)

        # the current stream of a device as a number, without a Stream object
        # where torch offers that (0.1 us instead of 1.9)
        self._stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                               lambda index: torch.cuda.current_stream(index).cuda_stream)
        self._current = torch.cuda.current_device

    def _call(self, fn, *args):
        """fn(handle, *args, stream) with the handle's device current."""
        index = self.device.index
        if self._current() == index:
            rc = fn(self.h, *args, self._stream(index))
        else:
            with self.torch.cuda.device(index):
                rc = fn(self.h, *args, self._stream(index))
        if rc:
            _check(rc, fn.__name__)

    def _addresses(self, ts, want, what, optional=False):
        """want: (numel, dtype code) of each tensor."""
        if len(ts) != len(want):
            raise ValueError(f"{what}: {len(ts)} tensors for a plan of {len(want)}")
        arr = (_P * len(want))()
        for i, (t, (n, dt)) in enumerate(zip(ts, want)):
            if t is None:
                if not optional and n:
                    raise ValueError(f"{what}[{i}] is required")
                continue
            if (t.dtype != self._types[dt] or not t.is_contiguous() or t.device != self.device
                    or t.numel() != n):
                raise ValueError(f"{what}[{i}] must be a contiguous {self._types[dt]} tensor of "
                                 f"{n} elements on {self.device}")
            arr[i] = t.data_ptr() if n else None
        return arr

    def close(self):
        if getattr(self, "h", None):
            self._destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GradNorm(_Bound):
    """Global norm of the gradients of many tensors: [(numel, dtype), ...]."""

    def __init__(self, tensors: Sequence[Tuple[int, str]], device="cuda"):
        L = lib()
        self._destroy = L.shampoo_gradnorm_destroy
        self.want = [(int(n), DTYPES[dt]) for n, dt in tensors]
        descs = (GradDesc * len(self.want))(*[GradDesc(n, dt, 0) for n, dt in self.want])
        h = _P()
        _check(L.shampoo_gradnorm_create(len(self.want), descs, ctypes.byref(h)),
               "shampoo_gradnorm_create")
        self.h = h
        self._open(device)
        size = ctypes.c_size_t()
        _check(L.shampoo_gradnorm_state_bytes(h, ctypes.byref(size)), "shampoo_gradnorm_state_bytes")
        self.state = self.torch.empty(size.value, dtype=self.torch.uint8, device=self.device)
        self._call(L.shampoo_gradnorm_bind_state, self.state.data_ptr(), size.value)
        at = _P()
        _check(L.shampoo_gradnorm_record(h, ctypes.byref(at)), "shampoo_gradnorm_record")
        self.record_ptr = at.value
        self.computed = False
        off = at.value - self.state.data_ptr()
        #: [norm, coefficient] of the last compute, on the device
        self.record = self.state[off:off + 8].view(self.torch.float32)
        #: 1 where that norm is not finite, or none has run yet, on the device
        self.nonfinite = self.state[off + 8:off + 12].view(self.torch.int32)

    def bind(self, grads, outs=None):
        """Gradients from now on (None: absent), and the fp32 tensors that
        clip_into fills (the gradient itself where it is fp32, or memory of its
        own; None: none)."""
        g = self._addresses(grads, self.want, "grads", optional=True)
        o = None
        if outs is not None:
            o = self._addresses(outs, [(n, 0) for n, _ in self.want], "outs", optional=True)
        self._call(lib().shampoo_gradnorm_bind_grads, g, o)
        self._held = (list(grads), None if outs is None else list(outs))

    def compute(self, max_norm: float = float("inf"), grad_scale: float = 1.0):
        """Norm and coefficient of the bound gradients into ``record``."""
        self._call(lib().shampoo_gradnorm_compute, max_norm, grad_scale)
        self.computed = True

    def clip_into(self):
        """The clipped gradients into the bound outputs."""
        self._call(lib().shampoo_gradnorm_clip_into)


class AdamW(_Bound):
    """One AdamW step over many tensors (specs from ``tensor``).

    per_tensor_steps: the bias corrections count the steps in which a tensor had
    a gradient, for tensors whose gradients start late or come now and then.
    Otherwise they count the handle's steps, and a first gradient after a
    thousand of them moves its tensor by 2.5 lr."""

    def __init__(self, tensors: Sequence[AdamWTensor], cfg: Optional[AdamWConfig] = None,
                 device="cuda", per_tensor_steps: bool = False):
        L = lib()
        self._destroy = L.shampoo_adamw_destroy
        self.tensors = list(tensors)
        self.cfg = make_config() if cfg is None else cfg
        descs = (AdamWTensor * len(self.tensors))(*self.tensors)
        h = _P()
        _check(L.shampoo_adamw_create(ctypes.byref(self.cfg), len(self.tensors), descs,
                                      ctypes.byref(h)), "shampoo_adamw_create")
        self.h = h
        self.per_tensor_steps = bool(per_tensor_steps)
        _check(L.shampoo_adamw_set_counting(h, int(self.per_tensor_steps)), "shampoo_adamw_set_counting")
        self.layout = AdamWLayout()
        _check(L.shampoo_adamw_get_layout(h, ctypes.byref(self.layout)), "shampoo_adamw_get_layout")
        self._open(device)
        self.state = self.torch.empty(self.layout.total, dtype=self.torch.uint8, device=self.device)
        self._call(L.shampoo_adamw_bind_state, self.state.data_ptr(), self.layout.total)
        self._held = [None, None]

    def bind(self, params=None, grads=None):
        """Weights and gradients from now on; None keeps those bound before.
        A gradient that is None leaves its tensor as it is."""
        p = g = None
        if params is not None:
            p = self._addresses(params, [(t.numel, t.param_type) for t in self.tensors], "params")
        if grads is not None:
            g = self._addresses(grads, [(t.numel, t.grad_type) for t in self.tensors], "grads",
                                optional=True)
        self._call(lib().shampoo_adamw_bind_tensors, p, g)
        self._held = [self._held[0] if params is None else list(params),
                      self._held[1] if grads is None else list(grads)]

    def step(self, lr, clip: Optional[GradNorm] = None):
        """One step.  lr: a number, or one fp32 element on the device that the
        step reads when it runs.  clip: scale the gradients by the coefficient
        of its last compute, and skip the step where its norm is not finite.
        The gradients are those before clipping: not ones that clip_into has
        scaled in place."""
        dev_lr = None
        if isinstance(lr, self.torch.Tensor):
            if lr.dtype != self.torch.float32 or lr.numel() != 1 or lr.device != self.device:
                raise ValueError(f"lr must be a number or one fp32 element on {self.device}")
            dev_lr, lr = lr.data_ptr(), 0.0
        if clip is not None and (clip.device != self.device or not clip.computed):
            raise ValueError(f"clip must be on {self.device} and have computed a norm")
        self._call(lib().shampoo_adamw_step, lr, dev_lr, None if clip is None else clip.record_ptr)

    def set_step(self, t: int):
        """Set the number of steps done, the handle's and every tensor's own,
        e.g. after restoring the moments."""
        self._call(lib().shampoo_adamw_set_step, t)

    def set_tensor_steps(self, steps: Sequence[int]):
        """Set every tensor's own number of steps (with per_tensor_steps)."""
        if len(steps) != len(self.tensors):
            raise ValueError(f"{len(steps)} counts for a plan of {len(self.tensors)}")
        self._call(lib().shampoo_adamw_set_tensor_steps, (ctypes.c_int64 * len(self.tensors))(*steps))

    def tensor_steps(self) -> List[int]:
        """Every tensor's own number of steps, 0 for an empty one (waits for the
        GPU)."""
        at = []
        for i in range(len(self.tensors)):
            off = ctypes.c_int64()
            _check(lib().shampoo_adamw_tensor_count(self.h, i, ctypes.byref(off)),
                   "shampoo_adamw_tensor_count")
            at.append(off.value)
        index = self.torch.tensor([max(o, 0) // 8 for o in at], device=self.device)
        got = self.state.view(self.torch.int64)[index].tolist()
        return [k if o >= 0 else 0 for k, o in zip(got, at)]

    # ---- views into the state buffer
    def _view(self, off, count, dtype):
        es = self.torch.empty((), dtype=dtype).element_size()
        return self.state[off:off + count * es].view(dtype)

    @property
    def t(self):
        """Steps done: one int64 on the device."""
        return self._view(self.layout.off_clock, 1, self.torch.int64)

    def state_tensors(self) -> Dict[str, object]:
        """The moments and remainders of every tensor, one after another in
        whole runs of 256 elements: "m", "v" in fp32; "m8", "s8" as e4m3
        values of m and sqrt(v) with their scales "m_scale", "s_scale" (one per
        run); "rem", what bf16 weights lack of their fp32 value (zero it when
        the weights are replaced)."""
        lay, t = self.layout, self.torch
        out = {}
        if lay.runs32:
            out["m"] = self._view(lay.off_m, lay.runs32 * RUN, t.float32)
            out["v"] = self._view(lay.off_v, lay.runs32 * RUN, t.float32)
        if lay.runs8:
            out["m8"] = self._view(lay.off_m8, lay.runs8 * RUN, t.float8_e4m3fn)
            out["s8"] = self._view(lay.off_s8, lay.runs8 * RUN, t.float8_e4m3fn)
            out["m_scale"] = self._view(lay.off_m_scale, lay.runs8, t.float32)
            out["s_scale"] = self._view(lay.off_s_scale, lay.runs8, t.float32)
        if lay.runs_rem:
            out["rem"] = self._view(lay.off_rem, lay.runs_rem * RUN, t.int16)
        return out

    def state_dict(self) -> Dict[str, object]:
        """Copies of the moments and remainders, and the number of steps done
        (waits for the GPU)."""
        out = {"t": int(self.t), **{k: x.clone() for k, x in self.state_tensors().items()}}
        if self.per_tensor_steps:
            out["tensor_steps"] = self.tensor_steps()
        return out

    def load_state_dict(self, saved: Dict[str, object]):
        """Restore what ``state_dict`` of a handle with the same tensors gave."""
        held = self.state_tensors()
        names = {"t", *held} | ({"tensor_steps"} if self.per_tensor_steps else set())
        counts = saved.get("tensor_steps", [])
        if (set(saved) != names or len(counts) != len(self.tensors) * self.per_tensor_steps
                or any(saved[k].shape != x.shape or saved[k].dtype != x.dtype for k, x in held.items())):
            raise ValueError("the state is of other tensors, or counts their steps in another way")
        if any(t < 0 for t in (saved["t"], *counts)):      # before anything is changed
            raise ValueError("a number of steps is not negative")
        for k, x in held.items():
            x.copy_(saved[k])
        self.set_step(saved["t"])
        if self.per_tensor_steps:
            self.set_tensor_steps(counts)
