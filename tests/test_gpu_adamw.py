"""The first-order operators on the GPU against the fp64 oracle: one AdamW step
over many tensors with moments in 32 and in 8 bits, and the global gradient
norm.  Every bound is the oracle's count of fp32 roundings along the formula."""
import ctypes

import numpy as np
import pytest

from oracle import adamw_oracle as O
from second_order_optimizer_amd import adamw as A
from second_order_optimizer_amd import shampoo as S

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FILLER = 1 << 20        # tensors larger than this only fill a plan and are not checked
GUARD = 16      # elements beside a tensor that nothing may touch
SENTINEL = -77.0


def np64(t):
    return t.detach().double().cpu().numpy()


def guarded(values, dtype, offset):
    """A device tensor of `values` inside a buffer of sentinels, starting
    `offset` elements past an aligned address; and the buffer."""
    n = values.size
    buf = torch.full((n + 2 * GUARD + 4,), SENTINEL, dtype=dtype, device="cuda")
    t = buf[GUARD + offset:GUARD + offset + n]
    t.copy_(torch.from_numpy(values).to(dtype))
    return t, buf


def untouched(buf, offset, n):
    b = buf.float().cpu().numpy()
    assert np.all(b[:GUARD + offset] == SENTINEL) and np.all(b[GUARD + offset + n:] == SENTINEL)


class Run:
    """An AdamW handle over tensors with random weights, gradients and moments,
    and the oracle's check of one step of it."""

    def __init__(self, specs, seed, *, offset=0, beta1=0.9, beta2=0.999, eps=1e-8, t0=0, warm=True):
        self.rng = np.random.default_rng(seed)
        self.specs, self.offset = specs, offset
        self.cfg = A.make_config(beta1=beta1, beta2=beta2, eps=eps, seed=seed)
        self.opt = A.AdamW(specs, self.cfg)
        self.types = [("f32", "bf16")[s.param_type] for s in specs]
        self.gtypes = [("f32", "bf16", "f16")[s.grad_type] for s in specs]
        self.sigma = [10 ** self.rng.uniform(-4, 0) for _ in specs]
        self.params, self.grads, self.bufs = [], [], []
        for s, dt in zip(specs, self.types):
            w = (0.02 * self.rng.standard_normal(min(s.numel, FILLER))).astype(np.float32)
            w = np.resize(w, s.numel)
            t, b = guarded(w, TORCH[dt], offset)
            self.params.append(t)
            self.bufs.append((b, s.numel))
        for i in range(len(specs)):
            t, b = guarded(self.draw(i), TORCH[self.gtypes[i]], offset)
            self.grads.append(t)
            self.bufs.append((b, specs[i].numel))
        if warm:
            self.warm()
        self.opt.set_step(t0)
        self.t = t0
        self.opt.bind(self.params, self.grads)

    def draw(self, i):
        if self.specs[i].numel > FILLER:
            return np.zeros(self.specs[i].numel, np.float32)
        return (self.sigma[i] * self.rng.standard_normal(self.specs[i].numel)).astype(np.float32)

    def place(self, i):
        st, rm = ctypes.c_int64(), ctypes.c_int64()
        assert S.lib().shampoo_adamw_tensor_runs(self.opt.h, i, ctypes.byref(st), ctypes.byref(rm)) == 0
        return st.value, rm.value

    def parts(self, i):
        """Views of tensor i's state: elements, and its runs' scales."""
        s, held = self.specs[i], self.opt.state_tensors()
        st, rm = self.place(i)
        n, runs = s.numel, -(-s.numel // 256)
        cut = lambda x, r: x[r * 256:r * 256 + n]
        out = {}
        if n == 0:
            return out
        if s.state_bits == 32:
            out.update(m=cut(held["m"], st), v=cut(held["v"], st))
        else:
            out.update(m8=cut(held["m8"].view(torch.uint8), st), s8=cut(held["s8"].view(torch.uint8), st),
                       m_scale=held["m_scale"][st:st + runs], s_scale=held["s_scale"][st:st + runs])
        if rm >= 0:
            out["rem"] = cut(held["rem"], rm)
        return out

    def warm(self):
        for i, s in enumerate(self.specs):
            q = self.parts(i)
            n, runs = s.numel, -(-s.numel // 256)
            if n > FILLER:
                continue
            if "m" in q:
                q["m"].copy_(torch.from_numpy(0.3 * self.draw(i)))
                q["v"].copy_(torch.from_numpy(self.draw(i) ** 2))
            elif n:
                q["m8"].copy_(torch.from_numpy(self.codes(n, True)))
                q["s8"].copy_(torch.from_numpy(self.codes(n, False)))
                for k in ("m_scale", "s_scale"):
                    x = self.sigma[i] / 448 * (0.5 + self.rng.random(runs))
                    q[k].copy_(torch.from_numpy(x.astype(np.float32)))
            if "rem" in q:
                q["rem"].copy_(torch.from_numpy(self.rng.integers(-32768, 32768, n).astype(np.int16)))

    def codes(self, n, signed):
        c = self.rng.integers(0, 127, n)
        if signed:
            c |= 128 * self.rng.integers(0, 2, n)
        return c.astype(np.uint8)

    def read(self):
        """Weights (as fp32 values), moments and their errors, in fp64."""
        got = []
        for i, s in enumerate(self.specs):
            q = {k: x.cpu().numpy().copy() for k, x in self.parts(i).items()}
            w = self.params[i].detach().cpu()
            if s.numel > FILLER:
                got.append(q)
                continue
            if "rem" in q:
                q["p"] = O.bf16_join(w.view(torch.int16).numpy().view(np.uint16), q["rem"]).astype(np.float64)
            else:
                q["p"] = w.double().numpy()
            if "m8" in q:
                n = s.numel
                q["m"] = O.decode(q["m8"]) * np.repeat(q["m_scale"].astype(np.float64), 256)[:n]
                root = O.decode(q["s8"]) * np.repeat(q["s_scale"].astype(np.float64), 256)[:n]
                q["v"] = root * root
                q["m_err"], q["v_err"] = O.U * np.abs(q["m"]), 3 * O.U * q["v"]
            elif s.numel:
                q["m"], q["v"] = q["m"].astype(np.float64), q["v"].astype(np.float64)
                q["m_err"] = q["v_err"] = 0.0
            else:
                q["m"] = q["v"] = np.zeros(0)
                q["m_err"] = q["v_err"] = 0.0
            q["g"] = np64(self.grads[i]) if self.grads[i] is not None else None
            got.append(q)
        return got

    def hyper(self, i, lr):
        s, c = self.specs[i], self.cfg
        return O.Hyper(c.beta1, c.beta2, c.eps, lr, s.weight_decay, s.lr_scale)

    def check(self, before, lr, coef=1.0):
        """The state now is one step on from `before`."""
        self.t += 1
        assert int(self.opt.t) == self.t
        after = self.read()
        for i, (a, b) in enumerate(zip(before, after)):
            s = self.specs[i]
            if s.numel == 0 or s.numel > FILLER:
                continue
            # eps and the scalars reach the kernel as fp32: within U of these
            p, m, root, v, pe, me, re, ve = O.step(a["p"], a["g"], a["m"], a["v"], self.t,
                                                   self.hyper(i, lr), coef, a["m_err"], a["v_err"])
            assert np.all(np.abs(b["p"] - p) <= pe), (i, np.max(np.abs(b["p"] - p) / pe))
            if s.state_bits == 32:
                assert np.all(np.abs(b["m"] - m) <= me), i
                assert np.all(np.abs(b["v"] - v) <= ve), i
                continue
            rm, rs = O.random_bits(self.cfg.seed, self.t, i, np.arange(s.numel))
            for x, xe, code, scale, r, pos in ((m, me, "m8", "m_scale", rm, False),
                                               (root, re, "s8", "s_scale", rs, True)):
                want = O.run_scales(x)
                top = np.maximum.reduceat(xe, np.arange(0, s.numel, 256))
                assert np.all(np.abs(b[scale] - want) <= top / 448 + 3 * O.U * want), (i, scale)
                lo, hi = O.store_range(x, xe, want, r, pos)
                z = O.decode(b[code])
                assert np.all((np.abs(z) >= lo) & (np.abs(z) <= hi)), (i, code)
                sure = (lo > 0) & (np.abs(x) > xe)
                assert np.all((np.sign(z) == np.sign(x))[sure])
                if pos:
                    assert np.all(z[root > re] > 0)

    def rest_untouched(self):
        for b, n in self.bufs:
            untouched(b, self.offset, n)
        for i, s in enumerate(self.specs):      # state behind the last element stays 0
            if s.numel % 256 == 0:
                continue
            st, rm = self.place(i)
            held = self.opt.state_tensors()
            names = [("m", st), ("v", st)] if s.state_bits == 32 else [("m8", st), ("s8", st)]
            for name, r in names + ([("rem", rm)] if rm >= 0 else []):
                x = held[name].view(torch.uint8) if "8" in name else held[name]
                gap = x[r * 256 + s.numel:(r + -(-s.numel // 256)) * 256]
                assert not bool(gap.any()), (i, name)


SIZES = [1, 2, 3, 5, 63, 255, 256, 257, 0, 511, 512, 513, 1000, 2047, 4097, 70001]


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"),
                                        ("bf16", "bf16"), ("bf16", "f32"), ("bf16", "f16")])
def test_step(param, grad, bits, offset):
    rng = np.random.default_rng(offset)
    specs = [A.tensor(n, param=param, grad=grad, state_bits=bits,
                      weight_decay=float(rng.choice([0.0, 0.1])), lr_scale=float(rng.choice([1.0, 0.5])))
             for n in SIZES]
    run = Run(specs, 11 + offset, offset=offset, t0=offset * 40)
    for lr in (1e-3, 3e-4, 0.0):
        before = run.read()
        run.opt.step(lr)
        run.check(before, lr)
        for i, g in enumerate(run.grads):
            g.copy_(torch.from_numpy(run.draw(i)))
    run.rest_untouched()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"),
                                        ("bf16", "bf16"), ("bf16", "f32"), ("bf16", "f16")])
def test_step_past_the_caches(param, grad, bits):
    """A plan of more than 96 MiB takes the kernels that pass the caches by."""
    specs = [A.tensor(n, param=param, grad=grad, state_bits=bits, weight_decay=0.1) for n in SIZES]
    run = Run(specs[:8] + [A.tensor(13 << 20, param=param, grad=grad, state_bits=bits)] + specs[8:], 31, offset=1)
    for lr in (1e-3, 3e-4):
        before = run.read()
        run.opt.step(lr)
        run.check(before, lr)
        for i, g in enumerate(run.grads):
            g.copy_(torch.from_numpy(run.draw(i)))
    run.rest_untouched()


def test_saved_and_restored():
    """Steps after a restored state are the steps that would have followed."""
    specs = [A.tensor(n, param=p, state_bits=b, grad="bf16") for n in (700, 5000) for p in ("f32", "bf16") for b in (32, 8)]
    a, b = Run(specs, 4), Run(specs, 4, warm=False)
    for _ in range(3):
        a.opt.step(1e-3)
    saved = a.opt.state_dict()
    for x, y in zip(b.params, a.params):
        x.copy_(y)
    b.opt.load_state_dict(saved)
    for r in (a, b):
        for _ in range(2):
            r.opt.step(1e-3)
    assert int(b.opt.t) == 5
    for x, y in zip(a.read(), b.read()):
        for k in x:
            assert np.array_equal(x[k], y[k], equal_nan=True), k
    with pytest.raises(ValueError):
        A.AdamW(specs[:3]).load_state_dict(saved)


def test_first_steps_from_nothing():
    """From zero moments, with t from 1: 8-bit runs whose values are all zero,
    and runs where only some gradients are not."""
    specs = [A.tensor(n, state_bits=b) for n in (300, 1024) for b in (32, 8)]
    run = Run(specs, 5, warm=False)
    for k in range(4):
        for i, g in enumerate(run.grads):
            x = run.draw(i)
            x[k::3] = 0.0
            x[:256 if k == 0 else 0] = 0.0
            g.copy_(torch.from_numpy(x))
        before = run.read()
        run.opt.step(1e-2)
        run.check(before, 1e-2)


@pytest.mark.parametrize("beta1,beta2,eps,t0", [(0.0, 0.0, 1e-8, 0), (0.9, 0.95, 1e-6, 3), (0.99, 0.9999, 1e-15, 100000)])
def test_hyperparameters(beta1, beta2, eps, t0):
    specs = [A.tensor(5000, state_bits=b, weight_decay=0.01) for b in (32, 8)]
    run = Run(specs, 3, beta1=beta1, beta2=beta2, eps=eps, t0=t0)
    for _ in range(3):
        before = run.read()
        run.opt.step(1e-3)
        run.check(before, 1e-3)


@pytest.mark.parametrize("exponent", [-30, -20, -12, 12])
def test_range_of_gradients(exponent):
    """Gradients whose squares leave the normal range of fp32 on the low side,
    and large ones."""
    specs = [A.tensor(2000, state_bits=b) for b in (32, 8)]
    run = Run(specs, 9, warm=False, eps=1e-20 if exponent < 0 else 1e-8)
    for i, g in enumerate(run.grads):
        g.copy_(torch.from_numpy((run.rng.standard_normal(2000) * 10.0 ** exponent).astype(np.float32)))
    for _ in range(2):
        before = run.read()
        run.opt.step(1e-3)
        run.check(before, 1e-3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", ["usual", "wide", "low", "zeros"])
def test_every_rounding(kind, bits):
    """Bit for bit the fp32 operations of the formula, each rounded to nearest,
    over the range of fp32: roots of denormal and of huge second moments, small
    and large quotients."""
    n = 64 * 256
    rng = np.random.default_rng(len(kind))
    lo, hi = {"usual": (-3, 0), "wide": (-21, 18), "low": (-24, -12), "zeros": (-6, 0)}[kind]
    draw = lambda: (rng.standard_normal(n) * 10.0 ** rng.uniform(lo, hi, n)).astype(np.float32)
    h = O.Hyper(lr=1e-3, weight_decay=0.1, eps=1e-25 if kind == "low" else 1e-8)
    opt = A.AdamW([A.tensor(n, state_bits=bits, weight_decay=0.1)], A.make_config(eps=h.eps, seed=9))
    w = rng.standard_normal(n).astype(np.float32)
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    p, g = torch.from_numpy(w.copy()).cuda(), torch.zeros(n, device="cuda")
    opt.bind([p], [g])
    held = opt.state_tensors()
    same = lambda a, b: np.array_equal(np.asarray(a).view(np.uint32), np.asarray(b).view(np.uint32))
    for t in (1, 2, 3):
        x = draw()
        if kind == "zeros":
            x[rng.random(n) < 0.5] = 0.0
        g.copy_(torch.from_numpy(x))
        opt.step(h.lr)
        w, m, root, v = O.step32(w, x, m, v, t, h)
        assert np.isfinite(v).all()
        assert same(p.cpu().numpy(), w), t
        if bits == 32:
            assert same(held["m"].cpu().numpy(), m) and same(held["v"].cpu().numpy(), v)
            continue
        rm, rs = O.random_bits(9, t, 0, np.arange(n))
        for value, r, code, scale, pos in ((m, rm, "m8", "m_scale", False), (root, rs, "s8", "s_scale", True)):
            c, s = O.codes32(value, r, pos)
            assert same(held[scale].cpu().numpy(), s), (t, scale)
            assert np.array_equal(held[code].view(torch.uint8).cpu().numpy(), c), (t, code)
        spread = lambda k: np.repeat(held[k].cpu().numpy(), 256)
        dec = lambda k: O.decode(held[k].view(torch.uint8).cpu().numpy()).astype(np.float32)
        with np.errstate(under="ignore"):
            m = dec("m8") * spread("m_scale")
            root = dec("s8") * spread("s_scale")
            v = root * root


def test_many_tensors_of_mixed_kinds():
    """More tensors than one launch of the pointer kernel carries, every kind of
    them in one plan, some without a gradient."""
    rng = np.random.default_rng(2)
    specs = []
    for _ in range(450):
        param = ("f32", "bf16")[rng.integers(2)]
        specs.append(A.tensor(int(rng.integers(0, 900)), param=param, grad=("f32", "bf16", "f16")[rng.integers(3)],
                              state_bits=int(rng.choice([8, 32])), weight_decay=float(rng.choice([0, 0.1]))))
    run = Run(specs, 21, offset=1)
    absent = set(range(0, 450, 7))
    grads = [None if i in absent else g for i, g in enumerate(run.grads)]
    run.opt.bind(grads=grads)
    before = run.read()
    run.opt.step(1e-3)
    after = run.read()
    for i in absent:
        for k in ("p", "m", "v", "rem", "m8", "s8", "m_scale", "s_scale"):
            if k in before[i]:
                assert np.array_equal(before[i][k], after[i][k]), (i, k)
    run.opt.bind(grads=run.grads)      # and all of them again
    run.t += 1
    before = after
    run.opt.step(1e-3)
    run.check(before, 1e-3)
    run.rest_untouched()


def test_bf16_weights_are_the_fp32_ones():
    """bf16 weights with their remainder follow fp32 weights bit for bit."""
    n = 3001
    w = np.random.default_rng(1).standard_normal(n).astype(np.float32)
    hi, rem = O.bf16_split(w)
    p32 = torch.from_numpy(w).cuda()
    p16 = torch.from_numpy(hi.view(np.int16)).cuda().view(torch.bfloat16)
    a = A.AdamW([A.tensor(n, weight_decay=0.1)])
    b = A.AdamW([A.tensor(n, param="bf16", grad="f32", weight_decay=0.1)])
    b.state_tensors()["rem"][:n].copy_(torch.from_numpy(rem))
    g = torch.empty(n, device="cuda")
    a.bind([p32], [g])
    b.bind([p16], [g])
    for k in range(30):
        g.normal_(0, 10.0 ** (k % 5 - 3))
        a.step(1e-3)
        b.step(1e-3)
    got = O.bf16_join(p16.view(torch.int16).cpu().numpy().view(np.uint16),
                      b.state_tensors()["rem"][:n].cpu().numpy())
    assert np.array_equal(got.view(np.uint32), p32.cpu().numpy().view(np.uint32))


def test_not_finite_gradients_stay_where_they_are():
    """Without a clip, an infinite or NaN gradient spoils its own element, not
    its run."""
    n = 1000
    bad = {3: np.inf, 300: -np.inf, 301: np.nan, 999: np.nan}
    rest = np.setdiff1d(np.arange(n), list(bad))
    run = Run([A.tensor(n, state_bits=b) for b in (32, 8)], 4)
    for i, g in enumerate(run.grads):
        x = run.draw(i)
        x[list(bad)] = 0.0
        g.copy_(torch.from_numpy(x))
    twin = Run([A.tensor(n, state_bits=b) for b in (32, 8)], 4)
    for x, y in zip(run.grads, twin.grads):
        y.copy_(x)
    for g in run.grads:
        for k, v in bad.items():
            g[k] = v
    run.opt.step(1e-3)
    twin.opt.step(1e-3)
    a, b = run.read(), twin.read()
    for x, y in zip(a, b):
        assert np.array_equal(x["p"][rest], y["p"][rest])
        for k in ("m8", "s8", "m_scale", "s_scale"):
            if k in x and x[k].size == n:
                assert np.array_equal(x[k][rest], y[k][rest])
    assert np.array_equal(a[1]["s_scale"][1:3], b[1]["s_scale"][1:3])
    for k in bad:
        assert a[1]["s8"][k] == 127 and a[1]["m8"][k] & 127 == 127


def test_skips_a_step_that_is_not_finite():
    run = Run([A.tensor(3000, state_bits=b, param=p, grad="bf16") for b in (32, 8) for p in ("f32", "bf16")], 6)
    norm = A.GradNorm([(3000, "bf16")] * 4)
    norm.bind(run.grads)
    run.grads[2][1234] = float("inf")
    before = run.read()
    norm.compute(1.0)
    run.opt.step(1e-3, clip=norm)
    after = run.read()
    assert int(run.opt.t) == 0 and int(norm.nonfinite) == 1 and float(norm.record[1]) == 0.0
    for a, b in zip(before, after):
        for k in a:
            assert np.array_equal(a[k], b[k], equal_nan=True), k
    run.grads[2][1234] = 1.0
    before = run.read()
    norm.compute(1.0)
    run.opt.step(1e-3, clip=norm)
    run.check(before, 1e-3, float(norm.record[1]))


def test_rounding_is_fair():
    """The mean of what is stored is the value: over the 2^16 elements of equal
    moments, within 6 standard deviations of a fair choice between the two
    codes next to it."""
    n = 1 << 16
    opt = A.AdamW([A.tensor(n, state_bits=8)], A.make_config(beta1=0.5, beta2=0.5, seed=3))
    g = torch.full((n,), 0.37, device="cuda")
    g[::256] = 1.0           # sets each run's scale
    p = torch.zeros(n, device="cuda")
    opt.bind([p], [g])
    opt.step(1e-3)
    held = opt.state_tensors()
    keep = np.arange(n) % 256 != 0
    for name, scale, x in (("m8", "m_scale", 0.5 * 0.37), ("s8", "s_scale", np.sqrt(0.5) * 0.37)):
        s = float(held[scale][0])
        z = O.decode(held[name].view(torch.uint8).cpu().numpy())[keep]
        y = np.float64(np.float32(x)) / s
        lo, hi = O.store(np.array([y, y]), np.array([0.0, 65535.0]), False)
        assert set(np.unique(z)) == {lo, hi}
        share = (y - lo) / (hi - lo)
        # fp32 places y within 8 U of itself, the hash resolves 2^-16 of a code
        slack = 8 * O.U * y + (hi - lo) * 2.0 ** -16
        assert abs(z.mean() - y) <= 6 * (hi - lo) * np.sqrt(share * (1 - share) / keep.sum()) + slack


def test_small_roots_are_never_zero():
    n = 512
    opt = A.AdamW([A.tensor(n, state_bits=8)])
    g = torch.zeros(n, device="cuda")
    g[0], g[1:256] = 1e3, 1e-9
    p = torch.zeros(n, device="cuda")
    opt.bind([p], [g])
    for _ in range(3):
        opt.step(1e-3)
    s = opt.state_tensors()["s8"].view(torch.uint8)
    assert bool((s[:256] > 0).all()) and not bool(s[256:].any())
    assert bool(torch.isfinite(p).all()) and float(p[1:].abs().max()) <= 3 * 1e-3


def test_repeats_bit_for_bit_and_by_tensor_alignment():
    """The same step twice, from buffers of another alignment, gives the same
    bits."""
    specs = [A.tensor(n, param="bf16", state_bits=8) for n in (100, 5000, 70000)]
    got = []
    for offset in (0, 0, 3):
        run = Run(specs, 8, offset=offset)
        for _ in range(3):
            run.opt.step(1e-3)
        got.append(run.read())
    for other in got[1:]:
        for a, b in zip(got[0], other):
            for k in ("p", "rem", "m8", "s8", "m_scale", "s_scale"):
                assert np.array_equal(a[k], b[k]), k


def test_learning_rate_on_the_device():
    run = Run([A.tensor(1000, state_bits=b) for b in (32, 8)], 2)
    lr = torch.tensor([1e-3], device="cuda")
    for x in (1e-3, 5e-4):
        lr.fill_(x)
        before = run.read()
        run.opt.step(lr)
        run.check(before, float(np.float32(x)))


def test_captured_and_replayed():
    """Norm and step in a graph: every replay is the eager step, with eager work
    of the same handle, new gradients, another learning rate, and a gradient
    that is not finite between replays."""
    sizes = (700, 5000, 40000)
    make = lambda: Run([A.tensor(n, param="bf16", grad="bf16", state_bits=b, weight_decay=0.1)
                        for n in sizes for b in (32, 8)], 13)
    eager, graph = make(), make()
    norms = [A.GradNorm([(s.numel, "bf16") for s in r.specs]) for r in (eager, graph)]
    lrs = [torch.tensor([1e-3], device="cuda") for _ in range(2)]

    def go(k):
        (eager, graph)[k].opt.bind((eager, graph)[k].params, (eager, graph)[k].grads)
        norms[k].bind((eager, graph)[k].grads)
        norms[k].compute(1.0)
        (eager, graph)[k].opt.step(lrs[k], clip=norms[k])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(1)
    go(0)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(1)
    for k in range(6):
        for i in range(len(eager.specs)):
            x = torch.from_numpy(eager.draw(i)).to(torch.bfloat16).cuda()
            if k == 3 and i == 2:
                x[17] = float("nan")
            eager.grads[i].copy_(x)
            graph.grads[i].copy_(x)
        for lr in lrs:
            lr.fill_(1e-3 / (k + 1))
        go(0)
        g.replay()
        if k == 2:
            torch.cuda.synchronize()
            go(0)
            go(1)
        torch.cuda.synchronize()
        assert int(eager.opt.t) == int(graph.opt.t)
        assert torch.equal(norms[0].record, norms[1].record) or k == 3
        for a, b in zip(eager.read(), graph.read()):
            for key in a:
                assert np.array_equal(a[key], b[key], equal_nan=True), (k, key)


def test_two_graphs_of_the_same_handles():
    """One graph with the clip and one without, in turn, against eager steps."""
    sizes = (700, 40000)
    make = lambda: Run([A.tensor(n, state_bits=b, weight_decay=0.1) for n in sizes for b in (32, 8)], 19)
    eager, run = make(), make()
    norms = [A.GradNorm([(s.numel, "f32") for s in r.specs]) for r in (eager, run)]
    for n, r in zip(norms, (eager, run)):
        n.bind(r.grads)

    def go(k, clip):
        r = (eager, run)[k]
        if clip:
            norms[k].compute(0.5)
        r.opt.step(1e-3, clip=norms[k] if clip else None)

    for k in (0, 1):
        go(k, True)
    graphs = []
    for clip in (True, False):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(1, clip)
        graphs.append(g)
    for k in (0, 1, 1, 0, 1, 0):
        for i in range(len(eager.specs)):
            x = torch.from_numpy(eager.draw(i)).cuda()
            eager.grads[i].copy_(x)
            run.grads[i].copy_(x)
        go(0, k == 0)
        graphs[k].replay()
    torch.cuda.synchronize()
    for a, b in zip(eager.read(), run.read()):
        for key in a:
            assert np.array_equal(a[key], b[key]), key


def test_gradients_of_new_addresses_every_step():
    """Gradients that are allocated anew, bound and freed at every step."""
    specs = [A.tensor(n, param="bf16", state_bits=b) for n in (5, 3000, 90001) for b in (32, 8)]
    a, b = Run(specs, 6), Run(specs, 6)
    for _ in range(4):
        new = [torch.from_numpy(a.draw(i)).to("cuda", torch.bfloat16) for i in range(len(specs))]
        for g, x in zip(b.grads, new):
            g.copy_(x)
        a.opt.bind(grads=new)
        a.opt.step(1e-3)
        del new, x
        b.opt.step(1e-3)
    for x, y in zip(a.read(), b.read()):
        for k in x:
            if k != "g":
                assert np.array_equal(x[k], y[k]), k


def test_another_stream():
    a, b = Run([A.tensor(50000, state_bits=8)], 1), Run([A.tensor(50000, state_bits=8)], 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            a.opt.step(1e-3)
    for _ in range(3):
        b.opt.step(1e-3)
    torch.cuda.synchronize()
    assert np.array_equal(a.read()[0]["p"], b.read()[0]["p"])


def test_more_than_2_to_32_elements():
    """Offsets and the hash past 32 bits: head, middle and tail of one tensor."""
    n = (1 << 32) + 700
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    opt = A.AdamW([A.tensor(n, param="bf16", state_bits=8)], A.make_config(seed=5))
    rng = np.random.default_rng(0)
    spots = [0, 1 << 31, (1 << 32) - 256, 1 << 32, n - 700 % 256]
    for s in spots:
        k = min(256, n - s)
        g[s:s + k] = torch.from_numpy(rng.standard_normal(k)).to("cuda", torch.bfloat16)
    opt.bind([p], [g])
    opt.step(1e-3)
    held = opt.state_tensors()
    assert int(torch.count_nonzero(p)) == sum(min(256, n - s) for s in spots)
    for s in spots:
        k = min(256, n - s)
        gg = np64(g[s:s + k])
        m, root = 0.1 * gg, np.sqrt(0.001) * np.abs(gg)
        rm, rs = O.random_bits(5, 1, 0, s + np.arange(k))
        for x, code, r, pos in ((m, "m8", rm, False), (root, "s8", rs, True)):
            lo, hi = O.store_range(x, 8 * O.U * np.abs(x), O.run_scales(x), r, pos)
            z = np.abs(O.decode(held[code].view(torch.uint8)[s:s + k].cpu().numpy()))
            assert np.all((z >= lo) & (z <= hi)), (s, code)
    del p, g, opt, held
    torch.cuda.empty_cache()


# ------------------------------------------------------------ gradient norm
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("scale,grad_scale", [(1e-3, 1.0), (1.0, 0.5), (1e3, 2.0 ** -10)])
def test_norm(offset, scale, grad_scale):
    rng = np.random.default_rng(7)
    kinds = ("f32", "bf16", "f16")
    sizes = SIZES + [2048, 2049, 123457]
    grads, bufs, want = [], [], []
    for i, n in enumerate(sizes):
        t, b = guarded((scale * rng.standard_normal(n)).astype(np.float32), TORCH[kinds[i % 3]], offset)
        grads.append(t)
        bufs.append((b, n))
        want.append(np64(t))
    outs, obufs = [], []
    for n in sizes:
        t, b = guarded(np.zeros(n, np.float32), torch.float32, 3 - offset)
        outs.append(t)
        obufs.append((b, n))
    norm = A.GradNorm([(n, kinds[i % 3]) for i, n in enumerate(sizes)])
    norm.bind(grads, outs)
    n64, c64 = O.norm(want, 1.0, grad_scale)
    norm.compute(1.0, grad_scale)
    norm.clip_into()
    got = np64(norm.record)
    # fp64 sums: 2^-53 a term at most, then one rounding to fp32
    assert abs(got[0] - n64) <= 2 * O.U * n64 and abs(got[1] - c64) <= 2 * O.U * c64
    for o, w in zip(outs, want):
        assert np.all(np.abs(np64(o) - c64 * w) <= 4 * O.U * np.abs(c64 * w) + O.TINY)
    for b, n in bufs:
        untouched(b, offset, n)
    for b, n in obufs:
        untouched(b, 3 - offset, n)
    first = norm.record.clone()
    norm.compute(1.0, grad_scale)
    assert torch.equal(first, norm.record)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_norm_past_the_caches(kind):
    """More gradients than the caches hold; one value in each of a few places."""
    n = (204 << 20) // (4 if kind == "f32" else 2) + 77
    g = torch.zeros(n + 3, dtype=TORCH[kind], device="cuda")[3:]
    for i, k in enumerate((0, 1023, 1024, n // 2, n - 78, n - 1)):
        g[k] = 2.0 ** i
    small = torch.full((5,), 0.5, dtype=TORCH[kind], device="cuda")
    norm = A.GradNorm([(5, kind), (n, kind)])
    norm.bind([small, g])
    for _ in range(3):
        norm.compute(1.0)
        want = np.sqrt(5 * 0.25 + sum(4.0 ** i for i in range(6)))
        assert abs(float(norm.record[0]) - want) <= 2 * O.U * want
        assert abs(float(norm.record[1]) - 1 / want) <= 2 * O.U / want


def test_norm_clips_in_place_and_leaves_absent_ones():
    rng = np.random.default_rng(3)
    a, b, c = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() for n in (5000, 300, 40))
    keep = [x.clone() for x in (a, b, c)]
    norm = A.GradNorm([(5000, "f32"), (300, "f32"), (40, "f32"), (9, "bf16")])
    norm.bind([a, b, c, None], [a, None, c, None])
    norm.compute(1.0)
    n64, c64 = O.norm([np64(x) for x in keep], 1.0)
    norm.clip_into()
    assert abs(float(norm.record[0]) - n64) <= 2 * O.U * n64
    assert np.allclose(np64(a), c64 * np64(keep[0]), rtol=4 * O.U, atol=0)
    assert torch.equal(b, keep[1])
    assert np.allclose(np64(c), c64 * np64(keep[2]), rtol=4 * O.U, atol=0)
    now = a.clone()
    norm.compute(float("inf"))         # nothing to clip
    norm.clip_into()
    assert torch.equal(a, now) and float(norm.record[1]) == 1.0


def test_norm_edges():
    norm = A.GradNorm([(4, "f32"), (0, "bf16")])
    out = torch.full((4,), 5.0, device="cuda")
    g = torch.zeros(4, device="cuda")
    norm.bind([g, None], [out, None])
    def go(values, max_norm=1.0):
        g.copy_(torch.tensor(values))
        norm.compute(max_norm)
        norm.clip_into()
        torch.cuda.synchronize()
        return float(norm.record[0]), float(norm.record[1]), int(norm.nonfinite)
    assert go([0.0] * 4) == (0.0, 1.0, 0) and not bool(out.any())
    n, c, bad = go([3e38, 3e38, 0.0, 0.0])       # squares past fp32, the norm past it too
    # the coefficient 2.4e-39 is a denormal: it is rounded by up to 2^-150
    true = 1 / np.hypot(np.float64(np.float32(3e38)), np.float64(np.float32(3e38)))
    assert n == float("inf") and bad == 0 and abs(c - true) <= O.TINY / 2
    n, c, bad = go([1e-30, 0, 0, 0])             # a square below fp32
    assert abs(n / 1e-30 - 1) < 4 * O.U and (c, bad) == (1.0, 0)
    for x in (float("inf"), float("-inf"), float("nan")):
        n, c, bad = go([1.0, x, 2.0, 3.0])
        assert (c, bad) == (0.0, 1) and not bool(out.any())
    assert go([1.0, 0.0, 0.0, 0.0])[1:] == (1.0, 0) and float(out[0]) == 1.0
    empty = A.GradNorm([(0, "f32")])
    empty.bind([torch.empty(0, device="cuda")])
    empty.compute(1.0)
    assert empty.record.tolist() == [0.0, 1.0]


def test_refusals():
    opt = A.AdamW([A.tensor(8), A.tensor(4, param="bf16")])
    p = [torch.zeros(8, device="cuda"), torch.zeros(4, device="cuda", dtype=torch.bfloat16)]
    with pytest.raises(S.ShampooError):
        opt.step(1e-3)                                    # nothing bound
    opt.bind(p, p)
    for bad in ([p[0]], [p[0], None], [p[0], p[0][:4]], [p[0][::2], p[1]], [p[0].cpu(), p[1]],
                [torch.zeros(16, device="cuda")[::2], p[1]]):
        with pytest.raises(ValueError):
            opt.bind(bad)
    with pytest.raises(S.ShampooError):
        opt.bind()
    twice = A.AdamW([A.tensor(8), A.tensor(4), A.tensor(0)])
    nothing = torch.empty(0, device="cuda")
    for bad in ([p[0], p[0][:4], nothing], [p[0], p[0][4:], nothing]):
        with pytest.raises(S.ShampooError):
            twice.bind(bad)                               # a weight that is listed twice
    twice.bind([p[0], torch.zeros(4, device="cuda"), nothing])
    with pytest.raises(ValueError):
        opt.step(torch.tensor([1e-3]))
    with pytest.raises(ValueError):
        opt.step(torch.tensor([1e-3], device="cuda", dtype=torch.float64))
    with pytest.raises(S.ShampooError):
        opt.step(float("nan"))
    with pytest.raises(S.ShampooError):
        opt.set_step(-1)
    norm = A.GradNorm([(4, "bf16")])
    with pytest.raises(S.ShampooError):
        norm.compute(1.0)
    with pytest.raises(ValueError):
        norm.bind([p[0][:4]])
    with pytest.raises(ValueError):
        norm.bind([p[1]], [p[1]])                         # outputs are fp32
    norm.bind([p[1]])
    with pytest.raises(S.ShampooError):
        norm.compute(0.0)
    with pytest.raises(ValueError):
        opt.step(1e-3, clip=norm)                         # no norm computed yet
    norm.compute(1.0)
    with pytest.raises(S.ShampooError):
        norm.clip_into()                                  # no outputs bound
    norm.bind([p[1]], [torch.empty(4, device="cuda")])
    norm.clip_into()
    two = A.GradNorm([(4, "f32"), (4, "f32")])
    x = torch.zeros(16, device="cuda")
    two.bind([x[:4], x[4:8]], [x[:4], x[8:12]])
    for outs in ([x[4:8], None], [x[2:6], None], [x[8:12], x[10:14]], [x[:4], x[3:7]]):
        with pytest.raises(S.ShampooError):
            two.bind([x[:4], x[4:8]], outs)
    with pytest.raises(ValueError):
        A.AdamW([A.tensor(4)], device="cpu")


def test_empty_tensors_count_steps():
    """A plan whose tensors are all empty counts its steps like any other, and
    skips those whose norm is not finite."""
    nothing = torch.empty(0, device="cuda")
    opt = A.AdamW([A.tensor(0), A.tensor(0, state_bits=8)])
    opt.bind([nothing, None], [nothing, None])
    g = torch.ones(4, device="cuda")
    norm = A.GradNorm([(4, "f32")])
    norm.bind([g])
    for t, x in ((1, 1.0), (2, 1.0), (2, float("nan")), (3, 1.0)):
        g[0] = x
        norm.compute(1.0)
        opt.step(1e-3, clip=norm)
        assert int(opt.t) == t
    opt.set_step(7)
    opt.step(1e-3)
    assert int(opt.t) == 8
    # an address that is given for nothing is not read
    at = (S._P * 2)(g.data_ptr(), g.data_ptr())
    assert S.lib().shampoo_adamw_bind_tensors(opt.h, at, at, None) == 0
    opt.step(1e-3)
    assert int(opt.t) == 9 and g[1:].tolist() == [1.0, 1.0, 1.0]


def test_refused_state_changes_nothing():
    run = Run([A.tensor(n, param="bf16", state_bits=b) for n in (300, 1000) for b in (32, 8)], 3, t0=5)
    before = {k: x.view(torch.uint8).clone() for k, x in run.opt.state_tensors().items()}
    saved = {k: x.zero_() if k != "t" else -1 for k, x in run.opt.state_dict().items()}
    with pytest.raises(ValueError):
        run.opt.load_state_dict(saved)
    assert int(run.opt.t) == 5
    for k, x in run.opt.state_tensors().items():
        assert torch.equal(x.view(torch.uint8), before[k]), k


def test_a_norm_that_has_not_run_skips_the_step():
    """Between the capture of a norm and the first replay its record holds no
    coefficient: steps that read it change nothing, clipped gradients are 0."""
    run = Run([A.tensor(n, state_bits=b, weight_decay=0.1) for n in (300, 1000) for b in (32, 8)], 3, t0=5)
    out = [torch.full_like(g, 7.0) for g in run.grads]
    norm = A.GradNorm([(s.numel, "f32") for s in run.specs])
    norm.bind(run.grads, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm.compute(1.0)
    before = run.read()
    run.opt.step(1e-3, clip=norm)
    norm.clip_into()
    assert int(run.opt.t) == 5 and not any(bool(o.any()) for o in out)
    for a, b in zip(before, run.read()):
        for k in a:
            assert np.array_equal(a[k], b[k]), k
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        before = run.read()
        run.opt.step(1e-3, clip=norm)
        run.check(before, 1e-3, float(norm.record[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_first_gradient_after_a_thousand_steps(bits):
    """From zero moments: the first update is lr where the tensor's own steps
    are counted, and 2.5 lr where the handle's are."""
    n, lr = 1000, 1e-3
    g = np.random.default_rng(3).standard_normal(n).astype(np.float32)
    for own, t in ((True, 1), (False, 1001)):
        p = torch.zeros(n, device="cuda")
        opt = A.AdamW([A.tensor(n, state_bits=bits)], per_tensor_steps=own)
        opt.set_step(1000)
        if own:
            opt.set_tensor_steps([0])
        opt.bind([p], [torch.from_numpy(g).cuda()])
        opt.step(lr)
        zero = np.zeros(n)
        want, _, _, _, err = O.step(zero, g.astype(np.float64), zero, zero, t, O.Hyper(lr=lr))[:5]
        assert np.all(np.abs(np64(p) - want) <= err)
        # |g| / (|g| + eps) is 1 to 1e-8 / |g|; 0.1 / sqrt(0.001 / (1 - 0.999^1001)) = 2.515
        size = np.abs(np64(p))[np.abs(g) > 0.1] / lr
        assert np.allclose(size, 1.0 if own else 2.515, rtol=1e-3)
        assert int(opt.t) == 1001 and opt.tensor_steps() == [t]


def test_tensors_count_their_own_steps():
    """Gradients that come now and then: each tensor is corrected as by a handle
    of its own that only steps when there is one, eager and replayed, with steps
    whose norm is not finite between; a saved state goes on alike."""
    kinds = [(n, p, b) for n in (700, 5000) for p in ("f32", "bf16") for b in (32, 8)] + [(0, "f32", 32)]
    specs = [A.tensor(n, param=p, grad="f32", state_bits=b, weight_decay=0.1) for n, p, b in kinds]
    rng = np.random.default_rng(8)
    start = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().to(TORCH[p]) for n, p, _ in kinds]
    grads = [torch.zeros(n, device="cuda") for n, _, _ in kinds]
    every = A.AdamW(specs, per_tensor_steps=True)
    weights = [w.clone() for w in start]
    every.bind(weights, grads)
    single, alone = [A.AdamW([s]) for s in specs], [w.clone() for w in start]
    for o, w, g in zip(single, alone, grads):
        o.bind([w], [g])
    norm = A.GradNorm([(n, "f32") for n, _, _ in kinds])
    norm.bind(grads)
    counts, t = [0] * len(kinds), 0
    graph = None
    for k in range(14):
        if k == 4:      # the state goes on in another handle
            saved, old = every.state_dict(), every
            every = A.AdamW(specs, per_tensor_steps=True)
            every.load_state_dict(saved)
            every.bind(weights, grads)
            assert every.tensor_steps() == old.tensor_steps() == counts
        present = [(k + i) % 3 != 0 or k >= 10 for i in range(len(kinds))]
        bad = k in (2, 12)
        for i, g in enumerate(grads):
            g.normal_(0, 1e-2)
        if bad:
            grads[1][3] = float("inf")
        norm.compute()
        if k < 10:
            every.bind(grads=[g if here else None for g, here in zip(grads, present)])
            every.step(1e-3, clip=norm)
        else:
            if graph is None:
                every.bind(grads=grads)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    every.step(1e-3, clip=norm)
            graph.replay()
        t += not bad
        for i, here in enumerate(present):
            if here:
                single[i].step(1e-3, clip=norm)
                counts[i] += not bad and kinds[i][0] > 0
        torch.cuda.synchronize()
        assert int(every.t) == t and every.tensor_steps() == counts
        for i, (n, _, b) in enumerate(kinds):
            # the rounding of 8-bit moments goes by the handle's step: equal until it has been read
            if b == 32 or counts[i] <= 1:
                assert torch.equal(weights[i], alone[i]), (k, i)
    with pytest.raises(ValueError):
        A.AdamW(specs).load_state_dict(every.state_dict())
    with pytest.raises(ValueError):
        every.load_state_dict(A.AdamW(specs).state_dict())
    with pytest.raises(ValueError):
        every.set_tensor_steps([1])
    with pytest.raises(S.ShampooError):
        every.set_tensor_steps([-1] + counts[1:])
    with pytest.raises(S.ShampooError):
        single[0].set_tensor_steps([1])
    assert every.tensor_steps() == counts
    assert S.lib().shampoo_adamw_set_counting(every.h, 0) == -2       # its state is bound


def test_captured_clip():
    """Norm and clipped copies in a graph, one of them in place: every replay is
    the eager result, with a gradient that is not finite among them."""
    kinds = [(700, "f32"), (40000, "bf16"), (5000, "f16"), (300, "f32")]
    rng = np.random.default_rng(5)
    sets = []
    for _ in range(2):
        grads = [torch.zeros(n, dtype=TORCH[k], device="cuda") for n, k in kinds]
        outs = [grads[0]] + [torch.zeros(n, device="cuda") for n, _ in kinds[1:]]
        norm = A.GradNorm(kinds)
        norm.bind(grads, outs)
        sets.append((grads, outs, norm))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sets[1][2].compute(1.0)
        sets[1][2].clip_into()
    for k in range(5):
        for i, (n, kind) in enumerate(kinds):
            x = torch.from_numpy(rng.standard_normal(n)).cuda().to(TORCH[kind])
            if k == 2 and i == 1:
                x[5] = float("inf")
            for grads, _, _ in sets:
                grads[i].copy_(x)
        sets[0][2].compute(1.0)
        sets[0][2].clip_into()
        graph.replay()
        torch.cuda.synchronize()
        assert int(sets[1][2].nonfinite) == (k == 2)
        for a, b in zip(sets[0][1] + [sets[0][2].record], sets[1][1] + [sets[1][2].record]):
            assert torch.equal(a, b), k


# ------------------------------------------------- roots and quotients, counted
RUN_PAIR = 512          # elements of a wave: the two runs that take one path together


class Still:
    """A step that changes no moments: betas of 1 in fp32, corrections of 1 (no
    decay, zero gradients), so that p = -m / (sqrt(v) + 2^-100)."""

    def __init__(self, n):
        self.p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        almost = 1 - 2.0 ** -53
        self.opt = A.AdamW([A.tensor(n)], A.make_config(beta1=almost, beta2=almost, eps=2.0 ** -100))
        self.opt.set_step(1 << 62)
        self.opt.bind([self.p], [g])
        held = self.opt.state_tensors()
        self.m, self.v = held["m"], held["v"]

    def quotients(self):
        self.p.zero_()
        self.opt.step(1.0)
        return -self.p


def plain_quotients(m, v):
    zero = np.float32(0)
    with np.errstate(all="ignore"):
        return -(zero - (zero + m / (np.sqrt(v) + np.float32(2.0 ** -100))))


def short_waves(m, root, v, c, eps):
    """Which waves' elements are all in the range of the corrected estimates."""
    with np.errstate(all="ignore"):
        d = root.astype(np.float64) * c + eps
        a = np.abs(m.astype(np.float64))
        ok = np.isfinite(v) & (v >= 2.0 ** -96) & (a < 2.0 ** 79) & ((a == 0) | (a >= np.maximum(2.0 ** -100, d * 2.0 ** -124)))
    return ok.reshape(-1, RUN_PAIR).all(1)


def signed(rng, x):
    return (x * rng.choice([-1.0, 1.0], x.shape)).astype(np.float32)


def test_every_root_and_divisor():
    """Every significand at every exponent from 2^-96 on as a second moment,
    each under an m of its own: root and quotient are the rounded ones.  (The
    roots of [1, 4) take every significand of a divisor.)"""
    n = 1 << 24
    s = Still(n)
    rng = np.random.default_rng(0)
    significand = torch.arange(n, dtype=torch.int32, device="cuda")
    m = signed(rng, rng.uniform(1, 2, n))
    m[rng.random(n) < 0.05] = 0.0
    s.m.copy_(torch.from_numpy(m))
    for e in range(-96, 128, 2):
        s.v.copy_((significand + ((e + 127) << 23)).view(torch.float32))
        got = s.quotients()
        # fp64 has more than twice the bits, so that rounding twice is rounding once
        want = (s.m.double() / s.v.double().sqrt().float().double()).float()
        bad = torch.nonzero(got != want).flatten().cpu().numpy()
        if bad.size:
            v = s.v.cpu().numpy()[bad]
            assert np.array_equal(got.cpu().numpy()[bad], plain_quotients(m[bad], v)), (e, bad.size)


@pytest.mark.parametrize("m_range,v_range", [
    ((-149, -100), (-40, 0)),       # what a few hundred zero gradients leave of m
    ((-110, -90), (-96, -80)), ((-110, -60), (60, 128)), ((-30, 60), (-96, -60)), ((60, 127.9), (-96, -40)),
    ((60, 127.9), (60, 128)), ((-149, 127.9), (-149, 128))])
@pytest.mark.parametrize("mixed", [False, True])
def test_quotients_over_the_range(m_range, v_range, mixed):
    """Small and large quotients bit for bit, in waves of their own and among
    elements of an everyday size."""
    n = 64 * RUN_PAIR
    rng = np.random.default_rng(1)
    m = signed(rng, 2.0 ** rng.uniform(*m_range, n))
    v = np.minimum(2.0 ** rng.uniform(*v_range, n), 3.4e38).astype(np.float32)
    if mixed:
        usual = rng.random(n) < 0.9
        m[usual] = signed(rng, rng.uniform(1e-4, 1e-3, usual.sum()))
        v[usual] = rng.uniform(1e-8, 1e-6, usual.sum())
    s = Still(n)
    s.m.copy_(torch.from_numpy(m))
    s.v.copy_(torch.from_numpy(v))
    got, want = s.quotients().cpu().numpy(), plain_quotients(m, v)
    assert np.array_equal(got.view(np.uint32), want.view(np.uint32)), np.flatnonzero(got != want)[:5]


def test_an_element_does_not_depend_on_its_neighbours():
    """The same tiny m beside an everyday element and beside a second moment of
    zero."""
    n = 4 * RUN_PAIR
    rng = np.random.default_rng(2)
    m = signed(rng, 2.0 ** rng.uniform(-126, -118, n))
    v = rng.uniform(1e-8, 1e-6, n).astype(np.float32)
    got = []
    for beside in (1e-7, 0.0):
        v[::RUN_PAIR], m[::RUN_PAIR] = beside, 0.0
        s = Still(n)
        s.m.copy_(torch.from_numpy(m))
        s.v.copy_(torch.from_numpy(v))
        got.append(s.quotients().cpu().numpy())
    keep = np.arange(n) % RUN_PAIR != 0
    assert np.array_equal(got[0][keep].view(np.uint32), got[1][keep].view(np.uint32))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lo,hi", [(-8, 0), (-40, -20), (40, 63)])
def test_every_rounding_of_short_waves(lo, hi, bits):
    """Steps of waves whose elements all take the corrected estimates and, with
    8-bit moments, the hardware's conversion: bit for bit the fp32 formula.
    Signs stay and a wave's gradients are within a factor of 8, so that no value
    falls below 2^-6 of e4m3's range (448 / 2^-6 is 2^14.8)."""
    waves = 64
    n = waves * RUN_PAIR
    rng = np.random.default_rng(64 + hi)
    size = np.repeat(2.0 ** rng.uniform(lo, hi - 1, waves), RUN_PAIR)
    sign = rng.choice([-1.0, 1.0], n)
    eps = 2.0 ** -60
    h = O.Hyper(lr=1e-3, weight_decay=0.1, eps=eps)
    opt = A.AdamW([A.tensor(n, state_bits=bits, weight_decay=0.1)], A.make_config(eps=eps, seed=9))
    w = rng.standard_normal(n).astype(np.float32)
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    p, g = torch.from_numpy(w.copy()).cuda(), torch.zeros(n, device="cuda")
    opt.bind([p], [g])
    held = opt.state_tensors()
    same = lambda a, b: np.array_equal(np.asarray(a).view(np.uint32), np.asarray(b).view(np.uint32))
    for t in (1, 2, 3):
        x = (sign * size * rng.uniform(0.25, 2, n)).astype(np.float32)
        g.copy_(torch.from_numpy(x))
        opt.step(h.lr)
        w, m, root, v = O.step32(w, x, m, v, t, h)
        assert short_waves(m, root, v, 1 / np.sqrt(1 - h.beta2 ** t), eps).all()
        assert same(p.cpu().numpy(), w), t
        if bits == 32:
            assert same(held["m"].cpu().numpy(), m) and same(held["v"].cpu().numpy(), v)
            continue
        rm, rs = O.random_bits(9, t, 0, np.arange(n))
        for value, r, code, scale, pos in ((m, rm, "m8", "m_scale", False), (root, rs, "s8", "s_scale", True)):
            c, s = O.codes32(value, r, pos)
            assert np.all(np.abs(value).reshape(-1, 256) > 1.001 * 2.0 ** -6 * s[:, None])
            assert same(held[scale].cpu().numpy(), s), (t, scale)
            assert np.array_equal(held[code].view(torch.uint8).cpu().numpy(), c), (t, code)
        spread = lambda k: np.repeat(held[k].cpu().numpy(), 256)
        dec = lambda k: O.decode(held[k].view(torch.uint8).cpu().numpy()).astype(np.float32)
        m = dec("m8") * spread("m_scale")
        root = dec("s8") * spread("s_scale")
        v = root * root


# ------------------------------------------------------------ as they are used
def test_shampoo_and_adamw_under_one_norm():
    """A model's end of step: bf16 gradients under one norm, matrices on Shampoo
    with the clipped fp32 gradients, the vectors on AdamW with the coefficient."""
    rng = np.random.default_rng(17)
    mats = [(256, 384), (128, 512)]
    vecs = [384, 512, 1000]
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to("cuda", torch.bfloat16)
    cfg = S.make_config(128, root_mode="auto")
    shapes = [(r, c, S.DENSE) for r, c in mats]
    ours, ref = S.Shampoo(shapes, cfg), S.Shampoo(shapes, cfg)
    W = [torch.zeros(r, c, device="cuda") for r, c in mats]
    W2 = [w.clone() for w in W]
    run = Run([A.tensor(n, param="bf16", state_bits=8 if n == 1000 else 32) for n in vecs], 3, warm=False)
    clipped = [torch.empty(r, c, device="cuda") for r, c in mats]
    norm = A.GradNorm([(r * c, "bf16") for r, c in mats] + [(n, "bf16") for n in vecs])
    for t in range(4):
        G = [mk(r, c) for r, c in mats]
        for i, n in enumerate(vecs):
            run.grads[i].copy_(mk(n))
        before = run.read()
        norm.bind(G + run.grads, clipped + [None] * len(vecs))
        norm.compute(1.0)
        norm.clip_into()
        ours.step(W, clipped, t, 2)
        run.opt.step(1e-3, clip=norm)
        coef = norm.record[1]
        n64, c64 = O.norm([np64(g).ravel() for g in G + run.grads], 1.0)
        assert abs(float(coef) - c64) <= 2 * O.U * c64
        ref.step(W2, [g.float() * coef for g in G], t, 2)
        for a, b in zip(W, W2):
            assert torch.equal(a, b)
        run.check(before, 1e-3, float(coef))
