"""First-order operators without a GPU: struct layouts, refusals, plans, and the
oracle's own pieces (codes, rounding, hash) against brute force."""
import ctypes

import numpy as np
import pytest

from oracle import adamw_oracle as O
from second_order_optimizer_amd import adamw as A
from second_order_optimizer_amd import shampoo as S

E_ARG, E_STATE, E_UNSUPPORTED = -1, -2, -5


def create(specs, cfg=None):
    h = S._P()
    descs = (S.AdamWTensor * max(len(specs), 1))(*specs)
    rc = S.lib().shampoo_adamw_create(ctypes.byref(cfg or A.make_config()), len(specs), descs,
                                      ctypes.byref(h))
    return rc, h


def create_norm(descs):
    h = S._P()
    arr = (S.GradDesc * max(len(descs), 1))(*descs)
    return S.lib().shampoo_gradnorm_create(len(descs), arr, ctypes.byref(h)), h


def test_struct_sizes():
    assert ctypes.sizeof(S.GradDesc) == 16
    assert ctypes.sizeof(S.AdamWConfig) == 32
    assert ctypes.sizeof(S.AdamWTensor) == 40
    assert ctypes.sizeof(S.AdamWLayout) == 96


@pytest.mark.parametrize("field,value,rc", [
    ("numel", -1, E_ARG), ("numel", (1 << 38) + 1, E_UNSUPPORTED), ("param_type", 3, E_ARG),
    ("param_type", -1, E_ARG), ("param_type", 2, E_UNSUPPORTED), ("grad_type", 3, E_ARG),
    ("state_bits", 16, E_ARG), ("reserved", 1, E_ARG), ("weight_decay", -0.1, E_ARG),
    ("weight_decay", float("nan"), E_ARG), ("lr_scale", -1.0, E_ARG),
    ("lr_scale", float("inf"), E_ARG)])
def test_adamw_create_refuses_tensor(field, value, rc):
    d = A.tensor(10)
    setattr(d, field, value)
    assert create([A.tensor(4), d])[0] == rc


@pytest.mark.parametrize("field,value", [
    ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0), ("beta2", float("nan")), ("eps", 0.0),
    ("eps", -1e-8), ("eps", float("inf")), ("eps", float("nan")), ("eps", 1e-60), ("eps", 7e-31), ("eps", 1e31), ("reserved", 1)])
def test_adamw_create_refuses_config(field, value):
    c = A.make_config()
    setattr(c, field, value)
    assert create([A.tensor(10)], c)[0] == E_ARG


def test_plans_past_a_launch():
    assert create([A.tensor(1 << 34), A.tensor(1 << 34), A.tensor(1)])[0] == E_UNSUPPORTED
    assert create_norm([S.GradDesc(1 << 36, 0, 0), S.GradDesc(1, 0, 0)])[0] == E_UNSUPPORTED


def test_nulls_and_unbound_handles():
    L = S.lib()
    assert create([])[0] == E_ARG
    assert L.shampoo_adamw_create(None, 1, (S.AdamWTensor * 1)(A.tensor(1)), ctypes.byref(S._P())) == E_ARG
    rc, h = create([A.tensor(10)])
    assert rc == 0
    ptrs = (S._P * 1)(256)
    assert L.shampoo_adamw_step(h, 1e-3, None, None, None) == E_STATE
    assert L.shampoo_adamw_step(None, 1e-3, None, None, None) == E_ARG
    assert L.shampoo_adamw_step(h, float("nan"), None, None, None) == E_ARG
    assert L.shampoo_adamw_step(h, 1e-3, 2, None, None) == E_ARG
    assert L.shampoo_adamw_step(h, 1e-3, None, 8, None) == E_ARG
    assert L.shampoo_adamw_bind_tensors(h, ptrs, ptrs, None) == E_STATE
    assert L.shampoo_adamw_bind_tensors(h, None, None, None) == E_ARG
    assert L.shampoo_adamw_set_step(h, 3, None) == E_STATE
    assert L.shampoo_adamw_set_step(h, -1, None) == E_ARG
    assert L.shampoo_adamw_bind_state(h, None, 0, None) == E_ARG
    assert L.shampoo_adamw_bind_state(h, 128, 1 << 20, None) == E_ARG
    assert L.shampoo_adamw_bind_state(h, 256, 16, None) == E_STATE
    assert L.shampoo_adamw_get_layout(h, None) == E_ARG
    assert L.shampoo_adamw_tensor_runs(h, 1, None, None) == E_ARG
    L.shampoo_adamw_destroy(h)

    assert create_norm([])[0] == E_ARG
    for d, rc in ((S.GradDesc(-1, 0, 0), E_ARG), (S.GradDesc(1, 3, 0), E_ARG),
                  (S.GradDesc(1, 0, 1), E_ARG), (S.GradDesc((1 << 38) + 1, 0, 0), E_UNSUPPORTED)):
        assert create_norm([S.GradDesc(4, 0, 0), d])[0] == rc
    rc, h = create_norm([S.GradDesc(10, 0, 0)])
    assert rc == 0
    assert L.shampoo_gradnorm_compute(h, 1.0, 1.0, None) == E_STATE
    for max_norm, scale in ((0.0, 1.0), (-1.0, 1.0), (float("nan"), 1.0), (1.0, 0.0), (1.0, -1.0),
                            (1.0, float("inf")), (1.0, float("nan"))):
        assert L.shampoo_gradnorm_compute(h, max_norm, scale, None) == E_ARG
    assert L.shampoo_gradnorm_clip_into(h, None) == E_STATE
    assert L.shampoo_gradnorm_bind_grads(h, ptrs, None, None) == E_STATE
    assert L.shampoo_gradnorm_bind_grads(h, None, None, None) == E_ARG
    assert L.shampoo_gradnorm_bind_state(h, 128, 1 << 20, None) == E_ARG
    assert L.shampoo_gradnorm_bind_state(h, 256, 16, None) == E_STATE
    assert L.shampoo_gradnorm_record(h, ctypes.byref(S._P())) == E_STATE
    L.shampoo_gradnorm_destroy(h)


def test_python_refusals_before_any_device():
    with pytest.raises(ValueError):
        A.make_config(seed=1 << 32)
    with pytest.raises(KeyError):
        A.tensor(4, param="fp8")
    with pytest.raises(S.ShampooError):
        A.AdamW([A.tensor(4, state_bits=16)])


@pytest.mark.parametrize("sizes", [[0], [1], [256], [257, 0, 1], [1000, 31, 5_000_000], [3] * 450])
def test_plan_layout(sizes):
    rng = np.random.default_rng(1)
    kinds = [(("f32", "bf16")[rng.integers(2)], (8, 32)[rng.integers(2)]) for _ in sizes]
    rc, h = create([A.tensor(n, param=p, state_bits=b) for n, (p, b) in zip(sizes, kinds)])
    assert rc == 0
    lay = S.AdamWLayout()
    assert S.lib().shampoo_adamw_get_layout(h, ctypes.byref(lay)) == 0
    runs = [-(-n // 256) for n in sizes]
    want = {32: 0, 8: 0}
    rem = 0
    for i, (k, (p, b)) in enumerate(zip(runs, kinds)):
        st, rm = ctypes.c_int64(), ctypes.c_int64()
        assert S.lib().shampoo_adamw_tensor_runs(h, i, ctypes.byref(st), ctypes.byref(rm)) == 0
        assert st.value == want[b]
        assert rm.value == (rem if p == "bf16" else -1)
        want[b] += k
        rem += k if p == "bf16" else 0
    assert (lay.runs32, lay.runs8, lay.runs_rem) == (want[32], want[8], rem)
    parts = [(lay.off_clock, 64), (lay.off_m, lay.runs32 * 1024), (lay.off_v, lay.runs32 * 1024),
             (lay.off_m8, lay.runs8 * 256), (lay.off_s8, lay.runs8 * 256),
             (lay.off_m_scale, lay.runs8 * 4), (lay.off_s_scale, lay.runs8 * 4),
             (lay.off_rem, lay.runs_rem * 512)]
    end = 0
    for off, size in sorted(p for p in parts if p[1]):
        assert off % 256 == 0 and off >= end
        end = off + size
    assert end <= lay.total
    S.lib().shampoo_adamw_destroy(h)


def test_counting_of_steps():
    """Each tensor has a count of its own in the clocks' region, an empty one
    none."""
    L = S.lib()
    sizes = [5, 0, 2049, 300, 1, 70000]
    rc, h = create([A.tensor(n, state_bits=(8, 32)[i % 2]) for i, n in enumerate(sizes)])
    assert rc == 0
    lay = S.AdamWLayout()
    assert L.shampoo_adamw_get_layout(h, ctypes.byref(lay)) == 0
    at = []
    for i, n in enumerate(sizes):
        off = ctypes.c_int64()
        assert L.shampoo_adamw_tensor_count(h, i, ctypes.byref(off)) == 0
        if n == 0:
            assert off.value == -1
            continue
        assert off.value % 64 == 8 and off.value >= lay.off_clock
        at.append(off.value)
    clocks = sum(-(-n // 2048) for n in sizes)
    assert len(set(at)) == len(at) and max(at) < lay.off_clock + 64 * clocks
    off = ctypes.c_int64()
    assert L.shampoo_adamw_tensor_count(h, len(sizes), ctypes.byref(off)) == E_ARG
    assert L.shampoo_adamw_tensor_count(h, -1, ctypes.byref(off)) == E_ARG
    assert L.shampoo_adamw_tensor_count(h, 0, None) == E_ARG
    assert L.shampoo_adamw_tensor_count(None, 0, ctypes.byref(off)) == E_ARG
    steps = (ctypes.c_int64 * len(sizes))()
    assert L.shampoo_adamw_set_tensor_steps(h, steps, None) == E_STATE       # the handle's are counted
    for bad in (-1, 2):
        assert L.shampoo_adamw_set_counting(h, bad) == E_ARG
    assert L.shampoo_adamw_set_counting(None, 1) == E_ARG
    assert L.shampoo_adamw_set_counting(h, 1) == 0
    assert L.shampoo_adamw_set_tensor_steps(h, steps, None) == E_STATE       # no state bound
    assert L.shampoo_adamw_set_tensor_steps(h, None, None) == E_ARG
    L.shampoo_adamw_destroy(h)


# ------------------------------------------------------------ the oracle itself
def test_oracle_codes_are_e4m3():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.decode(codes), ref, equal_nan=True)


def test_oracle_store_brackets_and_mean():
    """Every y goes to one of the two codes next to it, upward for that share of
    the 65536 random values that makes the mean y (to the resolution 2^-16 of a
    code); a code goes to itself."""
    vals = O.e4m3_values()
    r = np.arange(65536.0)
    rng = np.random.default_rng(3)
    for y in np.concatenate([448 * 2.0 ** rng.uniform(-20, 0, 60), [0.0, 2.0 ** -9, 2.0 ** -6, 448.0]]):
        z = O.store(np.full(r.size, y), r, False)
        k = np.searchsorted(vals, y, side="right") - 1
        up = vals[min(k + 1, 126)]
        assert set(np.unique(z)) <= {vals[k], up}
        assert abs(z.mean() - y) <= (up - vals[k]) * 2.0 ** -16
    assert O.store(np.array([1e-30]), np.array([0.0]), True)[0] == 2.0 ** -9
    assert O.store(np.array([0.0]), np.array([65535.0]), True)[0] == 0.0


def test_oracle_hash_is_even():
    """Bits, and neighbouring elements, steps and tensors, are as independent as
    random ones: 6 standard deviations of a fair coin over 2^16 draws."""
    n = 1 << 16
    e = np.arange(n)
    base = O.random_bits(7, 3, 2, e)
    others = [O.random_bits(7, 4, 2, e), O.random_bits(7, 3, 3, e), O.random_bits(8, 3, 2, e),
              O.random_bits(7, 3, 2, e + 1), O.random_bits(7, 3, 2, e + (1 << 32))]
    bound = 6 * 0.5 / np.sqrt(n)
    for half in (0, 1):
        a = base[half].astype(np.int64)
        for b in range(16):
            assert abs(((a >> b) & 1).mean() - 0.5) < bound
            for o in others:
                assert abs((((a ^ o[half].astype(np.int64)) >> b) & 1).mean() - 0.5) < bound
    cross = base[0].astype(np.int64) ^ base[1].astype(np.int64)
    for b in range(16):
        assert abs(((cross >> b) & 1).mean() - 0.5) < bound


def test_oracle_bf16_split_is_exact_and_nearest():
    rng = np.random.default_rng(5)
    w = rng.integers(0, 1 << 32, 200_000, dtype=np.uint64).astype(np.uint32).view(np.float32)
    w = np.concatenate([w[np.isfinite(w)], np.float32([0, -0.0, 1, 2.0 ** -140, 3.3e38, -3.4e38])])
    hi, rem = O.bf16_split(w)
    assert np.array_equal(O.bf16_join(hi, rem).view(np.uint32), w.view(np.uint32))
    wide = (hi.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    fine = np.isfinite(wide) & (np.abs(w) > 2.0 ** -126)
    assert np.all(np.abs(wide[fine] - w[fine]) <= 2.0 ** -8 * np.abs(w[fine].astype(np.float64)))


def test_oracle_step_against_differences():
    """The step is a descent on a quadratic: with beta 0 it is sign descent with
    its decay, and one step from zero moments moves by lr whatever g."""
    g = np.array([3.0, -1e-3, 0.0, 5e4])
    p = np.array([1.0, 2.0, 3.0, 4.0])
    h = O.Hyper(lr=0.1, eps=1e-300)
    with np.errstate(invalid="ignore", divide="ignore"):
        p1 = O.step(p, g, 0 * g, 0 * g, 1, h)[0]
    assert np.allclose(p1, p - 0.1 * np.sign(g), rtol=1e-12)
    h = O.Hyper(beta1=0.0, beta2=0.0, lr=0.1, weight_decay=0.5, eps=1e-300)
    p1 = O.step(p, g, 0 * g, 0 * g, 5, h)[0]
    assert np.allclose(p1, p * 0.95 - 0.1 * np.sign(g), rtol=1e-12)


def test_oracle_norm():
    assert O.norm([np.array([3.0]), np.array([4.0])], 10.0) == (5.0, 1.0)
    assert O.norm([np.array([3.0]), np.array([4.0])], 1.0, 2.0) == (10.0, 0.2)
    assert O.norm([np.zeros(3)], 1.0) == (0.0, 1.0)
    assert O.norm([np.array([np.inf])], 1.0)[1] == 0.0
