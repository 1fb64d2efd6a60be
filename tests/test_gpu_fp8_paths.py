"""The 8-bit operators on the paths that only some sizes take."""
import pytest

from test_gpu_fp8 import HALF, U, depth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from second_order_optimizer_amd import fp8 as F  # noqa: E402


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
