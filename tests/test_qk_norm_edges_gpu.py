"""fa_qk_norm_rope and its backward where fp32 ends: rows, weights and eps far from
one, with results that are held to their own type's smallest step."""
import pytest
import torch

import branch_ref as branch
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# half of the type's smallest step
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def still(x, back):
    """No rotation."""
    return x


def forward_is(got, x, w, eps):
    """One rounding, and 2^-20 of each value in fp32: r from a sum of up to 256 squares (13 steps of
    2^-24 one after another, halved by the root), rsqrt (2^-22), two products."""
    want = branch.norm(x, w, eps, 0.0, still)
    bound = torch.finfo(got.dtype).eps / 2 * want.abs() * 1.001 + LEAST[got.dtype] + 2.0 ** -20 * want.abs()
    return bool(((got.cpu().double() - want).abs() <= bound).all())


def backward_is(got, dy, x, w, eps):
    """u and h are off by 2^-20 each; the mean of their products adds 13 steps of 2^-24, its product
    with h one: 2^-19 of r (|u| + |h| mean |u h|)."""
    want, _ = branch.norm_backward(dy, x, w, eps, 0.0, still)
    x, f = x.double(), 1.0 if w is None else w.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u, h = (dy.double() * f).abs(), (x * r).abs()
    bound = torch.finfo(got.dtype).eps / 2 * want.abs() * 1.001 + LEAST[got.dtype] \
        + 2.0 ** -19 * r * (u + h * (u * h).mean(-1, keepdim=True))
    return bool(((got.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype,power,dy_power", [
    (torch.bfloat16, 100, 100), (torch.bfloat16, 66, 66), (torch.bfloat16, 100, 60), (torch.bfloat16, 62, 62),
    (torch.bfloat16, 124, 110), (torch.bfloat16, 66, 0), (torch.bfloat16, -50, -50), (torch.float16, 13, 13)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_of_rows_far_from_one(dtype, power, dy_power, d, interleaved):
    """Rows whose squares leave fp32 (from 2^64 on) are taken times 2^-70, and r is brought back.  The
    check turns down a gradient of zeros and, where rows are taken so, one that is not brought back."""
    g = torch.Generator().manual_seed(d + power)
    x = (torch.randn(1, 3, 9, d, generator=g) * 2.0 ** power).to(dtype)
    dy = (torch.randn(1, 3, 9, d, generator=g) * 2.0 ** dy_power).to(dtype)
    w = torch.rand(d, generator=g).add(0.5).to(dtype)
    table = binding.Rope([0.0] * 8, None, interleaved)       # (turns of 0: another layout of the slots)
    eps = 2.0 ** -99 if power < 0 else 1e-6
    y, _ = binding.qk_norm_rope(x.to(DEV), None, w.to(DEV), None, eps, None, table)
    dx, _, dw, _ = binding.qk_norm_rope_backward(dy.to(DEV), None, x.to(DEV), None, w.to(DEV), None, eps, None, table)
    binding.device_status()
    assert forward_is(y, x, w, eps)
    assert backward_is(dx, dy, x, w, eps)
    assert not backward_is(torch.zeros_like(dx), dy, x, w, eps)
    for wrong in (2.0 ** 70, 2.0 ** -70):
        assert not backward_is((dx.double() * wrong).to(dtype), dy, x, w, eps)
    want_dw = branch.norm_backward(dy, x, w, eps, 0.0, still)[1]
    size = (dy.double() * branch.norm(x, None, eps, 0.0, still)).abs().sum((0, 1, 2))
    assert ((dw.cpu().double() - want_dw).abs() <= 2.0 ** -17 * size).all()


@pytest.mark.parametrize("power,w_power,eps", [
    (60, 70, 1e-6), (30, 110, 1e-6), (100, 120, 1e-6), (-60, -80, 2.0 ** -99), (-20, -110, 1e-6), (66, -100, 1e-6)])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weights_far_from_one(power, w_power, eps, d, interleaved):
    """y = (x r) w: where x w leaves fp32, but the result does not."""
    g = torch.Generator().manual_seed(d + power)
    x = (torch.randn(1, 3, 9, d, generator=g) * 2.0 ** power).bfloat16()
    w = torch.rand(d, generator=g).add(0.5) * 2.0 ** w_power
    for table in (None, binding.Rope([0.0] * (d // 2), None, interleaved)):
        y, _ = binding.qk_norm_rope(x.to(DEV), None, w.to(DEV), None, eps, None, table)
        binding.device_status()
        assert forward_is(y, x, w, eps)


@pytest.mark.parametrize("power,eps", [(63.5, 2.0 ** 127), (62.0, 2.0 ** 127), (64.0, 2.0 ** 126), (60.0, 1.999 * 2.0 ** 127),
                                       (0.0, 2.0 ** 127), (66.0, 2.0 ** 120)])
@pytest.mark.parametrize("d", [64, 256])
def test_eps_of_any_size(power, eps, d):
    """Also beside rows whose squares leave fp32, and where the mean and eps together do."""
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(1, 3, 9, d, generator=g).clamp(-1.9, 1.9) * 2.0 ** power).bfloat16()
    dy = (torch.randn(1, 3, 9, d, generator=g) * 2.0 ** 60).bfloat16()
    y, _ = binding.qk_norm_rope(x.to(DEV), None, None, None, eps)
    dx, *_rest = binding.qk_norm_rope_backward(dy.to(DEV), None, x.to(DEV), None, None, None, eps)
    binding.device_status()
    assert forward_is(y, x, None, eps)
    assert backward_is(dx, dy, x, None, eps)
