"""fa_rope at far positions with frequencies on both sides of a turn, against
angles reduced in exact arithmetic (a 64-bit product of position and frequency
is itself off there)."""
import math
from fractions import Fraction

import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PI = Fraction(int("314159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798"),
              10 ** 101)


def angle_of(pos, freq):
    """pos * freq modulo a turn, in [0, 2 pi)."""
    turns = Fraction(freq) * pos / (2 * PI)
    return float(turns - math.floor(turns)) * 2 * math.pi


FREQS = [1.0, 3.7, 19.0, 100.0, -100.0, 1000.0, -1e-3, 12345.678, -0.75, 2.0 ** 30, 1e-9, 0.1, -1e6, 6.0, 2.5, 1e9]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_far_positions_with_any_frequency(interleaved, back):
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 1, 123456789, -987654321, 1000003, 7, 0]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 40, len(pos), 64, generator=g).half()
    table = binding.Rope(FREQS, interleaved=interleaved)
    call = binding.rope_backward if back else binding.rope
    got, _ = call(x.to(DEV), None, torch.tensor([pos], dtype=torch.int32, device=DEV), table)
    a = torch.tensor([[angle_of(p, f) for f in FREQS] for p in pos], dtype=torch.float64)
    c, s = a.cos(), a.sin() * (-1 if back else 1)
    P = len(FREQS)
    one = slice(0, 2 * P, 2) if interleaved else slice(0, P)
    two = slice(1, 2 * P, 2) if interleaved else slice(P, 2 * P)
    want = x.double()
    y = want.clone()
    want[..., one] = y[..., one] * c - y[..., two] * s
    want[..., two] = y[..., two] * c + y[..., one] * s
    # one rounding of the result; angles, sines and the sum in fp32: 2^-21 of
    # |x1| + |x2|; results below f16's normal range round to 2^-25
    bound = ref.half_step(x.dtype) * want.abs() * 1.001 + 2.0 ** -25 + 2.0 ** -21 * ref.rotate_slack(x, P, interleaved)
    err = (got.cpu().double() - want).abs()
    assert (err <= bound).all(), (float((err - bound).max()), [FREQS[i] for i in range(P) if not (err <= bound)[..., one][..., i].all()])
