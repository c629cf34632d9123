"""The 8-bit parts that stand for a row of q in the many-row cache attention,
by enumeration: e4m3 parts, the last one e5m2, over every significand and
every power of two below the row's largest element (in [2^7, 2^8))."""
import pytest
import torch


@pytest.mark.parametrize("bits,parts,exact_from", [(8, 2, -6), (11, 3, -3)])
def test_what_the_parts_leave(bits, parts, exact_from):
    for e in range(7, -20, -1):
        left = (torch.arange(1 << (bits - 1), 1 << bits, dtype=torch.float64) * 2.0 ** (e - bits + 1)).half()
        for n in range(parts):
            part = left.float().to(torch.float8_e5m2 if n + 1 == parts else torch.float8_e4m3fn)
            rest = left.double() - part.double()
            left = rest.half()
            assert torch.equal(left.double(), rest)      # a subtraction of f16 is exact here
        worst = float(left.double().abs().max())
        assert worst == 0 if e >= exact_from else worst <= 2.0 ** -14, e
