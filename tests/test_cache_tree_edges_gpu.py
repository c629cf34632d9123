"""fa_fwd_cache_tree where parts of a row's keys are joined: parts that weigh nothing
beside the others but hold a NaN."""
import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# drafts, of one or two heads: a unit of the few-row kernel; a tile of the other, whose
# keys its two softmax groups share out at d <= 128; two tiles and more
ROWS = [4, 40, 100, 150]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cache_of(codes, scales, table):
    return binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("low", [0, 1])
def test_nan_values_in_halves_that_weigh_nothing(dtype, d, N, low):
    """Keys of one half of each 128 stand 2^230 below the others and one of them, ahead of the drafts,
    has a NaN value: 0 * NaN, so that every row has it in that column, and only there."""
    g = torch.Generator().manual_seed(d + N)
    page, L = 64, 512 + N
    width = -(-L // page)
    codes, scales, table = ref.make_cache(width + 1, 1, page, d, 1, width, g, [L])
    for n in range(width):
        codes[0][int(table[0, n])] = torch.full((1, page, d), -1.0 if n % 2 == low else 1.0).to(torch.float8_e4m3fn)
    one = torch.ones_like(scales[0])
    at, col = 128 * 2 + 64 * low + 11, 3
    codes[1].view(torch.uint8)[int(table[0, at // page]), 0, at % page, col] = 0x7F
    sees = torch.ones(N, N, dtype=torch.bool).tril()
    q = torch.ones(1, 2, N, d, dtype=dtype)
    scale = 80.0 / d                       # scores of 80 and -80
    o, lse = binding.forward_cache_tree(q.to(DEV), cache_of(codes, (one, scales[1]), table), ints([L]),
                                        branch.pack(sees, N)[None].to(DEV), scale)
    binding.device_status()
    assert o[..., col].isnan().all()
    V = ref.Paged(codes[1], scales[1])
    V.values[int(table[0, at // page]), 0, at % page, col] = 0.0
    want, l_want, o_slack, l_slack = branch.attend_tree(q, ref.Paged(codes[0], one), V, table, [L], [sees], scale)
    err = (o.cpu().double() - want).abs()
    err[..., col] = 0
    assert (err <= ref.half_step(dtype) * want.abs() * 1.001 + 2.0 ** -25 + o_slack).all()
    assert ((lse.cpu().double() - l_want).abs() <= l_slack + 2.0 ** -23 * l_want.abs()).all()
