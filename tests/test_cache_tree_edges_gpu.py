"""fa_fwd_cache_tree where parts of a row's keys are joined: parts that weigh nothing
beside the others but hold a NaN, parts whose value scales lie far apart."""
import math

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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("L", [700, 9000])
@pytest.mark.parametrize("down", [1.0, 8.0, 16.5])
def test_value_scales_far_apart_between_parts(d, N, L, down):
    """One page of 64 keys has value scale 1, all others 2^-100 and weights 2^-down of its keys':
    2^-116.5 at most, which the joins have to keep (down to 2^-118).  The others are many, so that
    together they count in the sum."""
    page = 64
    width = -(-(L + N) // page)
    lens = [L + N]
    g = torch.Generator().manual_seed(d + N)
    codes, scales, table = ref.make_cache(width, 1, page, d, 1, width, g, lens)
    high = int(table[0, width // 2])
    codes[0][:] = torch.zeros(1).to(torch.float8_e4m3fn)
    codes[0][high] = torch.ones(1, page, d).to(torch.float8_e4m3fn)
    # one of the page's keys stands above the others alone
    codes[0][high, 0, 1:] = torch.zeros(page - 1, d).to(torch.float8_e4m3fn)
    ks, vs = torch.ones(width, 1), torch.full((width, 1), 2.0 ** -100)
    vs[high] = 1.0
    codes[1][high] = torch.full((1, page, d), 256.0).to(torch.float8_e4m3fn)
    sees = torch.ones(N, N, dtype=torch.bool).tril()
    q = torch.ones(1, 1, N, d, dtype=torch.float16)
    scale = down * math.log(2.0) / d
    o, lse = binding.forward_cache_tree(q.to(DEV), cache_of(codes, (ks, vs), table), ints(lens),
                                        branch.pack(sees, N)[None].to(DEV), scale)
    binding.device_status()
    K, V = ref.Paged(codes[0], ks), ref.Paged(codes[1], vs)
    want, l_want, o_slack, l_slack = branch.attend_tree(q, K, V, table, lens, [sees], scale)
    assert ((lse.cpu().double() - l_want).abs() <= l_slack + 2.0 ** -23 * l_want.abs()).all()
    # weights: half a step of f16, and the scores' and the sums' error on either side
    err = (o.cpu().double() - want).abs()
    assert (err <= want.abs() * (2.0 ** -11 * 1.001 + 2.0 ** -11 + 2 * l_slack[..., None])).all()
