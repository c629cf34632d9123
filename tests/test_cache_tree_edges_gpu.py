"""fa_fwd_cache_tree where parts of a row's keys are joined: parts that weigh nothing
beside the others but hold a NaN, parts whose value scales lie far apart; and with
outputs, streams and layouts of pages of the caller's own."""
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


def some(d, H, Hkv, N, lens, page, g, pages=None):
    """(q, codes, scales, table, trees) of a batch with N drafts each."""
    width = max(-(-n // page) for n in lens)
    codes, scales, table = ref.make_cache(pages or len(lens) * width + 1, Hkv, page, d, len(lens), width, g, lens)
    q = torch.randn(len(lens), N, H, d, generator=g).bfloat16().transpose(1, 2)
    return q, codes, scales, table, [branch.sees_of(branch.random_tree(N, g)) for _ in lens]


def packed(sees, N):
    return torch.stack([branch.pack(s, N) for s in sees]).to(DEV)


def check(o, lse, q, codes, scales, table, lens, sees, scale):
    K, V = (ref.Paged(codes[i], scales[i]) for i in (0, 1))
    want, l_want, o_slack, l_slack = branch.attend_tree(q, K, V, table, lens, sees, scale)
    err = (o.cpu().double() - want).abs()
    assert (err <= ref.half_step(o.dtype) * want.abs() * 1.001 + 2.0 ** -25 + o_slack).all()
    assert ((lse.cpu().double() - l_want).abs() <= l_slack + 2.0 ** -23 * l_want.abs()).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", [5, 60, 150])
def test_outputs_of_the_callers_on_a_stream_of_its_own(d, N):
    """An output inside a wider buffer, whose other elements stay, an lse, a workspace and a stream: the
    same bits as without."""
    g = torch.Generator().manual_seed(d + N)
    lens = [N + 3000, N, N + 65]
    q, codes, scales, table, sees = some(d, 4, 2, N, lens, 32, g)
    cache, mask, n = cache_of(codes, scales, table), packed(sees, N), ints(lens)
    q = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=DEV).copy_(q)
    want = binding.forward_cache_tree(q, cache, n, mask, 0.1)
    binding.device_status()
    check(*want, q.cpu(), codes, scales, table, lens, sees, 0.1)
    wide = torch.full((3, N, 6, 2 * d), 7.0, dtype=q.dtype, device=DEV)
    out = wide[:, :, 1:5, :d].transpose(1, 2)
    lse = torch.full((2, 3, 4, N), 7.0, device=DEV)
    ws = torch.full((binding.fwd_cache_tree_workspace_size(3, 4, 2, N, d),), 0xFF, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = binding.forward_cache_tree(q, cache, n, mask, 0.1, out=out, lse=lse[1], workspace=ws, stream=side)
        side.synchronize()
        assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse[1].data_ptr()
        assert torch.equal(out, want[0]) and torch.equal(lse[1], want[1])
        assert (lse[0] == 7).all() and (wide[:, :, 0] == 7).all() and (wide[:, :, 5] == 7).all()
        assert (wide[..., d:] == 7).all()
        out.fill_(3.0), lse[1].fill_(3.0)
        torch.cuda.synchronize()
    for bad in (dict(lse=lse[0, :, :, :1]), dict(lse=lse[0].double()), dict(lse=lse[0].transpose(0, 1)),
                dict(out=out[:2]), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            binding.forward_cache_tree(q, cache, n, mask, 0.1, **bad)
    with pytest.raises(binding.FaError):
        binding.forward_cache_tree(q, cache, n, mask, 0.1, workspace=ws[:-256])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", [5, 60, 150])
@pytest.mark.parametrize("apart", [1 << 20, 1 << 29])
def test_pages_inside_a_wider_buffer(d, N, apart):
    """K and V rows by turns in one buffer, heads and pages far apart in it (past 32 bits in all)."""
    g = torch.Generator().manual_seed(d + N)
    lens, page, Hkv = [N + 40], 64, 2
    pages = 9
    q, codes, scales, table, sees = some(d, 4, Hkv, N, lens, page, g, pages=pages)
    wide = torch.zeros(apart * (pages - 1) + 4 * Hkv * page * d, dtype=torch.uint8, device=DEV)
    views = []
    for i in (0, 1):
        v = torch.as_strided(wide, (pages, Hkv, page, d), (apart, 2 * page * d, 2 * d, 1), i * d)
        v.copy_(codes[i].view(torch.uint8))
        views.append(v)
    cache = cache_of(codes, scales, table)
    there = binding.Cache(*views, *cache.tensors[2:])
    mask = packed(sees, N)
    want = binding.forward_cache_tree(q.to(DEV), cache, ints(lens), mask, 0.1)
    got = binding.forward_cache_tree(q.to(DEV), there, ints(lens), mask, 0.1)
    binding.device_status()
    check(*got, q, codes, scales, table, lens, sees, 0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d,N", [(64, 3), (64, 40), (128, 3), (128, 40), (128, 140), (256, 3), (256, 12)])
def test_a_long_sequence(d, N):
    lens = [131072 - 37, N]
    q, codes, scales, table, sees = some(d, 2, 1, N, lens, 256, torch.Generator().manual_seed(d + N), pages=600)
    o, lse = binding.forward_cache_tree(q.to(DEV), cache_of(codes, scales, table), ints(lens), packed(sees, N), 0.05)
    binding.device_status()
    check(o, lse, q, codes, scales, table, lens, sees, 0.05)
