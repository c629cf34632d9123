"""How exact fa_fwd_cache is where it is hardest: query rows of tiny elements,
rows with one column far above the rest, and many keys far below one.

Bounds are those of the kernels' own roundings; here each kernel is held to
its own: q is exact to 2^-25 of a row's largest element with few rows, and to
2^-21 of it with many (where keys stay in 8 bits)."""
import math

import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}
FEW, MANY = 1, 90      # query rows of the two kernels at every head dim (one or two heads a key/value head)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def q_error(x, dtype, many):
    """What the operand that stands for a row x [d] of q may be off by, an
    element.  Few rows: f16 with the largest in [1, 2): 2^-25 of it at most (f16
    rows: nothing).  Many rows: the largest is brought to [2^7, 2^8) and parts
    of 8 bits are taken off one after another, the last of them with two
    mantissa bits and steps down to 2^-16.  What the parts before it leave is
    within half of their step 2^-9, so that it is off by half a step of 2^-13
    at most, 2^-14 or 2^-21 of the largest; and only where it has more than
    three bits: elements below 2^-6 (bf16: 8 bits, 4 of them in the first part)
    or 2^-3 (f16: 11 bits, 8 in the first two) of those with the largest at
    2^7 at least, 2^-13 and 2^-10 of it."""
    top = x.abs().max()
    if not many:
        return torch.full_like(x, float(top) * 2.0 ** -25) if dtype == "bf16" else torch.zeros_like(x)
    small = x.abs() < top * (2.0 ** -13 if dtype == "bf16" else 2.0 ** -10)
    return small.double() * top * 2.0 ** -21


def check(o, lse, q, codes, scales, table, lens, causal, scale, dtype, many):
    """Against 64 bits.  Scores: products summed in fp32 (2^-23 a step, in any
    order) and q's own error; exp2, the scaling and the running sums 2^-20
    together.  Weights: half a step of f16, 2^-11, or for small ones 2^-25 where
    the largest stands at 2^7 or above: 2^-32 of it."""
    k, v = (ref.Paged(codes[i], scales[i]) for i in (0, 1))
    B, H, N, d = q.shape
    Hkv = codes[0].shape[1]
    x, o, lse = q.double(), o.cpu().double(), lse.cpu().double()
    for b in range(B):
        for h in range(H):
            K, V = (c.rows(table[b], lens[b], h // (H // Hkv)) for c in (k, v))
            for i in range(N):
                see = lens[b] - N + i + 1 if causal else lens[b]
                S = (K[:see] @ x[b, h, i]) * scale
                L = torch.logsumexp(S, 0)
                P = torch.exp(S - L)
                want = P @ V[:see]
                size = float((K[:see].abs() @ x[b, h, i].abs()).max()) * scale
                off = float((K[:see].abs() @ q_error(x[b, h, i], dtype, many)).max()) * scale
                ds = size * d * 2.0 ** -23 + off + 2.0 ** -20 * (1 + float(S.abs().max()))
                slack = (P @ V[:see].abs()) * (2.0 ** -11 + 2 * ds + see * 2.0 ** -24) \
                    + see * 2.0 ** -32 * 448 * float(v.scales.max())
                bound = slack * 1.001 + ref.half_step(q.dtype) * (want.abs() + slack) + 2.0 ** -25
                err = (o[b, h, i] - want).abs()
                assert (err <= bound).all(), (b, h, i, float((err - bound).max()))
                l_err = abs(float(lse[b, h, i] - L))
                assert l_err <= ds + see * 2.0 ** -24 + 2.0 ** -21 * (1 + abs(float(L))), (b, h, i, l_err)


def cache_of(codes, scales, table):
    return binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [FEW, MANY])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -122, 2.0 ** -126, 2.0 ** 125])
def test_tiny_and_huge_queries(d, Nq, size):
    """bf16 rows at both ends of the type, with zeros among their elements, and
    a softmax scale that makes scores of ordinary size of them."""
    g = torch.Generator().manual_seed(d + Nq)
    lens = [300, 131]
    codes, scales, table = ref.make_cache(30, 1, 32, d, 2, 12, g, lens)
    q = torch.randn(2, 1, Nq, d, generator=g).clamp_(-5, 5)
    q[..., ::5] = 0
    if size > 1:
        q[..., 3] = 255 / 32      # the largest bf16
    q = (q.double() * size).bfloat16()
    scale = float(torch.tensor((0.1 if size < 1 else 0.8) / size, dtype=torch.float32))     # (a normal number)
    o, lse = binding.forward_cache(q.to(DEV), cache_of(codes, scales, table), ints(lens), True, scale)
    binding.device_status()
    check(o, lse, q, codes, scales, table, lens, True, scale, "bf16", Nq == MANY)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [FEW, MANY])
@pytest.mark.parametrize("column", [2.0 ** 7, 2.0 ** 10, 2.0 ** 13])
def test_queries_with_one_column_far_above_the_rest(dtype, d, Nq, column):
    """The large column meets keys of zero, so that the scores are the small
    columns'."""
    g = torch.Generator().manual_seed(d + Nq)
    lens = [140, 131]
    codes, scales, table = ref.make_cache(30, 1, 32, d, 2, 12, g, lens)
    codes[0].view(torch.uint8)[..., 7] = 0
    q = torch.randn(2, 1, Nq, d, generator=g)
    q[..., 7] = column * 1.5
    q = q.to(T[dtype])
    o, lse = binding.forward_cache(q.to(DEV), cache_of(codes, scales, table), ints(lens), True, 0.25)
    binding.device_status()
    check(o, lse, q, codes, scales, table, lens, True, 0.25, dtype, Nq == MANY)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [FEW, MANY])
def test_many_keys_far_below_one(dtype, d, Nq):
    """One key stands 17.4 above 2^17 others, of which each weighs 2^-25.1 of it
    and all together 2^-8: one sequence a CTA, so that no cut of the keys gives
    the small ones a maximum of their own.  (The sequences share their pages.)"""
    n, page = 1 << 17, 256
    B = torch.cuda.get_device_properties(0).multi_processor_count * (2 if Nq == FEW else 1)
    k = torch.zeros(n // page, 1, page, d, dtype=torch.uint8)
    v = torch.full((n // page, 1, page, d), 0x38, dtype=torch.uint8)      # 1.0
    k[0, 0, 0, 0] = 0x38
    v[0, 0, 0] = 0
    one = torch.ones(n // page, 1)
    table = torch.arange(n // page, dtype=torch.int32).expand(B, -1).contiguous()
    cache = cache_of((k, v), (one, one), table)
    q = torch.zeros(B, 1, Nq, d, dtype=T[dtype], device=DEV)
    q[..., 0] = 1
    scale = 17.4
    o, lse = binding.forward_cache(q, cache, ints([n] * B), False, scale)
    binding.device_status()
    w = math.exp(-scale)
    want = (n - 1) * w / (1 + (n - 1) * w)
    # weights: 2^-32 of the largest, each; score and exp2 2^-19.  The row sum is in
    # fp32, and what holds the largest weight takes n / 64 additions (few rows: a
    # lane has one key in 32 and adds two at a time; many: a row adds 64 keys'
    # sum), each rounding to 2^-24 of it: n 2^-30 = 2^-13.  (Two weights of
    # 2^-25.1 are just below half a step of 1, so that a lane loses all of its
    # 4096, 1.1e-4, as few rows do.)
    sums = n * 2.0 ** -30
    bound = n * 2.0 ** -32 + want * (2.0 ** -19 + sums + ref.half_step(T[dtype])) + 2.0 ** -25
    assert float((o.double() - want).abs().max()) <= bound
    assert float((lse.double() - scale - math.log1p((n - 1) * w)).abs().max()) <= 2.0 ** -18 * scale + sums


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [FEW, MANY])
@pytest.mark.parametrize("power", [-100, -99, 118, 119, 120])
def test_value_scales_at_both_ends(d, Nq, power):
    """The smallest and largest value scales: results are those of scales of one
    times the power, and L does not know of them."""
    g = torch.Generator().manual_seed(d + Nq)
    lens = [300, 131]
    codes, scales, table = ref.make_cache(30, 1, 32, d, 2, 12, g, lens)
    codes[1] = codes[1].float().div_(256).to(torch.float8_e4m3fn)       # below 2, so that 2^120 stays in bf16's range
    q = torch.randn(2, 2, Nq, d, generator=g).bfloat16().to(DEV)
    outs = []
    for p in (0, power):
        vs = torch.full_like(scales[1], 2.0 ** p)
        outs.append(binding.forward_cache(q, cache_of(codes, (scales[0], vs), table), ints(lens), True, 0.1))
    binding.device_status()
    (o, lse), (o_p, lse_p) = outs
    # sums of exponents of up to 2^7 round to 2^-18 (weights and L by as much, a
    # few times over: 2^-15), weights to half a step of f16 and o to one of bf16
    # on either side
    want = o.double()
    size = float(codes[1].float().abs().max())
    assert float((lse_p - lse).abs().max()) <= 2.0 ** -15
    assert ((o_p.double() / 2.0 ** power - want).abs() <= 2 * (2.0 ** -8 * want.abs() + 2.0 ** -11 * size)).all()
