"""The paged 8-bit cache: fa_cache_append and fa_fwd_cache against 64-bit plain
forms (cache_ref.py), and a run of them together as a server makes it."""
import math

import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}


def dev(x):
    return None if x is None else x.to(DEV)


def device_cache(codes, scales, table):
    return binding.Cache(codes[0].to(DEV), codes[1].to(DEV), scales[0].to(DEV), scales[1].to(DEV),
                         table.to(DEV))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ append
def check_pages(got_codes, got_scales, want, exact_rows, bound=None):
    """Codes and scales against a ref.Paged; `bound`: [pages, Hkv, page, d]
    slack of the values (0 where they are to be equal)."""
    values = ref.codes_to_values(got_codes)
    scales = got_scales.cpu().double()
    assert torch.equal(scales, want.scales)
    a, b = values * scales[..., None, None], want.values * want.scales[..., None, None]
    same = torch.isnan(a) & torch.isnan(b) | (a == b)
    if exact_rows:
        assert same.all()
    else:
        near = (a - b).abs() <= bound
        assert (same | near).all()
        assert same.double().mean() > 0.999


def run_append(dtype, d, page, Hkv, H, N, starts, new, axes, interleaved, pairs, given_pos,
               layout="bnhd", value=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * d + page + N)
    B = len(starts)
    lens = [s + n for s, n in zip(starts, new)]
    width = max(1, max(-(-n // page) for n in lens)) + 1
    codes, scales, table = ref.make_cache(B * width + 2, Hkv, page, d, B, width, g, lens)
    cache = device_cache(codes, scales, table)

    def tokens(heads):
        x = torch.randn(B, N, heads, d, generator=g) * value
        x = x * torch.exp(torch.randn(B, 1, heads, 1, generator=g))
        x = x.to(T[dtype])
        return x.transpose(1, 2) if layout == "bnhd" else x.transpose(1, 2).contiguous()

    q, k, v = tokens(H), tokens(Hkv), tokens(Hkv)
    freq = [10000.0 ** (-i / max(1, pairs)) for i in range(pairs)]
    axis = [i * axes // max(1, pairs) for i in range(pairs)]
    rope = binding.Rope(freq, axis, interleaved) if pairs else None
    pos = torch.randint(0, 200000, (axes, B, N), generator=g, dtype=torch.int32) if given_pos else None
    full = all(n == N for n in new)
    q_out = binding.cache_append(cache, dev(q), dev(k), dev(v), ints(lens),
                                 new_lens=None if full else ints(new), rope=rope, positions=dev(pos))
    binding.device_status()
    if pos is None:
        pos = torch.stack([torch.tensor([starts[b] + i for i in range(N)]) for b in range(B)])[None]
        pos = pos.expand(axes, B, N)
    kr, qr = ref.rotate(k, pos, freq, axis, interleaved), ref.rotate(q, pos, freq, axis, interleaved)
    slack = ref.rotate_slack(k, pairs, interleaved) * 2.0 ** -21
    want_k, want_v = ref.Paged(codes[0], scales[0]), ref.Paged(codes[1], scales[1])
    bound = torch.zeros_like(want_k.values)
    for b in range(B):
        want_k.append(kr[b, :, :new[b]], starts[b], table[b])
        want_v.append(v[b, :, :new[b]].double(), starts[b], table[b])
        for i in range(new[b]):
            p, r = int(table[b][(starts[b] + i) // page]), (starts[b] + i) % page
            # a value within the rotation's error of a border may round to the
            # other side: one step, 2^-3 of the value or 2^-9 of the scale
            bound[p, :, r] = slack[b, :, i] + torch.maximum(
                kr[b, :, i].abs() * 2.0 ** -3, want_k.scales[p][:, None] * 2.0 ** -9) * 1.01
    check_pages(cache.tensors[0], cache.tensors[2], want_k, pairs == 0, bound)
    check_pages(cache.tensors[1], cache.tensors[3], want_v, True)
    for b in range(B):
        qb = qr[b, :, :new[b]]
        lim = ref.half_step(q.dtype) * qb.abs() * 1.001 + 2.0 ** -25 \
            + 2.0 ** -21 * ref.rotate_slack(q, pairs, interleaved)[b, :, :new[b]]
        assert ((q_out[b, :, :new[b]].cpu().double() - qb).abs() <= lim).all()
        assert (q_out[b, :, new[b]:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,page,N", [(64, 16, 1), (128, 64, 1), (256, 32, 3), (128, 16, 40),
                                      (64, 32, 100), (128, 64, 150), (256, 64, 70), (128, 128, 200),
                                      (256, 256, 300)])
@pytest.mark.parametrize("axes,interleaved,part,given", [(1, False, 1, True), (3, True, 1, True),
                                                         (1, False, 2, False), (1, True, 0, False)])
def test_append(dtype, d, page, N, axes, interleaved, part, given):
    starts = [0, 5, page, page - 1, 2 * page + 3]
    run_append(dtype, d, page, 2, 6, N, starts, [N] * 5, axes, interleaved,
               d // 2 // part if part else 0, given)


@pytest.mark.parametrize("d,page,N", [(64, 16, 33), (128, 64, 9), (256, 128, 140)])
def test_append_padded_batch(d, page, N):
    run_append("f16", d, page, 4, 4, N, [0, 7, page, 30, 1, 0], [N, 1, 0, N // 2, N - 1, 0], 1, False,
               d // 2, False, layout="bhnd")


@pytest.mark.parametrize("value", [1e-6, 30.0, 60000.0 / 500])
def test_append_grows_or_keeps_the_scale(value):
    """Tokens far smaller and far larger than those that the page holds."""
    run_append("bf16", 128, 32, 2, 2, 7, [3, 31, 20, 40], [7, 7, 7, 7], 1, False, 0, False, value=value)


def test_append_one_by_one_keeps_what_is_there():
    """A page filled token by token, each larger than the last: the codes that
    are there are rounded again for every new scale, as the definition says."""
    g = torch.Generator().manual_seed(11)
    codes, scales, table = ref.make_cache(3, 1, 16, 64, 1, 2, g)
    cache = device_cache(codes, scales, table)
    want = ref.Paged(codes[1], scales[1])
    for t in range(20):
        x = (torch.randn(1, 1, 1, 64, generator=g) * 2.0 ** t / 100).half()
        binding.cache_append(cache, None, dev(x), dev(x), ints([t + 1]))
        want.append(x[0].double(), t, table[0])
    binding.device_status()
    check_pages(cache.tensors[1], cache.tensors[3], want, True)


def test_append_infinities_nan_zeros_and_extremes():
    g = torch.Generator().manual_seed(12)
    codes, scales, table = ref.make_cache(4, 1, 16, 64, 2, 2, g)
    cache = device_cache(codes, scales, table)
    x = torch.randn(2, 1, 16, 64, generator=g).bfloat16()
    x[0, 0, 2, 5], x[0, 0, 3, 6], x[0, 0, 4, 7] = math.inf, -math.inf, math.nan
    x[1] = 0
    x[1, 0, 1, 0] = 3.3895e38     # the largest bf16
    y = torch.zeros(2, 1, 16, 64).bfloat16()
    y[1, 0, 0, 0] = 1e-38
    binding.cache_append(cache, None, dev(x), dev(y), ints([16, 16]))
    binding.device_status()
    for which, t in ((0, x), (1, y)):
        want = ref.Paged(codes[which], scales[which])
        for b in range(2):
            want.append(t[b].double(), 0, table[b])
        check_pages(cache.tensors[which], cache.tensors[2 + which], want, True)


def test_append_into_strided_pages_leaves_the_rest():
    """Pages as [pages, page, heads, d] inside a wider buffer; what is not a new
    token's row stays, byte for byte."""
    g = torch.Generator().manual_seed(13)
    buf = torch.randint(0, 255, (6, 32, 2, 2, 128), generator=g, dtype=torch.uint8).to(DEV)
    kept = buf.clone()
    kc, vc = (buf[:, :, i].transpose(1, 2) for i in (0, 1))
    sc = [torch.ones(6, 2, device=DEV) for _ in range(2)]
    table = torch.tensor([[4, 1], [0, 5]], dtype=torch.int32)
    cache = binding.Cache(kc, vc, sc[0], sc[1], table.to(DEV))
    x = torch.randn(2, 2, 8, 128, generator=g).half()
    binding.cache_append(cache, None, dev(x), dev(x), ints([36, 8]))
    binding.device_status()
    changed = (buf != kept).any(-1).any(-1).any(-1).cpu()
    allowed = torch.zeros(6, 32, dtype=torch.bool)
    allowed[4, 28:], allowed[1, :4], allowed[0, :8] = True, True, True
    assert not (changed & ~allowed).any()
    assert torch.equal(kc[1, :, :4], vc[1, :, :4]) and bool((sc[0][[2, 3, 5]] == 1).all())


# ------------------------------------------------------------------ attention
def check_attention(o, lse, q, k, v, table, lens, new, causal, scale):
    want, l_want, slack, l_slack = ref.attend(q, k, v, table, lens, new, causal, scale)
    o, lse = o.cpu().double(), lse.cpu().double()
    empty = torch.isneginf(l_want)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    l_err = (lse - l_want)[~empty].abs()
    assert (l_err <= l_slack[~empty]).all(), float((l_err - l_slack[~empty]).max())
    err = (o - want).abs()
    bound = slack * 1.001 + ref.half_step(q.dtype) * (want.abs() + slack) + 2.0 ** -25
    assert (err <= bound).all(), float((err - bound).max())


def run_attention(dtype, d, page, H, Hkv, Nq, lens, new=None, causal=True, layout="bhnd", seed=0,
                  spread=1.0, splice=None):
    g = torch.Generator().manual_seed(seed + d + page + Nq + sum(lens))
    B = len(lens)
    width = max(1, max(-(-n // page) for n in lens)) + 2
    codes, scales, table = ref.make_cache(B * width + 3, Hkv, page, d, B, width, g, lens, spread)
    for c in codes:     # rows past a sequence's length hold anything, NaN among it
        for b in range(B):
            if lens[b] % page:
                c.view(torch.uint8)[int(table[b][lens[b] // page]), :, lens[b] % page:] = 0x7F
    if splice is not None:
        splice(codes, table)
    cache = device_cache(codes, scales, table)
    if layout == "bhnd":
        q = torch.randn(B, H, Nq, d, generator=g).to(T[dtype])
    else:
        q = torch.randn(B, Nq, H, d, generator=g).to(T[dtype]).transpose(1, 2)
    scale = 1.0 / math.sqrt(d)
    o, lse = binding.forward_cache(dev(q), cache, ints(lens), causal, scale,
                                   new_lens=None if new is None else ints(new))
    binding.device_status()
    check_attention(o, lse, q, ref.Paged(codes[0], scales[0]), ref.Paged(codes[1], scales[1]), table,
                    lens, [Nq] * B if new is None else new, causal, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (16, 1), (7, 1)])
def test_single_tokens(dtype, d, page, H, Hkv):
    run_attention(dtype, d, page, H, Hkv, 1, [1, 15, 16, 17, 100, 0, 300, 1031])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv,Nq", [(4, 2, 2), (4, 1, 3), (8, 2, 7), (2, 2, 33), (6, 2, 50),
                                      (2, 1, 150)])
def test_several_tokens(d, causal, H, Hkv, Nq):
    run_attention("bf16", d, 32, H, Hkv, Nq, [Nq, Nq + 1, 200, 333], causal=causal, layout="bnhd")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,page", [(64, 64), (128, 16), (128, 256), (256, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_prompts(dtype, d, page, causal):
    """Many rows: more than one tile and one unit of them, sequences that begin
    with this chunk and that are cached for the most part."""
    run_attention(dtype, d, page, 6, 2, 130, [130, 131, 257, 900, 129], [130, 130, 128, 130, 1],
                  causal=causal, layout="bnhd")


@pytest.mark.parametrize("d,page,B,Hkv,Nq,L", [
    (256, 32, 48, 32, 128, 128), (256, 64, 3, 16, 1500, 1900), (128, 16, 48, 32, 256, 128),
    (128, 128, 24, 16, 300, 700), (64, 64, 64, 32, 256, 128), (64, 16, 20, 16, 600, 640)])
def test_many_units_for_every_cta(d, page, B, Hkv, Nq, L):
    """Long runs of pieces of one key tile and of a few, every SM walking over
    many of them (rings and phases wrap many times), against fp64 on the GPU."""
    g = torch.Generator().manual_seed(d + L)
    lens = [max(1, L - 37 * (b % 3)) for b in range(B)]
    codes, scales, table = ref.make_cache(B * -(-L // page) + 1, Hkv, page, d, B, -(-L // page), g, lens)
    cache = device_cache(codes, scales, table)
    q = torch.randn(B, Hkv, Nq, d, device=DEV).half()
    for causal in (True, False):
        o, lse = binding.forward_cache(q, cache, ints(lens), causal, 0.06)
        binding.device_status()
        for b in range(0, B, 7):
            ids = table[b, :-(-lens[b] // page)].long().to(DEV)
            K, V = ((cache.tensors[i][ids].double() * cache.tensors[2 + i][ids].double()[..., None, None])
                    .transpose(0, 1).reshape(Hkv, -1, d)[:, :lens[b]] for i in (0, 1))
            S = q[b].double() @ K.transpose(-1, -2) * 0.06
            if causal:
                i = torch.arange(Nq, device=DEV)[:, None] + lens[b] - Nq
                S.masked_fill_(torch.arange(lens[b], device=DEV) > i, -math.inf)
            want_l = torch.logsumexp(S, -1)
            some = torch.isfinite(want_l)
            P = torch.where(some[..., None], (S - want_l[..., None]).exp(), 0.0)
            want = P @ V
            # weights to half a step of f16 and small ones to 2^-25, scores to
            # fp32 (2^-13 together, sums of d = 256 products of size up to 2^5)
            bound = (P @ V.abs()) * 2.0 ** -10 + 2.0 ** -11 * want.abs() + lens[b] * 2.0 ** -25 * 448 * 2.0 ** -5
            assert ((o[b].double() - want).abs() <= bound).all()
            assert torch.equal(torch.isneginf(lse[b]), ~some)
            assert float((lse[b].double() - want_l)[some].abs().max()) < 1e-3


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page,H,Nq,lens,news", [
    (64, 16, 3, 67, [20011], [67]), (128, 64, 3, 67, [20011, 150], [67, 60]),
    (256, 32, 3, 67, [9001], [66]), (128, 16, 7, 19, [1290, 1100], [19, 2])])
def test_a_unit_in_many_shares(d, page, H, Nq, lens, news, causal):
    """Many rows of few units: a unit's pieces are those of up to all CTAs, and
    its rows, odd in number, are joined four at a time."""
    run_attention("bf16", d, page, H, 1, Nq, lens, news, causal=causal)


@pytest.mark.parametrize("d,B,Nq", [(64, 700, 1), (128, 300, 2), (256, 1100, 1), (64, 600, 70),
                                    (128, 1100, 40)])
def test_more_sequences_than_a_block_has_threads(d, B, Nq):
    """The walk over the sequences' lengths takes several rounds of a block."""
    g = torch.Generator().manual_seed(B)
    lens = [Nq + int(x) for x in torch.randint(0, 90, (B,), generator=g)]
    lens[3] = lens[B - 2] = 0
    codes, scales, table = ref.make_cache(B * 12 + 1, 1, 16, d, B, 12, g, lens)
    q = torch.randn(B, 1, Nq, d, generator=g).bfloat16()
    cache = device_cache(codes, scales, table)
    o, lse = binding.forward_cache(dev(q), cache, ints(lens), False, 0.1)
    binding.device_status()
    some = list(range(0, B, 37)) + [3, B - 2, B - 1]
    check_attention(o[some], lse[some], q[some], ref.Paged(codes[0], scales[0]),
                    ref.Paged(codes[1], scales[1]), table[some], [lens[b] for b in some],
                    [Nq] * len(some), False, 0.1)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_padded_queries_and_short_sequences(d, page, causal):
    """Query rows that are no tokens, sequences shorter than their query rows,
    empty ones."""
    run_attention("f16", d, page, 4, 2, 12, [12, 40, 0, 3, 100, 5], [12, 3, 4, 9, 0, 5], causal=causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [3, 90])
def test_nan_in_later_tokens_reaches_only_the_rows_that_see_it(d, Nq):
    """A NaN among the last token's values is 0 * NaN for every earlier row of
    the same tile if the weights alone hide it."""
    lens = [100 + Nq]
    g = torch.Generator().manual_seed(5)
    codes, scales, table = ref.make_cache(16, 1, 16, d, 1, 14, g, lens)
    clean = device_cache(codes, scales, table)
    q = torch.randn(1, 2, Nq, d, generator=g).half()
    want, _ = binding.forward_cache(dev(q), clean, ints(lens), True, 0.1)
    last = lens[0] - 1
    for c in codes:
        c.view(torch.uint8)[int(table[0][last // 16]), 0, last % 16, 3] = 0xFF
    o, lse = binding.forward_cache(dev(q), device_cache(codes, scales, table), ints(lens), True, 0.1)
    binding.device_status()
    assert torch.equal(o[:, :, :-1], want[:, :, :-1])
    assert torch.isnan(o[:, :, -1]).all() and torch.isnan(lse[:, :, -1]).all()
    # NaN among the values only: only that column of the row that sees it
    codes[0].view(torch.uint8)[int(table[0][last // 16]), 0, last % 16, 3] = 0x11
    fine = device_cache(codes, scales, table)
    o, lse = binding.forward_cache(dev(q), fine, ints(lens), True, 0.1)
    hit = torch.isnan(o)
    assert hit[:, :, -1, 3].all() and int(hit.sum()) == 2 and torch.isfinite(lse).all()


def test_scales_of_unlike_size():
    """Pages whose value scales differ by 2^40 and more: the weights carry the
    scale, so the large ones must not drown or overflow the small ones' sums."""
    g = torch.Generator().manual_seed(6)
    lens = [500, 77]
    codes, scales, table = ref.make_cache(80, 2, 16, 128, 2, 33, g, lens)
    scales[1] = 2.0 ** torch.randint(-50, 20, (80, 2), generator=g).float()
    cache = device_cache(codes, scales, table)
    q = torch.randn(2, 4, 1, 128, generator=g).bfloat16()
    o, lse = binding.forward_cache(dev(q), cache, ints(lens), True, 0.05)
    binding.device_status()
    check_attention(o, lse, q, ref.Paged(codes[0], scales[0]), ref.Paged(codes[1], scales[1]), table,
                    lens, [1, 1], True, 0.05)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 60])
def test_queries_far_from_one(size):
    """bf16 rows beyond f16's range: scores are the same as for rows of size one
    with the scale taken over by the softmax scale."""
    g = torch.Generator().manual_seed(7)
    codes, scales, table = ref.make_cache(10, 1, 64, 128, 1, 5, g, [300])
    cache = device_cache(codes, scales, table)
    q = torch.randn(1, 4, 1, 128, generator=g).bfloat16()
    a = binding.forward_cache(dev(q), cache, ints([300]), True, 0.1)
    b = binding.forward_cache(dev((q.float() * size).bfloat16()), cache, ints([300]), True,
                              0.1 / size)
    binding.device_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,Nq", [(64, 1), (64, 90), (128, 3), (128, 90), (256, 1), (256, 90)])
def test_scales_whose_product_underflows(d, Nq):
    """Queries of 2^-100 on pages of 2^-60: every score is zero to fp32, and
    what is masked weighs nothing all the same."""
    g = torch.Generator().manual_seed(d + Nq)
    lens = [300, 131]
    codes, scales, table = ref.make_cache(30, 1, 32, d, 2, 12, g, lens)
    scales[0] = torch.full_like(scales[0], 2.0 ** -60)
    cache = device_cache(codes, scales, table)
    q = (torch.randn(2, 2, Nq, d, generator=g) * 2.0 ** -100).bfloat16()
    o, lse = binding.forward_cache(dev(q), cache, ints(lens), True, 0.1)
    binding.device_status()
    check_attention(o, lse, q, ref.Paged(codes[0], scales[0]), ref.Paged(codes[1], scales[1]), table,
                    lens, [Nq, Nq], True, 0.1)


def test_a_long_cache_and_byte_offsets_past_32_bits():
    """300,000 tokens of one sequence, at the far end of a pool of more than
    2^32 bytes; sampled against equal codes: the softmax of equal scores."""
    page, d, Hkv = 256, 128, 8
    pages = (1 << 32) // (Hkv * page * d) + 1300
    k = torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks, vs = torch.ones(pages, Hkv, device=DEV), torch.ones(pages, Hkv, device=DEV)
    n = 300000
    need = -(-n // page)
    table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV)[None]
    v[pages - need:] = 0x38                       # 1.0
    v[pages - 1, :, (n - 1) % page] = 0x40        # 2.0 at the last token
    v[pages - 1, :, (n - 1) % page + 1:] = 0x7F
    cache = binding.Cache(k, v, ks, vs, table)
    q = torch.randn(1, 16, 1, d, device=DEV).bfloat16()
    o, lse = binding.forward_cache(q, cache, ints([n]), True, 1.0)
    binding.device_status()
    assert float((lse - math.log(n)).abs().max()) < 1e-4
    assert float((o.float() - 1).abs().max()) <= 2.0 ** -8 and float(o.float().min()) >= 1.0
    x = torch.randn(1, Hkv, 1, d, device=DEV).bfloat16()
    binding.cache_append(cache, None, x, x, ints([n + 1]))
    binding.device_status()
    got = ref.codes_to_values(cache.tensors[1][pages - 1, :, n % page]) \
        * vs[pages - 1].cpu().double()[:, None]
    want = x[0, :, 0].cpu().double()
    assert bool((vs[pages - 1] == 1).all())       # the page's scale was larger than the token needs
    assert ((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))).all()


def test_the_same_bits_every_time_and_any_workspace():
    g = torch.Generator().manual_seed(8)
    lens = [3000, 1, 700, 2049]
    codes, scales, table = ref.make_cache(400, 4, 16, 128, 4, 190, g, lens)
    cache = device_cache(codes, scales, table)
    q = torch.randn(4, 8, 1, 128, generator=g).bfloat16().to(DEV)
    need = binding.fwd_cache_workspace_size(4, 8, 4, 1, 128)
    first = None
    for fill in (0, 0xFF, 0x3F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        out = binding.forward_cache(q, cache, ints(lens), True, 0.09, workspace=ws)
        if first is None:
            first = out
        assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    # a sequence alone gives what it gives in a batch, up to where its keys are split
    alone = binding.Cache(*cache.tensors[:4], cache.tensors[4][3:4].contiguous())
    o, lse = binding.forward_cache(q[3:4], alone, ints(lens[3:]), True, 0.09)
    assert float((lse - first[1][3:4]).abs().max()) < 1e-5
    assert float((o.float() - first[0][3:4].float()).abs().max()) <= 2.0 ** -8 * float(o.float().abs().max())
    binding.device_status()


def test_ranges_out_of_bounds_are_reported():
    """Lengths and pages outside their range are skipped on the device and
    reported; the other sequences are served."""
    g = torch.Generator().manual_seed(9)
    lens = [40, 40, 40]
    codes, scales, table = ref.make_cache(12, 2, 16, 64, 3, 3, g, lens)
    good = device_cache(codes, scales, table)
    q = torch.randn(3, 4, 1, 64, generator=g).half().to(DEV)
    want = binding.forward_cache(q, good, ints(lens), True, 0.1)
    binding.device_status()
    for bad in (49, -1):
        o, lse = binding.forward_cache(q, good, ints([40, bad, 40]), True, 0.1)
        with pytest.raises(binding.FaError) as e:
            binding.device_status()
        assert e.value.status == binding.FA_ERR_CACHE
        assert torch.equal(o[[0, 2]], want[0][[0, 2]])
        assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    for page in (12, -1):
        table2 = table.clone()
        table2[1, 1] = page
        cache = device_cache(codes, scales, table2)
        o, _ = binding.forward_cache(q, cache, ints(lens), True, 0.1)
        with pytest.raises(binding.FaError):
            binding.device_status()
        assert torch.equal(o[[0, 2]], want[0][[0, 2]])
        kept = [t.clone() for t in cache.tensors]
        x = torch.randn(3, 2, 9, 64, generator=g).half().to(DEV)
        binding.cache_append(cache, None, x, x, ints([8, 25, 9]))   # 8 < 9 new; rows 16.. on the bad page
        with pytest.raises(binding.FaError) as e:
            binding.device_status()
        assert e.value.status == binding.FA_ERR_CACHE
        touched = (cache.tensors[1].view(torch.uint8) != kept[1].view(torch.uint8)).any(-1).any(-1).any(-1)
        assert set(touched.nonzero()[:, 0].tolist()) == {int(table[2][0])}
    binding.device_status()


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (256, 64)])
def test_ranges_out_of_bounds_with_many_rows(d, page):
    """The same for chunks of prompts: the bad sequence is reported, the others
    are served as they are without it."""
    g = torch.Generator().manual_seed(d)
    lens = [200, 333, 150]
    width = -(-333 // page)
    codes, scales, table = ref.make_cache(3 * width + 1, 2, page, d, 3, width, g, lens)
    q = torch.randn(3, 4, 100, d, generator=g).bfloat16().to(DEV)
    want = binding.forward_cache(q, device_cache(codes, scales, table), ints(lens), True, 0.1)
    binding.device_status()
    for bad_len, bad_page in ((width * page + 1, None), (-5, None), (333, 3 * width + 1), (333, -1)):
        bad = table.clone()
        if bad_page is not None:
            bad[1, 2] = bad_page
        o, lse = binding.forward_cache(q, device_cache(codes, scales, bad), ints([200, bad_len, 150]),
                                       True, 0.1)
        with pytest.raises(binding.FaError) as e:
            binding.device_status()
        assert e.value.status == binding.FA_ERR_CACHE
        # (cut into other shares, so joined from other pieces: of both results the
        # weights are rounded to half a step of f16, 2^-11 of values up to 448
        # scales, and o to half a step of bf16, 2^-8)
        for b in (0, 2):
            assert float((o[b].float() - want[0][b].float()).abs().max()) <= 2 * (
                2.0 ** -8 * float(want[0][b].abs().max()) + 2.0 ** -11 * 448 * float(scales[1].max()))
            assert float((lse[b] - want[1][b]).abs().max()) <= 1e-4
        if bad_page is None:
            assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    binding.device_status()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,page,H,Hkv", [(64, 16, 4, 2), (128, 64, 8, 2), (256, 32, 2, 1)])
def test_a_server_s_run(d, page, H, Hkv):
    """Prompts of unlike length, then single tokens, in one captured graph whose
    lengths grow on the device; against fp64 over all tokens so far."""
    g = torch.Generator().manual_seed(10)
    B, N, scale = 3, 45, 1.0 / math.sqrt(d)
    new = [45, 17, 1]
    width = -(-(N + 8) // page)
    codes, scales, table = ref.make_cache(B * width + 1, Hkv, page, d, B, width, g)
    cache = device_cache(codes, scales, table)
    freq = [10000.0 ** (-i / (d // 2)) for i in range(d // 2)]
    rope = binding.Rope(freq)

    def tokens(n):
        return [torch.randn(B, n, h, d, generator=g).bfloat16().transpose(1, 2) for h in (H, Hkv, Hkv)]

    q, k, v = tokens(N)
    lens = ints(new)
    qr = binding.cache_append(cache, dev(q), dev(k), dev(v), lens, new_lens=ints(new), rope=rope)
    o, lse = binding.forward_cache(qr, cache, lens, True, scale, new_lens=ints(new))
    binding.device_status()

    def held():
        return [ref.Paged(cache.tensors[i], cache.tensors[2 + i]) for i in (0, 1)]

    check_attention(o, lse, qr.cpu(), *held(), table, new, new, True, scale)
    # single tokens, captured once
    q1, k1, v1 = (dev(x).contiguous() for x in tokens(1))
    ws = torch.empty(binding.fwd_cache_workspace_size(B, H, Hkv, 1, d), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        qg = binding.cache_append(cache, q1, k1, v1, lens, rope=rope)
        og, lg = binding.forward_cache(qg, cache, lens, True, scale, workspace=ws)
    for step in range(6):
        nq, nk, nv = tokens(1)
        q1.copy_(nq), k1.copy_(nk), v1.copy_(nv)
        graph.replay()
        binding.device_status()
        now = [n + step + 1 for n in new]
        assert lens.tolist() == now
        check_attention(og, lg, qg.cpu(), *held(), table, now, [1] * B, True, scale)
        # the key that was stored is the rotated one, to half a step of e4m3
        want = ref.rotate(nk, torch.tensor(now)[None, :, None] - 1, freq, [0] * len(freq), False)
        K = held()[0]
        for b in range(B):
            for h in range(Hkv):
                got = K.rows(table[b], now[b], h)[-1]
                s = float(K.scales[int(table[b][(now[b] - 1) // page]), h])
                lim = want[b, h, 0].abs() * 2.0 ** -4 + s * 2.0 ** -10 + 1e-5
                assert ((got - want[b, h, 0]).abs() <= lim).all()


def test_on_a_stream_of_its_own():
    """Calls on a given stream: what they allocate is that stream's, and inputs
    freed right after a call are not handed out under it."""
    g = torch.Generator().manual_seed(14)
    lens = [700, 130]
    codes, scales, table = ref.make_cache(60, 2, 16, 128, 2, 45, g, lens)
    cache = device_cache(codes, scales, table)
    q = torch.randn(2, 4, 3, 128, generator=g).bfloat16()
    k = torch.randn(2, 2, 3, 128, generator=g).bfloat16()
    here = binding.Cache(*(t.clone() for t in cache.tensors))
    rope = binding.Rope([10000.0 ** (-i / 64) for i in range(64)])
    n = ints(lens)
    qr = binding.cache_append(here, dev(q), dev(k), dev(k), n, rope=rope)
    want = binding.forward_cache(qr, here, n, True, 0.1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a, b, c = dev(q), dev(k), dev(k)
        s.wait_stream(torch.cuda.current_stream())
        qs = binding.cache_append(cache, a, b, c, n, rope=rope, stream=s)
        del a, b, c
        torch.full((2, 4, 3, 128), 7.0, device=DEV, dtype=torch.bfloat16)
        o, lse = binding.forward_cache(qs, cache, n, True, 0.1, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    binding.device_status(s)


def test_two_graphs_with_a_workspace_each_run_together():
    g = torch.Generator().manual_seed(15)
    lens = [3000, 2500]
    codes, scales, table = ref.make_cache(400, 2, 16, 128, 2, 190, g, lens)
    cache = device_cache(codes, scales, table)
    n, runs = ints(lens), []
    for i in range(2):
        q = torch.randn(2, 8, 1 + 40 * i, 128, generator=g).bfloat16().to(DEV)
        want = binding.forward_cache(q, cache, n, True, 0.1)
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = binding.forward_cache(q, cache, n, True, 0.1)
        runs.append((graph, s, out, want, q))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s, *_rest in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _graph, _s, out, want, _q in runs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    binding.device_status()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_of_another_device_than_the_current_one():
    g = torch.Generator().manual_seed(16)
    codes, scales, table = ref.make_cache(12, 2, 16, 64, 1, 10, g, [150])
    q = torch.randn(1, 4, 1, 64, generator=g).half()
    outs = []
    for d in ("cuda:0", "cuda:1"):
        c = binding.Cache(*(t.to(d) for t in (*codes, *scales, table)))
        n = torch.tensor([150], dtype=torch.int32, device=d)
        outs.append(binding.forward_cache(q.to(d), c, n, True, 0.1)[0].cpu())
    assert torch.equal(*outs)
