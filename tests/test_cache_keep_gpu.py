"""fa_cache_keep against its definition in 64 bits: every code and scale of the
cache, windows from one token to many pages, scales far apart, refusals, graphs."""
import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def choose(n, a, gen):
    return sorted(torch.randperm(n, generator=gen)[:a].tolist())


def make(d, page, Hkv, lens, g, spread=None):
    width = max(1, -(-max(lens) // page)) + 1
    B = len(lens)
    codes, scales, table = ref.make_cache(B * width + 2, Hkv, page, d, B, width, g, lens)
    if spread:
        scales = [2.0 ** torch.randint(*spread, s.shape, generator=g).float() for s in scales]
    return codes, scales, table, binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))


def same(cache, want):
    for i in (0, 1):
        got = ref.codes_to_values(cache.tensors[i])
        assert torch.equal(got.nan_to_num(-1.0), want[i].values.nan_to_num(-1.0)), int((got != want[i].values).sum())
        assert torch.equal(cache.tensors[2 + i].double().cpu(), want[i].scales)


def run(d, page, Hkv, lens, new, keeps, N=None, seed=0, spread=None):
    g = torch.Generator().manual_seed(seed + d + page + len(lens))
    codes, scales, table, cache = make(d, page, Hkv, lens, g, spread)
    K = max(1, max(len(k) for k in keeps))
    keep = ints([k + [-5] * (K - len(k)) for k in keeps])
    out = binding.cache_keep(cache, ints(lens), N or max(max(new), K), keep, keep_lens=ints([len(k) for k in keeps]),
                             new_lens=ints(new))
    binding.device_status()
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    for b, k in enumerate(keeps):
        for c in want:
            branch.keep(c, table[b], lens[b] - new[b], k)
    same(cache, want)
    assert out.tolist() == [t - n + len(k) for t, n, k in zip(lens, new, keeps)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_accepted_branches(d, page, Hkv):
    g = torch.Generator().manual_seed(d + page)
    new = [1, 1, 7, 25, 60, 33, 8, 64, 5]
    lens = [1, 18, 7, 300, 60, 49, 2 * page, page + 64, page]
    counts = [1, 0, 3, 6, 60, 1, 8, 9, 2]
    run(d, page, Hkv, lens, new, [choose(n, a, g) for n, a in zip(new, counts)])


@pytest.mark.parametrize("spread", [(-6, 6), (-100, 121)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16)])
def test_scales_far_apart(d, page, spread):
    g = torch.Generator().manual_seed(d)
    new, lens = [90, 100, 40], [130, 100, 47]
    run(d, page, 2, lens, new, [choose(n, a, g) for n, a in zip(new, (30, 77, 39))], spread=spread)


@pytest.mark.parametrize("d,page,Hkv,B", [(64, 16, 1, 1), (128, 64, 2, 1), (128, 16, 1, 2), (256, 256, 1, 1),
                                          (64, 256, 2, 2), (128, 128, 40, 4)])
def test_windows_of_many_pages(d, page, Hkv, B):
    """Windows that a cluster's CTAs share, several runs one after another."""
    g = torch.Generator().manual_seed(d + page)
    n = 300 if Hkv > 8 else 9000
    lens = [n + 37, n + page + 1, n, n + 5][:B]
    keeps = [choose(n, n // 2, g) if b % 2 == 0 else sorted(set(range(n)) - {3, n // 2}) for b in range(B)]
    run(d, page, Hkv, lens, [n] * B, keeps)


def test_the_first_tokens_stay_where_they_are():
    """Kept tokens that do not move leave every byte, and a scale that need not grow."""
    run(128, 64, 2, [200, 100], [120, 100], [list(range(50)), list(range(100))], spread=(-20, 20))
    run(128, 64, 2, [200, 100], [120, 100], [list(range(50)) + [119], [0] + list(range(2, 100))], spread=(-20, 20))


def test_defaults_and_given_outputs():
    g = torch.Generator().manual_seed(3)
    lens = [60, 45]
    codes, scales, table, cache = make(64, 16, 2, lens, g)
    out = torch.full((3,), 7, dtype=torch.int32, device=DEV)
    got = binding.cache_keep(cache, ints(lens), 20, ints([[0, 4, 9], [1, 2, 19]]), out_lens=out[:2])
    binding.device_status()
    assert got.data_ptr() == out.data_ptr() and out.tolist() == [43, 28, 7]
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    for b, k in enumerate([[0, 4, 9], [1, 2, 19]]):
        for c in want:
            branch.keep(c, table[b], lens[b] - 20, k)
    same(cache, want)


def test_codes_of_every_kind():
    """All 256 codes, NaN among them, moved under a scale that grows by 2^0 .. 2^20."""
    for shift in range(0, 21, 3):
        d, page = 128, 16
        codes = torch.zeros(6, 1, page, d, dtype=torch.uint8)
        codes[2, 0, 4:6] = torch.arange(256).reshape(2, d).to(torch.uint8)
        scales = torch.ones(6, 1)
        scales[4] = 2.0 ** shift
        table = torch.tensor([[2, 4]], dtype=torch.int32)
        both = [c.clone().view(torch.float8_e4m3fn) for c in (codes, codes)]
        cache = binding.Cache(*(t.to(DEV) for t in (*both, scales, scales.clone(), table)))
        keep = [4, 5, 20]       # the third comes from the page with the larger scale
        binding.cache_keep(cache, ints([22]), 22, ints([keep]))
        binding.device_status()
        want = [ref.Paged(c, scales) for c in both]
        for c in want:
            branch.keep(c, table[0], 0, keep)
        same(cache, want)


def test_any_positive_scales():
    """Scales that are no powers of two: to one rounding of the ratio and one of the code."""
    g = torch.Generator().manual_seed(9)
    codes, scales, table, _ = make(64, 16, 1, [64], g)
    scales = [s * (1 + torch.rand(s.shape, generator=g)) for s in scales]
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    keep = [0, 17, 18, 40, 63]
    binding.cache_keep(cache, ints([64]), 64, ints([keep]))
    binding.device_status()
    for i in (0, 1):
        before = ref.Paged(codes[i], scales[i]).rows(table[0], 64, 0)[keep]
        now = ref.Paged(cache.tensors[i].cpu(), cache.tensors[2 + i].cpu())
        s = float(now.scales[int(table[0, 0]), 0])
        assert s == max(float(scales[i][int(table[0, t // 16]), 0]) for t in keep)
        got = now.rows(table[0], 5, 0)
        assert ((got - before).abs() <= before.abs() * (2.0 ** -4 + 2.0 ** -22) + s * 2.0 ** -10).all()


def test_strided_pages_and_offsets_past_32_bits():
    d, page, Hkv = 64, 16, 1
    pages = 9
    apart = 1 << 29                                  # bytes from page to page: 4.5 GB in all
    g = torch.Generator().manual_seed(4)
    order = torch.randperm(pages, generator=g)[:4].to(torch.int32)
    table = order.reshape(1, 4)
    codes = [torch.randn(pages, Hkv, page, d, generator=g).mul_(60).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [2.0 ** torch.randint(-8, -4, (pages, Hkv), generator=g).float() for _ in range(2)]
    wide = torch.empty(apart * (pages - 1) + 2 * page * d * 3, dtype=torch.uint8, device=DEV)
    views = []
    for i in (0, 1):
        v = torch.as_strided(wide, (pages, Hkv, page, d), (apart, page * d, 2 * d, 1), i * d)
        v.copy_(codes[i].view(torch.uint8))
        views.append(v)
    cache = binding.Cache(*views, *(s.to(DEV) for s in scales), table.to(DEV))
    keep = [0, 9, 20, 21, 40, 41, 55]
    binding.cache_keep(cache, ints([60]), 56, ints([keep]))
    binding.device_status()
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    for c in want:
        branch.keep(c, table[0], 4, keep)
    same(cache, want)


def test_what_is_out_of_range_is_reported_and_left_alone():
    g = torch.Generator().manual_seed(5)
    lens = [60, 60]
    good = [[1, 5, 9], [0, 2, 40]]
    for lens0, new0, keep0, kept0 in ((-1, 50, [1, 5, 9], 3), (10 ** 6, 50, [1, 5, 9], 3), (60, 51, [1, 5, 9], 3),
                                      (60, -1, [1, 5, 9], 3), (40, 50, [1, 5, 9], 3), (60, 50, [1, 5, 9], 4),
                                      (60, 50, [1, 5, 9], -1), (60, 50, [1, 1, 9], 3), (60, 50, [5, 1, 9], 3),
                                      (60, 50, [1, 5, 50], 3), (60, 50, [-1, 5, 9], 3),
                                      (60, 8, [1, 5, 9], 3)):
        codes, scales, table, cache = make(64, 16, 2, lens, g)
        out = binding.cache_keep(cache, ints([lens0, 60]), 50, ints([keep0, good[1]]), keep_lens=ints([kept0, 3]),
                                 new_lens=ints([new0, 50]))
        assert binding.fa_get_device_status() == binding.FA_ERR_CACHE
        assert out.tolist() == [lens0, 13]
        want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
        for c in want:
            branch.keep(c, table[1], 10, good[1])
        same(cache, want)
    # a page out of range: what comes from it or goes to it is left out, the rest is done
    for bad in (-1, 99):
        codes, scales, table, cache = make(64, 16, 2, lens, g)
        cache.tensors[4][0, 3] = bad                 # tokens 48 on, none of them kept
        binding.cache_keep(cache, ints(lens), 50, ints(good))
        want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
        for b in (0, 1):
            for c in want:
                branch.keep(c, table[b], 10, good[b])
        binding.device_status()
        same(cache, want)
        # (a source in a page that is not there)
        binding.cache_keep(cache, ints(lens), 50, ints([[1, 5, 45], [0, 1, 2]]))
        assert binding.fa_get_device_status() == binding.FA_ERR_CACHE


def test_in_a_graph_with_lengths_that_grow():
    g = torch.Generator().manual_seed(6)
    d, page, Hkv, N = 128, 16, 2, 12
    lens = [30, 45]
    codes, scales, table = ref.make_cache(20, Hkv, page, d, 2, 9, g)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    n, keep, kept, out = ints(lens), torch.zeros(2, 4, dtype=torch.int32, device=DEV), ints([1, 1]), ints([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        binding.cache_keep(cache, n, N, keep, keep_lens=kept, out_lens=out)
        n.copy_(out)
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    now = list(lens)
    for step in range(5):
        chosen = [choose(N, 2 + (step + b) % 3, g) for b in range(2)]
        n.copy_(ints([t + N for t in now]))
        keep.copy_(ints([k + [0] * (4 - len(k)) for k in chosen]))
        kept.copy_(ints([len(k) for k in chosen]))
        graph.replay()
        binding.device_status()
        for b in range(2):
            for c in want:
                branch.keep(c, table[b], now[b], chosen[b])
        now = [t + len(k) for t, k in zip(now, chosen)]
        assert n.tolist() == now
        same(cache, want)


def test_refusals_of_the_binding():
    g = torch.Generator().manual_seed(7)
    *_rest, cache = make(64, 16, 2, [60, 60], g)
    n, k = ints([60, 60]), ints([[0, 1], [0, 1]])
    for bad in (dict(keep=k[:1]), dict(keep=k[0]), dict(keep=k.long()), dict(seq_lens=n.float()),
                dict(keep=k.transpose(0, 1)[:, :1].transpose(0, 1)), dict(new_lens=n[:1]), dict(out_lens=n.long())):
        a = {"seq_lens": n, "window": 9, "keep": k, **bad}
        with pytest.raises(ValueError):
            binding.cache_keep(cache, **a)
    for bad in (dict(window=1), dict(window=0), dict(out_lens=n)):
        a = {"seq_lens": n, "window": 9, "keep": k, **bad}
        with pytest.raises(binding.FaError):
            binding.cache_keep(cache, **a)
