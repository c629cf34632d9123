"""fa_cache_keep at the ends of what its interface allows: more tokens to keep than
a window has, at a table's last page; scales of 0; a stream of the caller's."""
import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def same(cache, want):
    for i in (0, 1):
        got = ref.codes_to_values(cache.tensors[i])
        assert torch.equal(got.nan_to_num(-1.0), want[i].values.nan_to_num(-1.0))
        assert torch.equal(cache.tensors[2 + i].double().cpu(), want[i].scales)


@pytest.mark.parametrize("d,page,N,K", [(64, 16, 40, 40), (128, 64, 9, 6), (256, 16, 300, 300)])
@pytest.mark.parametrize("given", [False, True])
def test_more_kept_tokens_than_the_window_has(d, page, N, K, given):
    """Of sequences that fill their tables; the last one's row is the table's last.  They keep
    everything and are reported, the sequence between them is thinned."""
    g = torch.Generator().manual_seed(d + N)
    width = -(-N // page) + 1
    lens, new = [width * page] * 3, [2, N, 0]
    codes, scales, table = ref.make_cache(3 * width, 2, page, d, 3, width, g, lens)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    keep = list(range(K))
    out = binding.cache_keep(cache, ints(lens), N, ints([keep] * 3), keep_lens=ints([K] * 3) if given else None,
                             new_lens=ints(new))
    assert binding.fa_get_device_status() == binding.FA_ERR_CACHE
    assert out.tolist() == [lens[0], lens[1] - N + K, lens[2]]
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    for c in want:
        branch.keep(c, table[1], lens[1] - N, keep)
    same(cache, want)


def keep_with_zeros(held, table_row, base, kept):
    """branch.keep where scales may be 0: a page whose tokens all come with 0 takes them as they are."""
    page = held.values.shape[2]
    old, scales = held.values.clone(), held.scales.clone()
    end = base + len(kept)
    for number in range(base // page, -(-end // page)):
        toks = range(number * page, min(end, (number + 1) * page))
        at = [divmod(t if t < base else base + kept[t - base], page) for t in toks]
        p = int(table_row[number])
        for h in range(scales.shape[1]):
            came = [(old[int(table_row[i]), h, r], float(scales[int(table_row[i]), h])) for i, r in at]
            top = max(s for _, s in came)
            for r, (x, s) in enumerate(came):
                held.values[p, h, r] = x if top == 0 else ref.to_e4m3(x * (s / top))
            held.scales[p, h] = top


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("zeros", [[0], [1], [2, 3], [1, 2, 3], [0, 1, 2, 3], [3]])
def test_pages_of_scale_zero(d, page, zeros):
    """Tokens from pages of scale 0 (with codes of every kind under it) to places that held
    others, among tokens with a scale and alone; places whose own page has none."""
    g = torch.Generator().manual_seed(d + page)
    L = 4 * page - 3
    for base, keep in ((page // 2, range(0, L - page // 2, 2)), (3, range(2 * page, 3 * page)), (0, range(page, 2 * page)),
                       (page, list(range(5)) + list(range(page, page + 9)))):
        keep = list(keep)
        codes, scales, table = ref.make_cache(6, 2, page, d, 1, 4, g)
        for x in codes:
            x.view(torch.uint8)[:, :, ::5, ::7] = 0x7F          # (0 * NaN is NaN)
            x.view(torch.uint8)[:, :, ::3, ::9] = 0x80
        for i in (0, 1):
            for n in zeros:
                scales[i][int(table[0, n]), i:] = 0.0 if n % 2 else -0.0
        cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
        out = binding.cache_keep(cache, ints([L]), L - base, ints([keep]))
        binding.device_status()
        assert out.tolist() == [base + len(keep)]
        want = [ref.Paged(codes[i], scales[i].abs()) for i in (0, 1)]
        for c in want:
            keep_with_zeros(c, table[0], base, keep)
        # (a page without tokens of the sequence keeps the sign of its 0)
        cache.tensors[2].abs_(), cache.tensors[3].abs_()
        same(cache, want)


def test_on_a_stream_of_its_own():
    g = torch.Generator().manual_seed(12)
    lens, N = [3000, 2900], 2800
    codes, scales, table = ref.make_cache(400, 2, 16, 128, 2, 190, g, lens)
    keeps = [sorted(torch.randperm(N, generator=g)[:1500].tolist()) for _ in lens]
    want = [ref.Paged(codes[i], scales[i]) for i in (0, 1)]
    for b, k in enumerate(keeps):
        for c in want:
            branch.keep(c, table[b], lens[b] - N, k)
    side = torch.cuda.Stream()
    for _ in range(5):
        cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
        n, keep = ints(lens), ints(keeps)
        torch.cuda.synchronize()
        out = binding.cache_keep(cache, n, N, keep, stream=side)
        del n, keep
        torch.full((2, 1500), -7, dtype=torch.int32, device=DEV)      # (the current stream's allocations)
        side.synchronize()
        assert out.tolist() == [1700, 1600]
        same(cache, want)
    binding.device_status()
