"""fa_cache_keep at the ends of what its interface allows: more tokens to keep than
a window has, at a table's last page."""
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
