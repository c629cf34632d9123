"""The codes that fa_cache_append writes, one by one: a rotated key may only
take the code on the other side of a border that its value lies within the
rotation's error of, and nothing but the new tokens' rows changes."""
import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,page,N", [(64, 16, 1), (128, 64, 1), (256, 32, 3), (128, 16, 40), (64, 32, 100),
                                      (128, 128, 200), (256, 256, 300)])
@pytest.mark.parametrize("axes,interleaved,part", [(1, False, 1), (3, True, 1), (2, False, 2)])
def test_every_new_code(dtype, d, page, N, axes, interleaved, part):
    g = torch.Generator().manual_seed(d + page + N + axes)
    starts = [0, 5, page, page - 1, 2 * page + 3]
    B, Hkv, lens = len(starts), 2, [s + N for s in starts]
    width = -(-max(lens) // page)
    codes, scales, table = ref.make_cache(B * width + 2, Hkv, page, d, B, width, g, lens)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    pairs = d // 2 // part
    freq, axis = [10000.0 ** (-i / pairs) for i in range(pairs)], [i * axes // pairs for i in range(pairs)]
    k, v = (torch.randn(B, Hkv, N, d, generator=g).to(T[dtype]) for _ in range(2))
    pos = torch.randint(0, 200000, (axes, B, N), generator=g, dtype=torch.int32)
    binding.cache_append(cache, None, k.to(DEV), v.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                         rope=binding.Rope(freq, axis, interleaved), positions=pos.to(DEV))
    binding.device_status()
    turned = ref.rotate(k, pos, freq, axis, interleaved)
    slack = ref.rotate_slack(k, pairs, interleaved) * 2.0 ** -21      # angles, sines and the sum, in fp32
    for which, x in ((0, turned), (1, v.double())):
        want = ref.Paged(codes[which], scales[which])
        for b in range(B):
            want.append(x[b], starts[b], table[b])
        got = ref.codes_to_values(cache.tensors[which])
        assert torch.equal(cache.tensors[2 + which].cpu().double(), want.scales)
        new = torch.zeros(got.shape[:3], dtype=torch.bool)
        for b in range(B):
            for i in range(N):
                p, r = int(table[b][(starts[b] + i) // page]), (starts[b] + i) % page
                new[p, :, r] = True
                s = want.scales[p][:, None]
                lo, hi = (ref.to_e4m3((x[b, :, i] + e) / s) for e in ((-slack[b, :, i], slack[b, :, i]) if which == 0
                                                                     else (0.0, 0.0)))
                assert ((got[p, :, r] == lo) | (got[p, :, r] == hi)).all()
        assert torch.equal(got[~new], want.values[~new])
