"""Views and given outputs: attention over pages inside a wider buffer gives the
bits that it gives over contiguous ones, writes nothing beside its outputs, and
the same call gives the same bits every time."""
import pytest
import torch

import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 256), (256, 16), (256, 64)])
@pytest.mark.parametrize("Nq", [1, 3, 90, 300])
def test_pages_and_outputs_inside_wider_buffers(d, page, Nq):
    g = torch.Generator().manual_seed(d + page + Nq)
    B, H, Hkv, lens = 3, 6, 2, [Nq + 400, Nq, 0]
    width = -(-max(lens) // page)
    codes, scales, table = ref.make_cache(B * width + 1, Hkv, page, d, B, width, g, lens)
    plain = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    # [pages, page, heads, K and V and a gap, d]
    wide = torch.full((B * width + 1, page, Hkv, 3, d), 0x7F, dtype=torch.uint8, device=DEV)
    for i in (0, 1):
        wide[:, :, :, i] = plain.tensors[i].view(torch.uint8).transpose(1, 2)
    views = [wide[:, :, :, i].transpose(1, 2) for i in (0, 1)]
    cache = binding.Cache(*views, *plain.tensors[2:])
    q = torch.randn(B, Nq, H, d, generator=g).bfloat16().to(DEV).transpose(1, 2)
    n = ints(lens)
    o, lse = binding.forward_cache(q, plain, n, True, 0.1)
    buf = torch.full((B, Nq, 2, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    mine, l_mine = buf[:, :, 1].transpose(1, 2), torch.full_like(lse, 7.0)
    for _ in range(3):
        got = binding.forward_cache(q, cache, n, True, 0.1, out=mine, lse=l_mine)
        assert got[0] is mine and got[1] is l_mine
        assert torch.equal(mine, o) and torch.equal(l_mine, lse)
        assert (buf[:, :, 0] == 7.0).all()
        mine.fill_(7.0)
    binding.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,page", [(1, 64), (70, 16)])
def test_append_with_shared_positions_and_q_in_place(dtype, N, page):
    g = torch.Generator().manual_seed(N)
    B, H, Hkv, d, lens = 4, 6, 2, 128, [N, N + 3, N + 40, N + 100]
    width = -(-max(lens) // page)
    codes, scales, table = ref.make_cache(B * width, Hkv, page, d, B, width, g, lens)
    one, two = (binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table))) for _ in range(2))
    q, k, v = (torch.randn(B, h, N, d, generator=g).to(dtype).to(DEV) for h in (H, Hkv, Hkv))
    rope = binding.Rope([10000.0 ** (-i / 48) for i in range(48)], [i % 3 for i in range(48)])
    pos = torch.randint(0, 9000, (3, 1, N), generator=g, dtype=torch.int32).to(DEV)
    a = binding.cache_append(one, q, k, v, ints(lens), rope=rope, positions=pos)
    same = q.clone()
    b = binding.cache_append(two, same, k, v, ints(lens), rope=rope,
                             positions=pos.expand(3, B, N).contiguous(), q_out=same)
    binding.device_status()
    assert b is same and torch.equal(a, b)
    assert torch.equal(a, binding.rope(q, None, pos, rope)[0])
    for x, y in zip(one.tensors, two.tensors):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
