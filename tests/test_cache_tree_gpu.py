"""fa_fwd_cache_tree against 64 bits: head layouts, tree sizes around words and
tiles, masks of every kind (rows that see nothing, bits past the drafts), NaN in
masked places, lengths out of range, graphs."""
import math

import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check(o, lse, q, K, V, table, lens, sees, scale):
    want, l_want, o_slack, l_slack = branch.attend_tree(q, K, V, table, lens, sees, scale)
    err = (o.cpu().double() - want).abs()
    bound = ref.half_step(o.dtype) * want.abs() * 1.001 + 2.0 ** -25 + o_slack
    assert (err <= bound).all(), float((err - bound).max())
    lse, none = lse.cpu().double(), l_want == -math.inf
    assert torch.equal(lse == -math.inf, none)
    assert ((lse - l_want).abs()[~none] <= (l_slack + 2.0 ** -23 * l_want.abs())[~none]).all()
    assert (o.cpu()[none] == 0).all()


def random_mask(n, gen, kind):
    if kind == "tree":
        return branch.sees_of(branch.random_tree(n, gen))
    if kind == "any":       # any bits: later tokens, not itself, nothing at all
        sees = torch.rand(n, n, generator=gen) < 0.4
        sees[torch.rand(n, generator=gen) < 0.2] = False
        return sees
    return torch.ones(n, n, dtype=torch.bool).tril()


def run(dtype, d, page, H, Hkv, N, lens, new=None, kind="tree", seed=0, shared=False, layout=True):
    g = torch.Generator().manual_seed(seed + d + page + N + H)
    B = len(lens)
    ns = new or [N] * B
    width = max(1, -(-max(lens) // page))
    codes, scales, table = ref.make_cache(B * width + 1, Hkv, page, d, B, width, g, lens)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    q = torch.randn(B, N, H, d, generator=g).to(T[dtype])
    q = q.transpose(1, 2) if layout else q.transpose(1, 2).contiguous()
    if shared:
        one = random_mask(N, g, kind)
        sees = [one[:n, :n] for n in ns]
        mask = branch.pack(one, N)[None]
    else:
        sees = [random_mask(n, g, kind) for n in ns]
        mask = torch.stack([branch.pack(s, N) for s in sees])
        # rows and bits behind a sequence's tokens are not looked at
        for b, n in enumerate(ns):
            mask[b, n:] = -1
            for i in range(n, N):
                mask[b, :, i // 32] |= (1 << (i % 32)) - (1 << 32 if i % 32 == 31 else 0)
    got = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=DEV).copy_(q)
    o, lse = binding.forward_cache_tree(got, cache, ints(lens), mask.to(DEV), d ** -0.5,
                                        new_lens=None if new is None else ints(new))
    binding.device_status()
    K, V = (ref.Paged(codes[i], scales[i]) for i in (0, 1))
    check(o, lse, q, K, V, table, lens, sees, d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv,N", [(4, 4, 1), (8, 2, 7), (7, 1, 5), (4, 1, 40)])
def test_small_trees(dtype, d, page, H, Hkv, N):
    run(dtype, d, page, H, Hkv, N, [N + 500, N, N + 3, N + 129])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["tree", "any", "causal"])
@pytest.mark.parametrize("N", [2, 31, 32, 33, 63, 64, 65, 127, 130, 200])
def test_sizes_around_words_and_tiles(d, kind, N):
    run("bf16", d, 32, 2, 2, N, [N + 100, N, N + 28, N + 255], kind=kind)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv,N", [(4, 2, 6), (16, 2, 9), (4, 4, 150)])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_padded_batches(d, H, Hkv, N, kind):
    new = [N, 0, N // 2, 1, max(1, N - 1)]
    run("f16", d, 16, H, Hkv, N, [N + 77, 40, N // 2, 90, N + 300], new=new, kind=kind)


@pytest.mark.parametrize("N", [5, 90])
def test_one_tree_for_every_sequence(N):
    run("bf16", 128, 64, 8, 2, N, [N + 9, N, N + 700], shared=True, new=[N, N // 2, N - 1])
    run("bf16", 128, 64, 8, 2, N, [N + 9, N, N + 700], kind="any", shared=True, layout=False)


@pytest.mark.parametrize("d,page,N,H,Hkv", [(64, 16, 3, 8, 4), (128, 64, 4, 8, 8), (128, 16, 40, 16, 4), (256, 64, 30, 4, 2)])
def test_a_unit_in_many_shares(d, page, N, H, Hkv):
    run("bf16", d, page, H, Hkv, N, [20000, 300], layout=False)


def test_more_sequences_than_a_block_has_threads():
    for N in (1, 70):
        run("bf16", 64, 16, 1, 1, N, [N + b % 7 for b in range(300)], seed=N)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N,H", [(4, 4), (6, 1), (70, 2), (150, 1)])
def test_nan_in_masked_places_reaches_only_the_rows_that_see_it(d, N, H):
    g = torch.Generator().manual_seed(d + N)
    L, page = N + 150, 16
    width = -(-L // page) + 1
    codes, scales, table = ref.make_cache(width + 1, 1, page, d, 1, width, g)
    sees = random_mask(N, g, "any")
    hidden, shown = N // 2, N - 1
    sees[:, hidden] = False                       # a draft that no row sees, all NaN
    sees[:, shown] = torch.arange(N) % 3 == 0     # one with a NaN that some rows see
    for which in (0, 1):
        x = codes[which].view(torch.uint8)
        for t, cols in ((L - N + hidden, slice(None)), (L, slice(None))):     # (and behind the sequence)
            x[int(table[0, t // page]), 0, t % page, cols] = 0x7F
    t = L - N + shown
    codes[1].view(torch.uint8)[int(table[0, t // page]), 0, t % page, 3] = 0xFF
    q = torch.randn(1, H, N, d, generator=g).bfloat16()
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    mask = branch.pack(sees, N)[None].to(DEV)
    o, lse = binding.forward_cache_tree(q.to(DEV), cache, ints([L]), mask, 0.1)
    binding.device_status()
    V = ref.Paged(codes[1], scales[1])
    mine = o.cpu()[..., 3].isnan()
    assert torch.equal(mine, sees[:, shown].expand(1, H, N))
    V.values[int(table[0, t // page]), 0, t % page, 3] = 0.0
    o = o.clone()
    o[..., 3] = 0
    want = branch.attend_tree(q, ref.Paged(codes[0], scales[0]), V, table, [L], [sees], 0.1)
    want[0][..., 3] = 0
    err = (o.cpu().double() - want[0]).abs()
    assert (err <= ref.half_step(o.dtype) * want[0].abs() * 1.001 + 2.0 ** -25 + want[2]).all()
    assert ((lse.cpu().double() - want[1]).abs() <= want[3] + 2.0 ** -23 * want[1].abs()).all()


@pytest.mark.parametrize("d,H", [(64, 2), (128, 2), (256, 1)])
@pytest.mark.parametrize("N", [4, 80])
def test_lengths_and_pages_out_of_range_are_reported(d, H, N):
    g = torch.Generator().manual_seed(1)
    codes, scales, table = ref.make_cache(40, 1, 64, d, 4, 8, g)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    q = torch.randn(4, H, N, d, generator=g).half().to(DEV)
    mask = binding.tree_mask([[-1] * N]).to(DEV)
    good = [300, 290, 200, N]
    want, l_want = binding.forward_cache_tree(q, cache, ints(good), mask, 0.1)
    binding.device_status()
    # fewer tokens than drafts; more than the table has; below zero; drafts out of range
    for b, lens, new in ((0, N - 1, N), (1, 513, N), (2, -1, N), (3, 300, N + 1), (1, 300, -1)):
        now, news = list(good), [N] * 4
        now[b], news[b] = lens, new
        o, lse = binding.forward_cache_tree(q, cache, ints(now), mask, 0.1, new_lens=ints(news))
        assert binding.fa_get_device_status() == binding.FA_ERR_CACHE
        assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
        for i in range(4):
            if i != b:
                assert (o[i] - want[i]).abs().max() <= 2.0 ** -9 * want[i].abs().max()
    cache.tensors[4][1, 2] = 40
    o, _ = binding.forward_cache_tree(q, cache, ints(good), mask, 0.1)
    assert binding.fa_get_device_status() == binding.FA_ERR_CACHE
    assert (o[0] - want[0]).abs().max() <= 2.0 ** -9 * want[0].abs().max()


@pytest.mark.parametrize("N", [3, 60])
def test_graphs_that_run_together_and_the_same_bits(N):
    g = torch.Generator().manual_seed(2)
    lens = [3000, 2500]
    codes, scales, table = ref.make_cache(400, 2, 16, 128, 2, 190, g, lens)
    cache = binding.Cache(*(t.to(DEV) for t in (*codes, *scales, table)))
    n, runs = ints(lens), []
    for i in range(2):
        q = torch.randn(2, 8, N + i, 128, generator=g).bfloat16().to(DEV)
        mask = torch.stack([branch.pack(random_mask(N + i, g, "tree"), N + i) for _ in range(2)]).to(DEV)
        want = binding.forward_cache_tree(q, cache, n, mask, 0.1)
        ws = torch.full((binding.fwd_cache_tree_workspace_size(2, 8, 2, N + i, 128),), 0xFF, dtype=torch.uint8, device=DEV)
        for x, y in zip(binding.forward_cache_tree(q, cache, n, mask, 0.1, workspace=ws), want):
            assert torch.equal(x, y)
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = binding.forward_cache_tree(q, cache, n, mask, 0.1)
        runs.append((graph, s, out, want, q, mask))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s, *_rest in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _graph, _s, out, want, *_rest in runs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", [3, 30, 200])
def test_a_batch_without_tokens(d, N):
    run("bf16", d, 64, 4, 2, N, [0, 70, 0], new=[0, 0, 0])
    run("bf16", d, 64, 4, 2, N, [0, N, 0], new=[0, N, 0], kind="any")


def test_refusals_of_the_binding():
    c = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    s = torch.ones(4, 2, device=DEV)
    cache = binding.Cache(c, c.clone(), s, s.clone(), torch.zeros(2, 2, dtype=torch.int32, device=DEV))
    q = torch.zeros(2, 2, 40, 64, dtype=torch.float16, device=DEV)
    good = torch.zeros(2, 40, 2, dtype=torch.int32, device=DEV)
    for bad in (good.long(), good[:, :39], good[:, :, :1], good[0], good.cpu(), good.repeat(2, 1, 1),
                good.transpose(1, 2)):
        with pytest.raises(ValueError):
            binding.forward_cache_tree(q, cache, ints([40, 40]), bad, 0.1)
