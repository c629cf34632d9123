"""fa_cache_fork against its definition: tables, counts, lengths, copies, what is
left as it was, lack of pages and numbers out of range, graphs; and a branching
decode of all the operators together."""
import math

import pytest
import torch

import branch_ref as branch
import cache_ref as ref
from exact_io_aware_20_gb300 import binding
from test_cache_tree_gpu import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """Random pages, sequences over them, and their twins on the CPU."""

    def __init__(self, d, page, Hkv, pages, B, width, seed=0):
        self.g = torch.Generator().manual_seed(seed + d + page)
        self.page, self.pages = page, pages
        self.codes = [torch.randint(0, 256, (pages, Hkv, page, d), generator=self.g, dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.rand(pages, Hkv, generator=self.g) + 0.5 for _ in range(2)]
        self.table = [[-1] * width for _ in range(B)]
        self.refs = [0] * pages
        self.lens = [0] * B
        self.upload()

    def upload(self):
        self.cache = binding.Cache(*(t.to(DEV) for t in (*self.codes, *self.scales)), ints(self.table))
        self.d_refs, self.d_lens = ints(self.refs), ints(self.lens)

    def fork(self, parents, reserve=None, status=binding.FA_OK, **kw):
        out = binding.cache_fork(self.cache, self.d_refs, ints(parents), self.d_lens,
                                 reserve_lens=None if reserve is None else ints(reserve), out_lens=self.d_lens, **kw)
        assert out.data_ptr() == self.d_lens.data_ptr()
        assert binding.fa_get_device_status() == status
        self.table, self.refs, self.lens, copies = branch.fork(self.table, self.refs, parents, self.lens, reserve, self.page)
        for src, dst, rows in copies:
            for i in (0, 1):
                self.codes[i][dst, :, :rows] = self.codes[i][src, :, :rows]
                self.scales[i][dst] = self.scales[i][src]
        self.check()
        return copies

    def check(self):
        assert self.d_lens.tolist() == self.lens
        assert self.cache.tensors[4].tolist() == self.table
        assert self.d_refs.tolist() == self.refs
        for i in (0, 1):
            assert torch.equal(self.cache.tensors[i].cpu().view(torch.uint8), self.codes[i])
            assert torch.equal(self.cache.tensors[2 + i].cpu(), self.scales[i])

    def grow(self, lens):
        """Tokens are there now, in the pages held."""
        self.lens = list(lens)
        self.d_lens.copy_(ints(lens))


@pytest.mark.parametrize("d,page,Hkv", [(64, 16, 1), (128, 64, 3), (256, 256, 2), (128, 128, 8), (64, 32, 5)])
def test_a_life_of_beams(d, page, Hkv):
    """Begin, fork, reorder, end, begin again, with random parents; whole pages and part-full ones."""
    B, width = 9, 7
    s = Server(d, page, Hkv, 140, B, width)
    s.fork([-1] * B, [3 * page, 0, 2 * page + 1, 5, 0, 0, 0, page, 0])          # nobody is there yet: they begin
    s.grow([2 * page + 3, 0, 2 * page, 5, 0, 0, 0, page, 0])
    assert s.fork([0, 0, 0, 3, 3, 2, 2, 7, 7], [2 * page + 4] * 9)
    for step in range(12):
        parents = torch.randint(-1, B, (B,), generator=s.g).tolist()
        lens = [s.lens[p] if p >= 0 else 0 for p in parents]
        more = torch.randint(0, page + 2, (B,), generator=s.g).tolist()
        want = [min(width * page, n + m) for n, m in zip(lens, more)]
        s.fork(parents, want)
        s.grow([max(n, w - 1) for n, w in zip(s.lens, want)])
        assert sum(s.refs) == sum(p >= 0 for row in s.table for p in row)
    s.fork([-1] * B)
    assert set(s.refs) == {0} and all(p == -1 for row in s.table for p in row)


def test_pages_that_others_count_are_never_kept_for_writing():
    s = Server(64, 16, 2, 40, 3, 4)
    s.fork([-1, -1, -1], [40, 20, 0])
    s.grow([40, 20, 0])
    s.refs[s.table[0][2]] += 1          # the part-full page is somebody's prefix too
    s.d_refs.copy_(ints(s.refs))
    held = s.table[0][2]
    copies = s.fork([0, 1, 1], [41, 21, 21])
    assert (held, s.table[0][2], 8) in copies and s.refs[held] == 1
    assert len(copies) == 2 and s.table[1][1] != s.table[2][1] and s.table[1][0] == s.table[2][0]


def test_the_identity_changes_nothing():
    s = Server(128, 32, 2, 30, 3, 5)
    s.fork([-1] * 3, [100, 33, 0])
    s.grow([97, 32, 0])
    before = [list(r) for r in s.table]
    s.fork([0, 1, 2], [100, 33, 0])
    assert s.table == before
    s.fork([0, 1, 2])                    # without a reserve the places behind the tokens are given back
    assert s.table[1][1] == -1 and s.table[0][3] == before[0][3]
    # a swap moves rows, no bytes
    assert s.fork([1, 0, 2]) == [] and s.table[0][0] == before[1][0]


def test_a_table_of_its_own_for_the_result():
    s = Server(64, 16, 1, 20, 2, 3)
    s.fork([-1, -1], [20, 16])
    s.grow([20, 16])
    old = [list(r) for r in s.table]
    to = torch.full((2, 3), 7, dtype=torch.int32, device=DEV)
    out = binding.cache_fork(s.cache, s.d_refs, ints([0, 0]), s.d_lens, block_table=to)
    binding.device_status()
    table, refs, lens, copies = branch.fork(s.table, s.refs, [0, 0], s.lens, None, 16)
    assert to.tolist() == table and s.d_refs.tolist() == refs and out.tolist() == lens and len(copies) == 1
    assert s.cache.tensors[4].tolist() == old and s.d_lens.tolist() == s.lens


@pytest.mark.parametrize("pages,B,width", [(70000, 40, 60), (8192, 3, 700), (8193, 300, 9), (100000, 2, 30000)])
def test_many_pages_and_sequences(pages, B, width):
    """Free pages in several chunks of the search, many of them for one sequence, few free ones far apart."""
    page = 16
    s = Server(64, page, 1, pages, B, width)
    taken = torch.rand(pages, generator=s.g) < 0.8
    s.refs = taken.int().tolist()
    s.d_refs.copy_(ints(s.refs))
    total = pages - int(taken.sum())
    each = min(width, total // B) * page
    s.fork([-1] * B, [each - 5 - b % 7 for b in range(B)])
    s.grow([each - 21 - b % 7 for b in range(B)])
    parents = [b // 2 for b in range(B)]
    lack = branch.fork(s.table, s.refs, parents, s.lens, [t + 3 for t in s.lens], page)
    lacks = any(-1 in row[:-(-(n + 3) // page)] for row, n in zip(lack[0], lack[2]))
    s.fork(parents, [s.lens[p] + 3 for p in parents], status=binding.FA_ERR_CACHE if lacks else binding.FA_OK)


def test_a_lack_of_pages_is_reported():
    s = Server(64, 16, 1, 6, 3, 4)
    s.fork([-1] * 3, [40, 33, 20], status=binding.FA_ERR_CACHE)        # 3 + 3 + 2 of 6
    assert s.table[2] == [-1] * 4 and s.refs == [1] * 6
    s.fork([0, -1, 0], None)
    assert 0 in s.refs


def test_numbers_out_of_range_are_reported():
    for parents, lens, reserve in (([0, 5], [20, 20], None), ([0, -2], [20, 20], None), ([0, 1], [20, 65], None),
                                   ([1, 0], [20, -1], None), ([0, 1], [20, 20], [30, 65])):
        s = Server(64, 16, 1, 30, 2, 4)
        s.fork([-1, -1], [30, 30])
        s.grow(lens)
        s.fork(parents, reserve, status=binding.FA_ERR_CACHE)
    # a parent's page that is not there: the full one's place stays empty, the part-full one's page is not copied
    for at, L in ((0, 20), (1, 20)):
        s = Server(64, 16, 1, 30, 2, 4)
        s.fork([-1, -1], [30, 30])
        s.grow([L, 30])
        s.table[0][at] = 30
        s.cache.tensors[4][0, at] = 30
        s.fork([0, 0], [30, 30], status=binding.FA_ERR_CACHE)


def test_on_streams_and_in_a_graph():
    s = Server(64, 16, 2, 60, 4, 5)
    s.fork([-1] * 4, [40, 20, 0, 3])
    s.grow([39, 20, 0, 3])
    parents, reserve = ints([0, 1, 2, 3]), ints([0] * 4)
    ws = torch.full((binding.cache_fork_workspace_size(4, 60, 5),), 0xFF, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        binding.cache_fork(s.cache, s.d_refs, parents, s.d_lens, reserve_lens=reserve, out_lens=s.d_lens, workspace=ws)
    for p, r in (([0, 0, 1, 3], [41, 41, 30, 9]), ([1, 0, 1, 0], [50, 50, 50, 50]), ([-1, 1, 2, 2], [3, 60, 60, 60])):
        parents.copy_(ints(p)), reserve.copy_(ints(r))
        graph.replay()
        binding.device_status()
        s.table, s.refs, s.lens, copies = branch.fork(s.table, s.refs, p, s.lens, r, 16)
        for src, dst, rows in copies:
            for i in (0, 1):
                s.codes[i][dst, :, :rows] = s.codes[i][src, :, :rows]
                s.scales[i][dst] = s.scales[i][src]
        s.check()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.fork([0, 1, 1, 3], [5, 60, 60, 60], stream=side)


def test_pages_far_apart():
    """Byte offsets past 32 bits, heads and rows inside a wider buffer."""
    d, page, Hkv, pages, apart = 64, 16, 2, 9, 1 << 29
    g = torch.Generator().manual_seed(8)
    codes = [torch.randint(0, 256, (pages, Hkv, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand(pages, Hkv, generator=g) + 0.5 for _ in range(2)]
    wide = torch.zeros(apart * (pages - 1) + 4 * Hkv * page * d, dtype=torch.uint8, device=DEV)
    views = []
    for i in (0, 1):
        v = torch.as_strided(wide, (pages, Hkv, page, d), (apart, 2 * page * d, 2 * d, 1), i * d)
        v.copy_(codes[i])
        views.append(v)
    table = [[7, 8, -1], [-1, -1, -1], [3, -1, -1]]
    refs, lens, parents = [0, 1, 0, 1, 2, 2, 2, 1, 1], [27, 0, 16], [0, 0, 2]
    cache = binding.Cache(*views, *(s.to(DEV) for s in scales), ints(table))
    d_refs = ints(refs)
    out = binding.cache_fork(cache, d_refs, ints(parents), ints(lens))
    binding.device_status()
    new, now, length, copies = branch.fork(table, refs, parents, lens, None, page)
    assert out.tolist() == length and cache.tensors[4].tolist() == new and d_refs.tolist() == now
    assert copies == [(8, 0, 11)]
    for src, dst, rows in copies:
        for i in (0, 1):
            codes[i][dst, :, :rows], scales[i][dst] = codes[i][src, :, :rows], scales[i][src]
    for i in (0, 1):
        assert torch.equal(views[i].cpu(), codes[i]) and torch.equal(cache.tensors[2 + i].cpu(), scales[i])


def test_refusals_of_the_binding():
    s = Server(64, 16, 1, 20, 2, 3)
    p, n = ints([0, 1]), ints([0, 0])
    for bad in (dict(refs=s.d_refs[:5]), dict(refs=s.d_refs.long()), dict(parents=p[:1]), dict(seq_lens=n.cpu()),
                dict(reserve_lens=n.float()), dict(out_lens=n[:1]), dict(block_table=s.cache.tensors[4][:, :2])):
        a = {"refs": s.d_refs, "parents": p, "seq_lens": n, **bad}
        with pytest.raises(ValueError):
            binding.cache_fork(s.cache, **a)
    with pytest.raises(binding.FaError):
        binding.cache_fork(s.cache, s.d_refs, p, n, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)[:64])


@pytest.mark.parametrize("d,page,H,Hkv", [(64, 16, 4, 2), (128, 64, 8, 2), (256, 32, 2, 1)])
def test_a_branching_decode(d, page, H, Hkv):
    """Prompts, then steps of drafts: pages reserved and sequences forked, q and k
    normed and turned, appended, the tree attended, a branch kept; against 64
    bits over what the cache holds, and against a cache in which the accepted
    tokens came one after another."""
    g = torch.Generator().manual_seed(11)
    B, N, steps, scale = 4, 13, 4, d ** -0.5
    width = -(-(40 + 12 * steps + N) // page) + 1
    pages = 3 * B * width
    codes = [torch.zeros(pages, Hkv, page, d, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    scales = [torch.ones(pages, Hkv, device=DEV) for _ in range(2)]
    cache = binding.Cache(*codes, *scales, torch.full((B, width), -1, dtype=torch.int32, device=DEV))
    refs, lens = torch.zeros(pages, dtype=torch.int32, device=DEV), ints([0] * B)
    rope = binding.Rope([10000.0 ** (-i / (d // 2)) for i in range(d // 2)])
    w = [torch.rand(d, generator=g).add(0.5).bfloat16().to(DEV) for _ in range(2)]

    def tokens(n):
        return [torch.randn(B, n, h, d, generator=g).bfloat16().to(DEV).transpose(1, 2) for h in (H, Hkv, Hkv)]

    # prompts of two sequences
    q, k, v = tokens(40)
    new = [40, 17, 0, 0]
    binding.cache_fork(cache, refs, ints([-1] * B), lens, reserve_lens=ints(new), out_lens=lens)
    lens.add_(ints(new))
    q, k = binding.qk_norm_rope(q, k, *w, 1e-6, None, rope)
    q = binding.cache_append(cache, q, k, v, lens, new_lens=ints(new))
    binding.forward_cache(q, cache, lens, True, scale, new_lens=ints(new))
    # each becomes two
    binding.cache_fork(cache, refs, ints([0, 0, 1, 1]), lens, reserve_lens=ints([41, 41, 18, 18]), out_lens=lens)
    binding.device_status()
    now = [40, 40, 17, 17]
    assert lens.tolist() == now
    rows = [cache.tensors[4][b].tolist() for b in range(B)]
    held = [ref.Paged(cache.tensors[i], cache.tensors[2 + i]) for i in (0, 1)]
    for a, b in ((0, 1), (2, 3)):
        assert rows[a][now[a] // page] != rows[b][now[a] // page]
        for c in held:
            for h in range(Hkv):
                assert torch.equal(c.rows(rows[a], now[a], h), c.rows(rows[b], now[b], h))
    for step in range(steps):
        parents = [[0, 1, 2, 3], [1, 1, 3, 2], [0, 0, 0, 3], [3, 2, 1, 0]][step]
        now = [now[p] for p in parents]
        binding.cache_fork(cache, refs, ints(parents), lens, reserve_lens=ints([t + N for t in now]), out_lens=lens)
        trees = [branch.random_tree(N, g) for _ in range(B)]
        depth = [[0] * N for _ in range(B)]
        for b in range(B):
            for i, p in enumerate(trees[b]):
                depth[b][i] = depth[b][p] + 1 if p >= 0 else 0
        pos = ints([[now[b] + x for x in depth[b]] for b in range(B)])
        q, k, v = tokens(N)
        lens.add_(N)
        qn, kn = binding.qk_norm_rope(q, k, *w, 1e-6, pos, rope)
        qn = binding.cache_append(cache, qn, kn, v, lens)
        o, lse = binding.forward_cache_tree(qn, cache, lens, binding.tree_mask(trees).to(DEV), scale)
        binding.device_status()
        assert lens.tolist() == [t + N for t in now]
        table = cache.tensors[4].cpu()
        K, V = (ref.Paged(cache.tensors[i], cache.tensors[2 + i]) for i in (0, 1))
        check(o, lse, qn.cpu(), K, V, table, lens.tolist(), [branch.sees_of(t) for t in trees], scale)
        # the branch of one draft of each sequence is accepted
        path = []
        for b in range(B):
            i, way = (step * 5 + 3 * b) % N, []
            while i >= 0:
                way.insert(0, i)
                i = trees[b][i]
            path.append(way)
        most = max(map(len, path))
        before = [[c.rows(table[b], now[b] + N, h) for c in (K, V) for h in range(Hkv)] for b in range(B)]
        out = binding.cache_keep(cache, lens, N, ints([w + [-1] * (most - len(w)) for w in path]),
                                 keep_lens=ints([len(w) for w in path]))
        lens.copy_(out)
        binding.device_status()
        now = [t + len(way) for t, way in zip(now, path)]
        assert lens.tolist() == now
        K, V = (ref.Paged(cache.tensors[i], cache.tensors[2 + i]) for i in (0, 1))
        for b in range(B):
            at = list(range(now[b] - len(path[b]))) + [now[b] - len(path[b]) + i for i in path[b]]
            for i, c in enumerate((K, V)):
                for h in range(Hkv):
                    want, got = before[b][i * Hkv + h][at], c.rows(table[b], now[b], h)
                    s = max(float(c.scales[int(p), h]) for p in table[b][:-(-now[b] // page)])
                    # the same values, or rounded once more as subnormals of a larger scale
                    assert ((got - want).abs() <= s * 2.0 ** -10).all()
        # the last accepted token's row saw what a causal row sees now
        last = torch.stack([qn[b, :, w[-1]] for b, w in enumerate(path)])[:, :, None].contiguous()
        again, _ = binding.forward_cache(last, cache, lens, True, scale)
        for b in range(B):
            was = o[b, :, path[b][-1]].float()
            assert (again[b, :, 0].float() - was).abs().max() <= 0.02 * was.abs().max()
    total = sum(int(p) >= 0 for p in cache.tensors[4].flatten().tolist())
    assert int(refs.sum()) == total and math.isfinite(float(o.float().sum()))
