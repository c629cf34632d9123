"""Host-side checks of the entry points of a branching decode and of the norms:
bad arguments are refused before anything touches a device."""
import ctypes

import pytest
import torch

import branch_ref as branch
from exact_io_aware_20_gb300 import binding
from test_cache_abi import BAD, BAD_CACHES, FAKE, UNSUP, WORK, bad_axis, bad_freq, cache, lib, spec, strides  # noqa: F401

OK4 = [(64, 64, 64)] * 4


def c_of(x):
    return None if x is None else ctypes.byref(x)


def tree(lib, **kw):
    a = dict(q=FAKE, cache=cache(), o=FAKE, lse=FAKE, B=2, H=4, Nq=9, scale=0.1, dtype=1, lens=FAKE, new=None,
             mask=FAKE, mask_batch=2, strides=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.fa_fwd_cache_tree(a["q"], c_of(a["cache"]), a["o"], a["lse"], a["B"], a["H"], a["Nq"], a["scale"],
                                 a["dtype"], a["lens"], a["new"], a["mask"], a["mask_batch"], a["strides"], a["ws"],
                                 a["ws_bytes"], None)


def keep(lib, **kw):
    a = dict(cache=cache(), B=2, N=9, K=4, lens=FAKE, new=None, keep=FAKE + 64, keep_lens=None, out=FAKE + 128)
    a.update(kw)
    return lib.fa_cache_keep(c_of(a["cache"]), a["B"], a["N"], a["K"], a["lens"], a["new"], a["keep"], a["keep_lens"],
                             a["out"], None)


def fork(lib, **kw):
    a = dict(cache=cache(), table=FAKE, refs=FAKE, B=2, parents=FAKE, lens=FAKE, reserve=None, out=FAKE, ws=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    return lib.fa_cache_fork(c_of(a["cache"]), a["table"], a["refs"], a["B"], a["parents"], a["lens"], a["reserve"],
                             a["out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("case,expect", BAD_CACHES)
def test_bad_caches_are_refused(lib, case, expect):  # noqa: F811
    for call in (tree, keep, fork):
        assert call(lib, cache=cache(**case)) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(cache=None), BAD), (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(lens=None), BAD),
    (dict(H=3), BAD), (dict(scale=0.0), BAD), (dict(scale=float("inf")), BAD), (dict(B=0), BAD), (dict(Nq=0), BAD),
    (dict(dtype=-1), UNSUP), (dict(q=FAKE + 8), BAD), (dict(new=FAKE + 1), BAD), (dict(mask=None), BAD),
    (dict(mask=FAKE + 2), BAD), (dict(mask_batch=0), BAD), (dict(mask_batch=3), BAD), (dict(ws=None), WORK),
    (dict(ws=FAKE + 16), WORK), (dict(strides=strides((8, 8, 8), (0, 8, 8))), BAD),
])
def test_tree_rejects(lib, case, expect):  # noqa: F811
    assert tree(lib, **case) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(cache=None), BAD), (dict(B=0), BAD), (dict(B=65536), BAD), (dict(N=0), BAD), (dict(K=0), BAD),
    (dict(K=10), BAD), (dict(lens=None), BAD), (dict(lens=FAKE + 2), BAD), (dict(new=FAKE + 3), BAD),
    (dict(keep=None), BAD), (dict(keep=FAKE + 1), BAD), (dict(keep_lens=FAKE + 2), BAD), (dict(out=None), BAD),
    (dict(out=FAKE + 2), BAD), (dict(out=FAKE), BAD), (dict(new=FAKE + 128), BAD), (dict(keep_lens=FAKE + 128), BAD),
    (dict(out=FAKE + 64), BAD), (dict(B=2, N=1 << 30, K=1 << 30), BAD),
])
def test_keep_rejects(lib, case, expect):  # noqa: F811
    assert keep(lib, **case) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(cache=None), BAD), (dict(table=None), BAD), (dict(refs=None), BAD), (dict(parents=None), BAD),
    (dict(lens=None), BAD), (dict(out=None), BAD), (dict(B=0), BAD), (dict(B=65536), BAD), (dict(table=FAKE + 2), BAD),
    (dict(refs=FAKE + 2), BAD), (dict(parents=FAKE + 1), BAD), (dict(reserve=FAKE + 1), BAD), (dict(ws=None), WORK),
    (dict(ws=FAKE + 16), WORK), (dict(ws_bytes=1023), WORK),
    (dict(B=65535, cache=cache(table_width=40000, page_size=16)), BAD),
])
def test_fork_rejects(lib, case, expect):  # noqa: F811
    assert fork(lib, **case) == expect


@pytest.mark.parametrize("case", [
    dict(out=FAKE + 4), dict(out=FAKE + 64 + 28), dict(out=FAKE + 60), dict(out=FAKE - 4), dict(new=FAKE + 132),
    dict(keep_lens=FAKE + 124),
])
def test_keep_refuses_outputs_that_overlap_inputs(lib, case):  # noqa: F811
    assert keep(lib, **case) == BAD


@pytest.mark.parametrize("at", [4, -4, 4 * (2 * 8 - 1), -4 * (2 * 8 - 1)])
def test_fork_refuses_tables_that_overlap(lib, at):  # noqa: F811
    c = cache(table_width=8)
    assert fork(lib, cache=c, table=c.block_table + at) == BAD


def norm(lib, back, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, dqo=FAKE, dko=FAKE, wq=FAKE, wk=FAKE, f32=0, eps=1e-6, offset=0.0, B=2,
             H=4, Hkv=2, N=8, d=64, dtype=1, spec=spec(), pos=FAKE, pos_batch=2, strides=None, dwq=FAKE, dwk=FAKE,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    tail = [a[n] for n in ("B", "H", "Hkv", "N", "d", "dtype")] + [c_of(a["spec"]), a["pos"], a["pos_batch"]]
    if back:
        return lib.fa_qk_norm_rope_bwd(a["dqo"], a["dko"], a["q"], a["k"], a["qo"], a["ko"], a["wq"], a["wk"], a["f32"],
                                       a["eps"], a["offset"], a["dwq"], a["dwk"], *tail, a["strides"], a["ws"],
                                       a["ws_bytes"], None)
    return lib.fa_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["wq"], a["wk"], a["f32"], a["eps"], a["offset"],
                               *tail, a["strides"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("case,expect", [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(N=0), BAD), (dict(Hkv=0), BAD), (dict(H=65536), BAD), (dict(d=96), UNSUP),
    (dict(dtype=2), UNSUP), (dict(q=None), BAD), (dict(qo=None), BAD), (dict(k=None), BAD), (dict(ko=None), BAD),
    (dict(k=None, ko=None), BAD), (dict(q=FAKE + 8), BAD), (dict(ko=FAKE + 2), BAD), (dict(wq=FAKE + 8), BAD),
    (dict(wk=FAKE + 4), BAD), (dict(f32=2), BAD), (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(eps=2.0 ** -101), BAD),
    (dict(offset=float("inf")), BAD), (dict(spec=spec(pairs=40)), BAD), (dict(spec=bad_freq()), BAD),
    (dict(spec=bad_axis()), BAD), (dict(pos_batch=3), BAD), (dict(pos=FAKE + 2), BAD),
    (dict(strides=strides((64, 64, 0), *[(64, 64, 64)] * 5)), BAD),
    (dict(strides=strides((64, 64, 64), (64, 12, 64), *[(64, 64, 64)] * 4)), BAD),
])
def test_norm_rejects(lib, back, case, expect):  # noqa: F811
    assert norm(lib, back, **case) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(dqo=None), BAD), (dict(dko=None), BAD), (dict(dqo=FAKE + 8), BAD), (dict(dwq=FAKE + 2), BAD),
    (dict(wq=None), BAD), (dict(wk=None), BAD), (dict(ws=None), WORK), (dict(ws=FAKE + 16), WORK),
    (dict(strides=strides(*OK4, (64, 64, 64), (64, 64, 4))), BAD),
])
def test_norm_backward_rejects(lib, case, expect):  # noqa: F811
    assert norm(lib, True, **case) == expect


def test_workspace_sizes_of_invalid_sizes(lib):  # noqa: F811
    for args in ((0, 9, 4), (2, 0, 4), (2, 9, 0), (65536, 9, 4), (65535, 9, 40000)):
        assert lib.fa_cache_fork_workspace_size(*args) == 0
    assert lib.fa_cache_fork_workspace_size(2, 9, 4) > 0
    for args in ((0, 4, 2, 1, 128), (1, 4, 3, 1, 128), (1, 4, 0, 1, 128), (1, 4, 2, 0, 128), (1, 4, 2, 1, 96)):
        assert lib.fa_fwd_cache_tree_workspace_size(*args) == 0
    for args in ((0, 4, 2, 8, 64), (1, 0, 2, 8, 64), (1, 4, -1, 8, 64), (1, 4, 2, 0, 64), (1, 4, 2, 8, 80)):
        assert lib.fa_qk_norm_rope_bwd_workspace_size(*args) == 0
    assert lib.fa_qk_norm_rope_bwd_workspace_size(1, 4, 0, 8, 64) > 0


def test_tree_masks():
    g = torch.Generator().manual_seed(1)
    trees = [branch.random_tree(n, g) for n in (1, 40, 33, 70)]
    mask = binding.tree_mask(trees)
    assert mask.shape == (4, 70, 3) and mask.dtype == torch.int32
    for b, t in enumerate(trees):
        assert torch.equal(mask[b], branch.pack(branch.sees_of(t), 70))
    assert binding.tree_mask([[-1] * 32])[0, 31, 0] == -2 ** 31
    for bad in ([[0]], [[-1, 1]], [[-2]], [[]], []):
        with pytest.raises(ValueError):
            binding.tree_mask(bad)


def test_the_binding_checks_what_it_marshals():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # not on a GPU
        binding.qk_norm_rope(q, None, w, None, 1e-6)
    with pytest.raises(ValueError):
        binding.qk_norm_rope_backward(q, None, q, None, w, None, 1e-6)
