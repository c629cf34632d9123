"""Host-side checks of the rotary and cache entry points: bad arguments are
refused before anything touches a device."""
import ctypes

import pytest
import torch

from exact_io_aware_20_gb300 import binding

FAKE = 1 << 20   # never dereferenced: every case below fails validation first
BAD, UNSUP, WORK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(binding.LIB_PATH):
        from exact_io_aware_20_gb300 import build
        build.build()
    return binding.load()


def strides(*vals):
    arr = (binding.FaStrides * len(vals))()
    for i, v in enumerate(vals):
        arr[i] = binding.FaStrides(*v)
    return arr


def spec(**kw):
    s = binding.Rope([0.5] * 16).spec
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def bad_freq():
    s = spec()
    s.freq[3] = float("nan")
    return s


def bad_axis():
    s = spec()
    s.axis[2] = 1
    return s


@pytest.mark.parametrize("case,expect", [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(N=0), BAD), (dict(Hkv=0), BAD), (dict(H=65536), BAD),
    (dict(N=1 << 26), BAD), (dict(d=96), UNSUP), (dict(dtype=2), UNSUP), (dict(q=None), BAD),
    (dict(q_out=None), BAD), (dict(k=None), BAD), (dict(k_out=None), BAD), (dict(q=FAKE + 8), BAD),
    (dict(k_out=FAKE + 2), BAD), (dict(spec=None), BAD), (dict(spec=spec(axes=0)), BAD),
    (dict(spec=spec(axes=5)), BAD), (dict(spec=spec(pairs=12)), BAD), (dict(spec=spec(pairs=0)), BAD),
    (dict(spec=spec(pairs=40)), BAD), (dict(spec=spec(interleaved=2)), BAD),
    (dict(spec=bad_freq()), BAD), (dict(spec=bad_axis()), BAD), (dict(pos_batch=3), BAD),
    (dict(pos=FAKE + 2), BAD), (dict(inverse=2), BAD),
    (dict(strides=strides((64, 64, 0), (64, 64, 64), (64, 64, 64), (64, 64, 64))), BAD),
    (dict(strides=strides((64, 64, 64), (64, 12, 64), (64, 64, 64), (64, 64, 64))), BAD),
])
def test_rope_rejects(lib, case, expect):
    a = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, B=2, H=4, Hkv=2, N=8, d=64, dtype=1, spec=spec(),
             pos=FAKE, pos_batch=2, inverse=0, strides=None)
    a.update(case)
    s = None if a["spec"] is None else ctypes.byref(a["spec"])
    assert lib.fa_rope(a["q"], a["k"], a["q_out"], a["k_out"], a["B"], a["H"], a["Hkv"], a["N"], a["d"],
                       a["dtype"], s, a["pos"], a["pos_batch"], a["inverse"], a["strides"],
                       None) == expect


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, pages=9, page_size=64,
             table_width=4, Hkv=2, d=128, k_strides=binding.FaStrides(0, 0, 0),
             v_strides=binding.FaStrides(0, 0, 0))
    a.update(kw)
    return binding._FaCache(*a.values())


BAD_CACHES = [(dict(k=None), BAD), (dict(v_scale=None), BAD), (dict(block_table=None), BAD),
              (dict(k=FAKE + 8), BAD), (dict(block_table=FAKE + 1), BAD), (dict(pages=0), BAD),
              (dict(table_width=0), BAD), (dict(page_size=48), UNSUP), (dict(page_size=8), UNSUP),
              (dict(page_size=512), UNSUP), (dict(d=80), UNSUP), (dict(Hkv=0), BAD),
              (dict(table_width=1 << 26), BAD),
              (dict(k_strides=binding.FaStrides(8192, 64, 24)), BAD),
              (dict(v_strides=binding.FaStrides(8192, 0, 128)), BAD)]


def append(lib, **kw):
    a = dict(cache=cache(), q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, B=2, H=4, N=3, dtype=1, lens=FAKE,
             new=None, spec=spec(), pos=FAKE, pos_batch=1, strides=None)
    a.update(kw)
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    s = None if a["spec"] is None else ctypes.byref(a["spec"])
    return lib.fa_cache_append(c, a["q"], a["k"], a["v"], a["q_out"], a["B"], a["H"], a["N"], a["dtype"],
                               a["lens"], a["new"], s, a["pos"], a["pos_batch"], a["strides"], None)


def attend(lib, **kw):
    a = dict(q=FAKE, cache=cache(), o=FAKE, lse=FAKE, B=2, H=4, Nq=1, causal=1, scale=0.1, dtype=1,
             lens=FAKE, new=None, strides=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    return lib.fa_fwd_cache(a["q"], c, a["o"], a["lse"], a["B"], a["H"], a["Nq"], a["causal"], a["scale"],
                            a["dtype"], a["lens"], a["new"], a["strides"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("case,expect", BAD_CACHES)
def test_bad_caches_are_refused(lib, case, expect):
    assert append(lib, cache=cache(**case)) == expect
    assert attend(lib, cache=cache(**case)) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(cache=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(q_out=None), BAD),
    (dict(q=None), BAD), (dict(lens=None), BAD), (dict(lens=FAKE + 2), BAD), (dict(new=FAKE + 2), BAD),
    (dict(B=0), BAD), (dict(N=0), BAD), (dict(H=0), BAD), (dict(dtype=5), UNSUP), (dict(k=FAKE + 8), BAD),
    (dict(spec=spec(pairs=72)), BAD), (dict(pos_batch=5), BAD),
    (dict(strides=strides((8, 8, 8), (8, 8, 8), (8, 8, 4), (8, 8, 8))), BAD),
])
def test_append_rejects(lib, case, expect):
    assert append(lib, **case) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(cache=None), BAD), (dict(q=None), BAD), (dict(o=None), BAD), (dict(lse=None), BAD),
    (dict(lens=None), BAD), (dict(H=3), BAD), (dict(causal=2), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(B=65536), BAD), (dict(Nq=0), BAD), (dict(dtype=-1), UNSUP),
    (dict(q=FAKE + 8), BAD), (dict(lse=FAKE + 2), BAD), (dict(new=FAKE + 1), BAD), (dict(ws=None), WORK),
    (dict(ws=FAKE + 16), WORK), (dict(strides=strides((8, 8, 8), (0, 8, 8))), BAD),
])
def test_attention_rejects(lib, case, expect):
    assert attend(lib, **case) == expect


def test_workspace_size_of_invalid_sizes(lib):
    for args in ((0, 4, 2, 1, 128), (1, 4, 3, 1, 128), (1, 4, 0, 1, 128), (1, 4, 2, 0, 128),
                 (1, 4, 2, 1, 96)):
        assert lib.fa_fwd_cache_workspace_size(*args) == 0


def test_the_binding_checks_what_it_marshals():
    with pytest.raises(ValueError):
        binding.Rope([])
    with pytest.raises(ValueError):
        binding.Rope([1.0] * 129)
    with pytest.raises(ValueError):
        binding.Rope([1.0] * 8, [0] * 7)
    with pytest.raises(ValueError):
        binding.Rope([1.0] * 8, [4] * 8)
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # not on a GPU
        binding.rope(q, None, None, binding.Rope([1.0] * 8))
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    s, t = torch.ones(2, 2), torch.zeros(1, 2, dtype=torch.int32)
    for bad in ((c, c[:1], s, s, t), (c.to(torch.int32), c.to(torch.int32), s, s, t),
                (c, c, s.double(), s, t), (c, c, s[:1], s, t), (c, c, s, s, t.long()),
                (c.transpose(2, 3), c.transpose(2, 3), s, s, t), (c, c, s, s, t)):
        with pytest.raises((ValueError, TypeError)):
            binding.Cache(*bad)
