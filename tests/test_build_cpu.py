"""Which objects a build makes anew: those of every file that a change reaches,
through headers and through a .cu that another one includes."""
import os
import shutil

import pytest

from exact_io_aware_20_gb300 import build


class Done:
    returncode, stdout, stderr = 0, "", ""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources, with a compiler that only writes what it is asked for."""
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    shutil.copytree(build.CSRC, csrc)
    shutil.copytree(build.INCLUDE, include)
    compiled = []

    def compiler(cmd, **_kw):
        out = cmd[cmd.index("-o") + 1]
        if "-c" in cmd:
            compiled.append(os.path.basename(cmd[cmd.index("-c") + 1]))
        with open(out, "w") as f:
            f.write("made")
        return Done()

    for name, to in (("CSRC", csrc), ("INCLUDE", include), ("BUILD_DIR", tmp_path / "_build"),
                     ("LIB_PATH", tmp_path / "lib.so")):
        monkeypatch.setattr(build, name, str(to))
    monkeypatch.setattr(build, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", compiler)

    def made(touched=None):
        """What a build compiles after `touched` has changed."""
        compiled.clear()
        for base in (csrc, include, tmp_path / "_build"):        # everything else is older than its object
            for f in base.iterdir() if base.exists() else ():
                os.utime(f, (2000, 2000) if base.name == "_build" else (1000, 1000))
        if touched:
            os.utime(touched, (3000, 3000))
        monkeypatch.setattr(build, "__file__", str(csrc / "fa_api.cu"))      # (as old as the sources)
        build.build()
        return set(compiled)

    return csrc, include, made


def test_a_kernel_that_is_compiled_twice_is_made_twice(tree):
    csrc, include, made = tree
    sources = {f.name for f in csrc.glob("*.cu")}
    assert made() == sources and made() == set()
    assert made(csrc / "fa_cache_fwd.cu") == {"fa_cache_fwd.cu", "fa_cache_fwd_tree.cu"}
    assert made(csrc / "fa_cache_prefill.cu") == {"fa_cache_prefill.cu", "fa_cache_prefill_tree.cu"}
    assert made(csrc / "fa_cache_fwd_tree.cu") == {"fa_cache_fwd_tree.cu"}
    both = {"fa_cache_fwd.cu", "fa_cache_fwd_tree.cu", "fa_cache_prefill.cu", "fa_cache_prefill_tree.cu"}
    assert made(csrc / "cache_work.cuh") == both
    # a header that a header includes
    assert both <= made(csrc / "sm103_ptx.cuh") and "fa_cache_api.cu" in made(include / "fa.h")


def test_every_included_file_is_found():
    """(a name that is not would be no dependency)"""
    for name in os.listdir(build.CSRC):
        path = os.path.join(build.CSRC, name)
        with open(path) as f:
            names = [line.split('"')[1] for line in f if line.lstrip().startswith("#") and "include" in line and '"' in line]
        found = {os.path.basename(p) for p in build.dependencies(path)}
        assert {os.path.basename(n) for n in names} <= found, name
