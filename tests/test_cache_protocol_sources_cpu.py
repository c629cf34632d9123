"""The barrier model of test_cache_protocol_cpu.py has the depths and the
arrival counts of the kernel: both are read from the kernel's source here."""
import os
import re

import pytest

from exact_io_aware_20_gb300 import build
from test_cache_protocol_cpu import Model

SOURCE = open(os.path.join(build.CSRC, "fa_cache_prefill.cu")).read()


def python(expr):
    """A C++ constant expression of the kernel's in Python: names without their
    struct, one conditional, whole division."""
    expr = expr.replace("L::", "").replace("/", "//")
    m = re.fullmatch(r"(.+?)\?(.+):(.+)", expr)
    return f"({python(m[2])}) if ({python(m[1])}) else ({python(m[3])})" if m else expr


def constants(d):
    known = {"D": d}
    body = SOURCE[SOURCE.index("struct Pre {"):SOURCE.index("static_assert(kAlloc")]
    for m in re.finditer(r"static constexpr \w+ (k\w+ = [^;]+);", re.sub(r"//[^\n]*", "", body)):
        for one in m[1].split(","):
            name, expr = one.split("=", 1)
            known[name.strip()] = eval(python(" ".join(expr.split())), {}, known)
    return known


def counts(known):
    """Barriers by name: how many there are of it, and what each is initialised with."""
    body = SOURCE[SOURCE.index("nan_seen[s] = 0;") - 2500:SOURCE.index("fence_barrier_init();")]
    body = re.sub(r"//[^\n]*", "", body[body.index("if (threadIdx.x == 0) {"):])
    found, times = {}, 1
    for line in body.splitlines():
        loop = re.search(r"for \(int s = 0; s < ([^;]+); \+\+s\)", line)
        if loop:
            times = eval(python(loop[1].strip()), {}, known)
        m = re.search(r"mbar_init\(bar\(L::(\w+)( \+ s)?\), (.+)\);", line)
        if m:
            found[m[1]] = (times if m[2] else 1, eval(python(m[3]), {}, known))
    return found


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_model_is_the_kernel_s(d):
    known, model = constants(d), Model(d, [], 0)
    bars = {"kQFull": [model.q_full], "kQEmpty": [model.q_empty], "kKFull": model.k_full, "kKEmpty": model.k_empty,
            "kVFull": model.v_full, "kVEmpty": model.v_empty, "kSFull": model.s_full, "kPFull": model.p_full,
            "kODone": model.o_done, "kRecFull": model.rec_full, "kRecEmpty": model.rec_empty,
            "kTileFull": model.tile_full, "kTileEmpty": model.tile_empty}
    found = counts(known)
    assert found.pop("kDrain") == (1, 1)      # (the issuer's own, at the end: no other role waits for it)
    assert found == {name: (len(b), b[0].count) for name, b in bars.items()}
    # the barriers' places do not overlap: each begins where the one before it ends
    names = sorted(found, key=lambda n: known[n])
    at = [known[n] for n in names] + [known["kNumBars"]]
    room = {n: b - a for n, a, b in zip(names, at, at[1:])}
    assert all(room[n] >= found[n][0] for n in names)
    assert (known["kTiles"], known["kKParts"], known["kVParts"]) == (model.tiles, model.k_parts, model.v_parts)
    assert (known["kSoftWarps"], known["kConvWarps"]) == (model.soft, model.conv)
    assert [len(model.nan)] == [int(n) for n in re.findall(r"s < (\d+); \+\+s\) \{\s*nan_seen", SOURCE)]


def test_parities_and_slots_are_the_model_s():
    """Every wait of the kernel that the model restates, as it stands there."""
    for wait in ("bar(L::kRecFull + (np & 3)), (np >> 2) & 1", "bar(L::kRecEmpty + (np & 3)), ((np >> 2) + 1) & 1",
                 "bar(L::kTileEmpty + (g & 7)), ((g >> 3) + 1) & 1", "bar(L::kTileFull + (g & 7)), (g >> 3) & 1",
                 "bar(L::kKEmpty + s), (kp / L::kKStages + 1) & 1",
                 "bar(L::kKFull + n % L::kKStages), (n / L::kKStages) & 1",
                 "bar(L::kVFull + n % L::kVStages), (n / L::kVStages) & 1",
                 "bar(L::kVEmpty + s), (n / L::kVStages + 1) & 1", "bar(L::kQFull), np & 1",
                 "bar(L::kQEmpty), (np - 1) & 1", "bar(L::kPFull + buf), (g >> 1) & 1",
                 "bar(L::kPFull + u), pf[u] & 1", "bar(L::kODone), od & 1"):
        assert wait in SOURCE, wait
