"""The barriers of the many-row cache attention where two softmax groups each take
half the keys of one tile of rows: the model of test_cache_protocol_cpu.py
with that kernel's products and softmax, and its counts, waits and places against
the source."""
import random

import pytest

from test_cache_protocol_cpu import Bar, Model
from test_cache_protocol_sources_cpu import SOURCE, constants


class SplitModel(Model):
    def __init__(self, d, pieces, seed, there=8, read=8):
        super().__init__(d, pieces, seed)
        self.there, self.read = Bar(there), Bar(read)
        self.stat = [{}, {}]
        self.half = [{}, {}]      # score buffer: by group, what its half holds

    def scores(self, u, buf, n, j, c, s):
        def run():
            assert self.k[s] == (n, j, c) and all(self.q[i] == n for i in range(self.conv))
            assert not self.half[buf] or all(x == "read" for x in self.half[buf].values())
            self.half[buf] = {0: ("S", n, j), 1: ("S", n, j)}
        self.pipe.append(run)

    def values(self, u, buf, n, j, h, s, fresh):
        def run():
            assert self.half[buf][u] == ("P", n, j)
            assert len([1 for x in self.v[s].values() if x == (n, j, h)]) == self.conv
            self.half[buf][u] = "read"
            self.o[u] = (n, 1) if fresh else (n, self.o[u][1] + 1)
            assert fresh or self.o[u][0] == n
        self.pipe.append(run)

    def products(self):
        kp = vp = g = 0
        for n in range(len(self.pieces) + 1):
            yield self.rec_full[n & 3], (n >> 2) & 1
            w = self.piece(n)
            self.rec_empty[n & 3].arrive()
            if w is None:
                return
            s0, s1 = w["s0"], w["s1"]
            yield self.q_full, n & 1

            def ahead(buf, j):
                nonlocal kp
                s = kp % self.k_stages
                self.scores(0, buf, n, j, 0, s)
                self.commit(self.k_empty[s])
                self.commit(self.s_full[buf])
                kp += 1

            for i in range(min(2, s1 - s0)):
                yield self.k_full[kp % self.k_stages], (kp // self.k_stages) & 1
                ahead((g + i) & 1, s0 + i)
            if s1 - s0 <= 2:
                self.commit(self.q_empty)
            for j in range(s0, s1):
                more = j + 2 < s1
                sv, sk = vp % self.v_stages, kp % self.k_stages
                # (one wait of several lanes: each barrier's phase, in any order)
                waits = [(self.v_full[sv], (vp // self.v_stages) & 1), (self.p_full[0], g & 1), (self.p_full[1], g & 1)]
                if more:
                    waits.append((self.k_full[sk], (kp // self.k_stages) & 1))
                self.rng.shuffle(waits)
                for x in waits:
                    yield x
                for u in range(2):
                    self.values(u, g & 1, n, j, 0, sv, j == s0)
                self.commit(self.v_empty[sv])
                self.commit(self.o_done[0])
                self.commit(self.tile_empty[g & 7])
                if more:
                    ahead(g & 1, j + 2)
                    if j + 3 == s1:
                        self.commit(self.q_empty)
                vp += 1
                g += 1

    def softmax(self, u, warp):
        cs = od = g = 0
        for n in range(len(self.pieces) + 1):
            yield self.rec_full[n & 3], (n >> 2) & 1
            w = self.piece(n)
            if w is None:
                return
            s0, s1 = w["s0"], w["s1"]
            for j in range(s0, s1):
                buf = cs & 1
                yield self.s_full[buf], (cs >> 1) & 1
                cs += 1
                if j == s0:
                    assert all(x == n for x in self.pow[n & 1].values())
                assert self.info[(g + j - s0) & 7] == g + j - s0
                assert self.half[buf][u] in (("S", n, j), ("P", n, j))
                if j > s0:      # O may be rescaled after this
                    yield self.o_done[0], od & 1
                    od += 1
                    assert self.o[u] == (n, j - s0)
                if n > 0 and j == s0:
                    yield self.read, (n - 1) & 1
                self.half[buf][u] = ("P", n, j)
                self.p_full[u].arrive()
            assert self.piece(n) is w
            self.stat[u][warp] = n
            self.there.arrive()
            yield self.o_done[0], od & 1
            yield self.there, n & 1
            od += 1
            for _ in range(2):      # the other group's statistics and both O, until the last row has been read
                assert self.stat[u ^ 1][warp] == n
                assert self.o[0] == self.o[1] == (n, s1 - s0)
                assert self.nan[n & 7] == (n if n else None)
                yield None
            self.rec_empty[n & 3].arrive()
            self.results[(n, u)] = self.results.get((n, u), 0) + 1
            self.read.arrive()
            g += s1 - s0


def pieces(rng, count, most):
    out = []
    for _ in range(count):
        s0 = rng.choice([0, 0, 3])
        s1 = s0 + rng.randint(1, most)
        out.append({"s0": s0, "s1": s1, "end": [s1, s1]})
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [1, 2, 3, 5, 12])
def test_no_schedule_stalls_or_reads_the_wrong_thing(d, most):
    for seed in range(12):
        rng = random.Random(1000 * d + 10 * most + seed)
        SplitModel(d, pieces(rng, 40 if most < 6 else 12, most), seed).run()


@pytest.mark.parametrize("there,read", [(7, 8), (8, 7)])
def test_the_model_sees_a_warp_that_is_not_counted(there, read):
    bad = 0
    for seed in range(8):
        try:
            SplitModel(128, pieces(random.Random(seed), 40, 3), seed, there, read).run()
        except (AssertionError, TypeError, KeyError):
            bad += 1
    assert bad == 8


def test_the_model_is_the_kernel_s():
    for d in (64, 128):
        known = constants(d)
        # what the groups exchange lies in the second tile of q
        assert known["kQOff"] + known["kQTile"] + 2 * 128 * 8 + 16 <= known["kKOff"]
        assert known["kSoftWarps"] == 8
    for line in ("mbar_init(there, L::kSoftWarps)", "mbar_init(read, L::kSoftWarps)",
                 "on = bar(L::kPFull + lane - 1);", "turn = g;", "turn = kp / L::kKStages;", "int turn = vp / L::kVStages;",
                 "wait_each(on, turn & 1, abort)", "sbase + Split<D>::kRead, (np - 1) & 1",
                 "bar(L::kODone), od & 1", "sbase + Split<D>::kThere, np & 1",
                 "bar(L::kSFull + buf), (kOneTile ? cs >> 1 : cs) & 1",
                 "static constexpr int kStatOff = L::kQOff + L::kQTile;",
                 "static constexpr int kThere = kStatOff + 2 * 128 * 8, kRead = kThere + 8;"):
        assert line in SOURCE, line
