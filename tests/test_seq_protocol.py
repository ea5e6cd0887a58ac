"""The barriers of the causal prompt forward and of its gradients, gone through on the CPU.

A model of one block: the loader, copies that land in any order, the issuing thread, a tensor pipe that completes products in the order
of issue, and the two softmax warpgroups as warps of their own, with barriers that are waited for by parity as the hardware's
are (a wait passes when the barrier's current phase has the other parity, be it one phase further or one phase behind). The
order of the products and the waits that follow from it are the kernel's own, from csrc/clear_seq_order.h. Random
schedules, with agents that stall for long, look for a wait that passes before its phase is complete, for an
accumulator that is read before its last product, for a half's sums that are read after they were replaced, and for tiles in the ring
that are not the ones meant. The gradients' kernel (its order has no such header) is restated from its code below.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "local_circular_window_b200", "csrc")
WARPS = 2  # of each warpgroup: enough for a fast one and a slow one

SOURCE = """
#include "clear_seq_order.h"
template <int B, bool S> struct X { static int f(int what, int nA, int nB, int x, int y) {
  const clear::PromptOrder<B, S> o{nA, nB};
  return what == 0 ? o.place(x, y) : what == 1 ? o.alone() : what == 2 ? o.first(x) : what == 3 ? o.looks_back(x, y) : o.sums(x);
} };
extern "C" int order(int bufs, int split, int what, int nA, int nB, int x, int y) {
  return bufs == 2 ? (split ? X<2, true>::f(what, nA, nB, x, y) : X<2, false>::f(what, nA, nB, x, y))
                   : (split ? X<3, true>::f(what, nA, nB, x, y) : X<3, false>::f(what, nA, nB, x, y));
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("order")
    (at / "order.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(at / "order.so"), str(at / "order.cpp")], check=True)
    return ctypes.CDLL(str(at / "order.so")).order


class Fault(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1


class Machine:
    """Agents that take steps in a random order, with stalls; `left` are the ones that have to end."""

    def __init__(self, rng):
        self.rng, self.pipe, self.flying, self.ring = rng, [], [], {}

    def wait(self, name, bar, n):
        """Waits for the end of the barrier's phase number n (from 0), by parity."""
        while bar.phase & 1 == n & 1:  # n = -1: the phase before the first, which counts as complete
            yield
        if bar.phase < n + 1:
            raise Fault(f"{name}: a wait for phase {n} passed in phase {bar.phase}")

    def copies(self):
        while True:
            if self.flying:
                bar, s, tile = self.flying.pop(int(self.rng.random() * len(self.flying)))
                if s is not None:
                    self.ring[s] = tile
                bar.arrive()
            yield

    def tensor(self):
        while True:
            if self.pipe:
                op = self.pipe.pop(0)
                if op[0] == "PV":
                    self.acc[op[2]].append(op[3])
                if op[1] is not None:
                    op[1].arrive()
            yield

    def go(self, agents, left):
        names, stalled = list(agents), {}
        rng, idle = self.rng, 0
        while left:
            idle += 1
            assert idle < 200000, "no progress"
            a = names[int(rng.random() * len(names))]
            if stalled.get(a, 0) > 0:
                stalled[a] -= 1
                continue
            if rng.random() < 0.04:
                stalled[a] = int(rng.random() * 60)
            if a in agents and next(agents[a], "end") == "end":
                del agents[a]


class Block(Machine):
    """items: for each its number of key tiles and whether it has a tile B."""

    def __init__(self, order, bufs, split, items, rng):
        super().__init__(rng)
        self.bufs, self.split, self.items = bufs, split, items
        self.order = lambda what, it, x=0, y=0: order(bufs, int(split), what, *self.counts(it), x, y)
        self.s = {(b, h): Bar(1) for b in range(bufs) for h in (0, 1)}
        self.p = {(b, i): Bar(WARPS) for b in range(bufs) for i in (0, 1)}
        self.o = [Bar(1), Bar(1)]
        self.join, self.joined = Bar(2 * WARPS), Bar(2 * WARPS)
        self.stages = {2: 5, 3: 8}[bufs]
        self.full, self.empty = ([Bar(1) for _ in range(self.stages)] for _ in range(2))
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.ml = {}
        self.acc = [[], []]   # key tiles whose P V has been added to each accumulator, (item, tile)

    def key_tile(self, half, i):
        return 2 * i + half if self.split else i

    def place(self, n, what, j):
        """Place in the ring of a tile of item n: K0 K1 V0 K2 V1 ... V(last), behind those of earlier items."""
        tiles = [t + 1 if two and not self.split else t for t, two in self.items]
        m = tiles[n]
        at = (0 if j == 0 else 2 * j - 1) if what == "K" else (2 * m - 1 if j == m - 1 else 2 * j + 2)
        return 2 * sum(tiles[:n]) + at

    def loader(self):
        at = 0
        for n, (t, two) in enumerate(self.items):
            m = t + 1 if two and not self.split else t
            yield from self.wait("Q empty", self.q_empty, n - 1)
            self.flying.append((self.q_full, None, None))
            for j in range(m + 1):
                for what, x in (("K", j), ("V", j - 1)):
                    if not 0 <= x < m:
                        continue
                    s = at % self.stages
                    assert self.place(n, what, x) == at
                    yield from self.wait("ring empty", self.empty[s], at // self.stages - 1)
                    self.ring[s] = None
                    self.flying.append((self.full[s], s, (n, what, x)))
                    at += 1
                    yield

    def tile(self, n, what, j):
        """Waits for a tile of the ring; returns its stage."""
        at = self.place(n, what, j)
        s = at % self.stages
        yield from self.wait(f"ring full, {what}", self.full[s], at // self.stages)
        if self.ring[s] != (n, what, j):
            raise Fault(f"{(n, what, j)} is not in the ring, but {self.ring[s]}")
        return s

    def counts(self, it):
        tiles, two = it
        return ((tiles + 1) // 2, tiles // 2) if self.split else (tiles, tiles + 1 if two else 0)

    def issuer(self):
        uses = [0] * self.bufs
        for n, it in enumerate(self.items):
            nA, nB = self.counts(it)
            places = {self.order(0, it, h, i): (h, i) for h, m in ((0, nA), (1, nB)) for i in range(m)}
            total = nA + nB
            assert sorted(places) == list(range(total))
            alone = self.order(1, it)
            ahead = 0

            users = {}  # products still to come for each tile in the ring
            for h, i in places.values():
                for what in "KV":
                    users[what, self.key_tile(h, i)] = users.get((what, self.key_tile(h, i)), 0) + 1

            def used(what, j, s):
                users[what, j] -= 1
                if users[what, j] == 0:
                    self.pipe.append(("commit", self.empty[s]))

            def issue(b):
                nonlocal ahead
                h, i = places[ahead]
                assert b == ahead % self.bufs
                j = self.key_tile(h, i)
                s = yield from self.tile(n, "K", j)
                self.pipe.append(("S", self.s[b, h]))
                used("K", j, s)
                ahead += 1
                if ahead == total:
                    self.pipe.append(("commit", self.q_empty))

            yield from self.wait("Q", self.q_full, n)
            while ahead < total and self.order(2, it, ahead):
                yield from issue(ahead % self.bufs)
            if self.split:
                yield from self.wait("accumulators", self.joined, n - 1)
            for g in range(total):
                h, i = places[g]
                s = yield from self.tile(n, "V", self.key_tile(h, i))
                for part in (0, 1):
                    yield from self.wait(f"P {part}", self.p[g % self.bufs, part], uses[g % self.bufs])
                uses[g % self.bufs] += 1
                self.pipe.append(("PV", self.o[h], h, (n, i)))
                used("V", self.key_tile(h, i), s)
                if ahead < total:
                    yield from issue((g + 1) % self.bufs if alone else g % self.bufs)
                yield

    def warp(self, half, w, left):
        no = joins = 0
        seen = [0] * self.bufs
        for n, it in enumerate(self.items):
            m = self.counts(it)[half]
            if m == 0 and not self.split:
                continue
            for i in range(m):
                b = self.order(0, it, half, i) % self.bufs
                yield from self.wait(f"S {half}", self.s[b, half], seen[b])
                seen[b] += 1
                yield
                if i > 0 and self.rng.random() < 0.3:  # the maximum moves: the accumulator is rescaled
                    yield from self.wait(f"P V {half}, rescaling", self.o[half], no + i - 1)
                diagonal = self.key_tile(half, i) == it[0] - 1 if self.split else i == m - 1 and (half == 1 or not it[1])
                if diagonal:  # value rows behind the sequence's end are cleared
                    yield from self.tile(n, "V", self.key_tile(half, i))
                self.p[b, 0].arrive()
                yield
                if self.order(3, it, half, i):
                    yield from self.wait(f"P V {half}, looking back", self.o[half], no + i - 1)
                self.p[b, 1].arrive()
                yield
            no += m
            if m > 0:
                yield from self.wait(f"P V {half}, last", self.o[half], no - 1)
            if not self.split:
                if self.acc[half][-1] != (n, m - 1):
                    raise Fault(f"the accumulator of {half} is read at {self.acc[half][-1]} and not {(n, m - 1)}")
                yield
                continue
            copy = self.order(4, it, joins)
            self.ml[copy, half, w] = n
            yield
            self.join.arrive()
            yield from self.wait("join", self.join, joins)
            yield
            joins += 1
            if self.ml[copy, 1 - half, w] != n:
                raise Fault(f"half {half} of item {n} reads the other's sums of item {self.ml[copy, 1 - half, w]}")
            for h in (0, 1):
                k = self.counts(it)[h]
                if k and self.acc[h][-1] != (n, k - 1):
                    raise Fault(f"the accumulator of {h} is read at {self.acc[h][-1]} and not {(n, k - 1)}")
            yield
            self.joined.arrive()
        left.remove((half, w))

    def run(self):
        left = {(h, w) for h in (0, 1) for w in range(WARPS)}
        agents = {("issuer", 0): self.issuer(), ("tensor", 0): self.tensor(), ("loader", 0): self.loader(), ("copies", 0): self.copies()}
        agents |= {x: self.warp(*x, left) for x in left}
        self.go(agents, left)


SHAPES = [[(1, True), (2, True), (4, True)], [(3, False), (1, False), (2, False)], [(3, True), (2, False), (1, True), (1, False)],
          [(5, False), (1, False), (1, False), (1, False), (1, False), (2, False)], [(6, True), (1, True), (1, True)]]


@pytest.mark.parametrize("bufs", [2, 3])
@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
def test_every_wait_sees_its_phase(order, bufs, split):
    rng = random.Random(bufs * 2 + split)
    for k in range(600):
        items = rng.choice(SHAPES)
        if split:
            items = [(n, False) for n, _ in items]
        Block(order, bufs, split, items, rng).run()


class Gradients(Machine):
    """The gradients' kernel. items: steps (pairs of streamed halves) of each; kv: the kernel of dK and dV, else of dQ, whose items of
    one step exchange the first rows' sums."""

    def __init__(self, bufs, kv, items, rng):
        super().__init__(rng)
        self.bufs, self.kv, self.items, self.stages = bufs, kv, items, {2: 4, 3: 8}[bufs]
        self.x_full, self.x_empty, self.acc_bar, self.acc_free = Bar(1), Bar(1), Bar(1), Bar(2 * WARPS)
        self.full = [Bar(2 if kv else 1) for _ in range(self.stages)]
        self.empty = [Bar(1) for _ in range(self.stages)]
        self.s, self.p = ([Bar(c) for _ in range(bufs)] for c in (1, WARPS))
        self.d = Bar(2 * WARPS)
        self.acc = [[]]
        self.far, self.sums = {}, {}

    def loader(self):
        at = 0
        for n, steps in enumerate(self.items):
            yield from self.wait("X empty", self.x_empty, n - 1)
            self.flying.append((self.x_full, None, None))
            for i in range(2 * steps):
                s = at % self.stages
                yield from self.wait("Y empty", self.empty[s], at // self.stages - 1)
                self.ring[s] = None
                self.flying.append((self.full[s], s, (n, i)))
                at += 1
                yield

    def statistics(self):
        at = 0
        for n, steps in enumerate(self.items):
            for i in range(2 * steps):
                s = at % self.stages
                yield from self.wait("Y empty, statistics", self.empty[s], at // self.stages - 1)
                self.far[s] = (n, i)
                yield
                self.full[s].arrive()
                at += 1
                yield

    def issuer(self):
        at, uses = 0, [0] * self.bufs
        for n, steps in enumerate(self.items):
            halves, ahead, stage = 2 * steps, 0, [0] * self.bufs

            def scores(b):
                nonlocal at, ahead
                s = at % self.stages
                yield from self.wait("Y", self.full[s], at // self.stages)
                if self.ring[s] != (n, ahead):
                    raise Fault(f"{(n, ahead)} is not in the ring, but {self.ring[s]}")
                at += 1
                self.pipe.append(("S", self.s[b]))
                ahead += 1
                if ahead == halves:
                    self.pipe.append(("commit", self.x_empty))
                stage[b] = s

            yield from self.wait("X", self.x_full, n)
            for b in range(min(self.bufs, halves)):
                yield from scores(b)
            yield from self.wait("accumulators", self.acc_free, n - 1)
            for g in range(halves):
                b = g % self.bufs
                yield from self.wait("P", self.p[b], uses[b])
                uses[b] += 1
                self.pipe.append(("PV", self.empty[stage[b]], 0, (n, g)))
                yield
                if ahead < halves:
                    yield from scores(b)
            self.pipe.append(("commit", self.acc_bar))

    def warp(self, half, w, left):
        ns, before, slot, joins = 0, [0] * self.bufs, 0, 0  # ns: as the kernel keeps the phases; before: uses of each buffer
        for n, steps in enumerate(self.items):
            for i in range(steps):
                b, other = (2 * i + half) % self.bufs, (2 * i + 1 - half) % self.bufs
                st = (2 * slot + half) % self.stages
                slot += 1
                phase = ns >> b & 1
                ns ^= 1 << b
                if self.bufs == 3:
                    ns ^= 1 << other
                mine = before[b] + (1 if half == 1 and other == b else 0)
                assert phase == mine & 1
                yield from self.wait(f"scores {half}", self.s[b], mine)
                before[b] += 1
                before[other] += self.bufs == 3  # with two buffers each half has one
                yield
                if self.ring[st] != (n, 2 * i + half) or self.kv and self.far[st] != (n, 2 * i + half):
                    raise Fault(f"stage {st} holds {self.ring[st]} and {self.far.get(st)}, not {(n, 2 * i + half)}")
                if not self.kv and steps == 1:
                    self.sums[half, w] = n
                    yield
                    self.d.arrive()
                    yield from self.wait("sums", self.d, joins)
                    joins += 1
                    yield
                    if self.sums[1 - half, w] != n:
                        raise Fault(f"half {half} of item {n} reads the other's sums of item {self.sums[1 - half, w]}")
                self.p[b].arrive()
                yield
            yield from self.wait("last product", self.acc_bar, n)
            if self.acc[0][-1] != (n, 2 * steps - 1):
                raise Fault(f"the accumulators are read at {self.acc[0][-1]} and not {(n, 2 * steps - 1)}")
            yield
            self.acc_free.arrive()
        left.remove((half, w))

    def run(self):
        left = {(h, w) for h in (0, 1) for w in range(WARPS)}
        agents = {x: getattr(self, x)() for x in ("issuer", "tensor", "loader", "copies")}
        if self.kv:
            agents["statistics"] = self.statistics()
        self.go(agents | {x: self.warp(*x, left) for x in left}, left)


@pytest.mark.parametrize("bufs", [2, 3])
@pytest.mark.parametrize("kv", [False, True], ids=["dq", "dkdv"])
def test_every_wait_of_the_gradients_sees_its_phase(bufs, kv):
    rng = random.Random(10 + bufs * 2 + kv)
    for k in range(600):
        Gradients(bufs, kv, rng.choice([[5, 3, 1, 1], [1, 1, 1, 2, 1], [4, 2, 2, 1], [7, 1, 6], [3, 3, 1, 1, 1]]), rng).run()
