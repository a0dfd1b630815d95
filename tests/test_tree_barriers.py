"""The barriers of the tree attention as a model on the CPU.

A wait for a phase of a barrier looks at a parity: it misses its phase, and never ends, when the barrier may be two phases on before
the warp looks, and it passes too early when the barrier may be two phases behind.  The model has the kernel's warps, rings and barriers
(csrc/tree.cu), copies that come late and warps that are late at any place; each wait checks that it ended with the phase it was for.
What keeps a barrier from running ahead of a wait (a tie) is left out in turn, which the model has to notice.
"""
import heapq
import random

import pytest

TILES = 8       # barriers of K tiles, of V tiles and of checked V tiles
LISTS = 16      # of a tile's keys that cannot be read
SLACK = 4       # most tiles that two pieces may differ in to run side by side
TIES = ("the V check frees K's slots", "each chain frees both Q tiles", "a chain without a tile waits for no O")


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0, "more arrivals than a phase has"
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count


class Model:
    def __init__(self, seed, slots, ahead, bias, short, ties):
        self.r = r = random.Random(seed)
        self.slots, self.ahead, self.bias = slots, ahead, bias
        self.v_tie, self.q_tie, self.o_tie = (t in ties for t in TIES)
        self.wrong, self.events, self.now = [], [], (0.0, 0)
        # items: mode, tiles of each chain, Q slot of a piece that both chains share
        self.items, slot = [], 1
        for _ in range(r.randint(4, 10)):
            mode = r.choice(("pair", "split", "split", "dual"))
            n = r.randint(1, 12)
            if mode == "split":
                n = r.choice((1, 1, 2, 3, 9) if short else (2, 3, 9))
                tiles = ((n + 1) // 2, n // 2)
            else:
                tiles = (n, n if mode == "pair" else max(1, n + r.randint(-SLACK, SLACK)))
            slot = slot ^ 1 if mode == "split" else 1
            self.items.append((mode, tiles, slot))
        # the row of tiles: the chains' take turns
        self.row, self.at = [], {}
        for k, (mode, tiles, _) in enumerate(self.items):
            for j in range(max(tiles)):
                for h in (0,) if mode == "pair" else (0, 1):
                    if j < tiles[h]:
                        self.at[k, h, j] = self.at[k, 1 if mode == "pair" else h, j] = len(self.row)
                        self.row.append(k)
        bars = lambda n, count: [Barrier(count) for _ in range(n)]
        self.k_full, self.v_full, self.v_ok = bars(TILES, 1), bars(TILES, 1), bars(TILES, 1)
        self.k_empty, self.v_empty = bars(slots, 3 if self.v_tie else 2), bars(slots, 2)
        self.s_full, self.p_full, self.o_done = (bars(4, n) for n in (1, 4, 1))   # [2 chains][2]
        self.q_full, self.q_empty = bars(2, 4 if bias else 1), bars(2, 3 if self.q_tie else 2)
        self.b_full, self.b_empty = bars(2, 1), bars(2, 4)
        self.item_full, self.item_empty = bars(2, 1), bars(2, 15 if bias else 13)
        self.o_free, self.ml = Barrier(8), Barrier(8)
        self.bad_keys = [None] * LISTS

    def late(self):
        return self.r.uniform(3, 40) if self.r.random() < 0.05 else self.r.uniform(0.0, 0.1)

    def copy(self, what):
        self.after(self.r.uniform(5, 30) if self.r.random() < 0.1 else self.r.uniform(0.3, 1.0), what)

    def after(self, dt, what):
        self.now = (self.now[0], self.now[1] + 1)
        heapq.heappush(self.events, (self.now[0] + dt, self.now[1], what))

    def wait(self, who, bar, phase):
        def ready():
            if (bar.phase & 1) == (phase & 1):
                return False
            if bar.phase != phase + 1:
                self.wrong.append(f"{who}: phase {phase} of a barrier that is in phase {bar.phase}")
            return True
        ready.who = who
        return ready

    def reads(self, who, x):
        if self.bad_keys[x % LISTS] != x:
            self.wrong.append(f"{who}: the list of tile {x} is that of tile {self.bad_keys[x % LISTS]}")

    def begin(self, k, who):
        return self.wait(f"{who}, item {k}", self.item_full[k % 2], k // 2)

    def end(self, k):
        self.item_empty[k % 2].arrive()

    # ---- the warps

    def producer(self, name, full, empty):
        x = 0
        for k in range(len(self.items)):
            yield self.begin(k, name)
            yield self.late()
            self.end(k)
            while x < len(self.row) and self.row[x] == k:
                if x >= self.slots:
                    yield self.wait(f"{name}, slot of tile {x}", empty[x % self.slots], x // self.slots - 1)
                if full is self.k_full:
                    self.bad_keys[x % LISTS] = x
                self.copy(lambda x=x: full[x % TILES].arrive())
                x += 1
                yield self.late()

    def scheduler(self):
        loads = [0, 0]
        for k, (mode, _, slot) in enumerate(self.items):
            if k >= 2:
                yield self.wait("scheduler", self.item_empty[k % 2], k // 2 - 1)
            yield self.late()
            self.item_full[k % 2].arrive()
            for s in () if self.bias else (slot,) if mode == "split" else (0, 1):
                if loads[s] > 0:
                    yield self.wait(f"scheduler, Q tile of item {k}", self.q_empty[s], loads[s] - 1)
                loads[s] += 1
                self.copy(lambda s=s: self.q_full[s].arrive())
                yield self.late()

    def products(self, h):
        sc = pc = merges = 0
        qn, merged = [0, 0], False
        for k, (mode, tiles, slot) in enumerate(self.items):
            who, n, pair, split = f"products {h}, item {k}", tiles[h], mode == "pair", mode == "split"
            s = slot if split else h
            yield self.begin(k, who)
            yield self.late()
            if not self.bias or n > 0:
                s = h if self.bias else s
                yield self.wait(who + ", Q", self.q_full[s], qn[s])
                qn[s] += 1
                yield self.late()
            if not self.bias and not split:
                yield self.wait(who + ", the other Q", self.q_full[h ^ 1], qn[h ^ 1])
                qn[h ^ 1] += 1
                yield self.late()

            def scores(j):
                nonlocal sc
                x = self.at[k, h, j]
                yield self.wait(f"{who}, K of tile {x}", self.k_full[x % TILES], x // TILES)
                yield self.late()
                c, last = sc, j + 1 == n
                sc += 1

                def done(s=s, split=split, pair=pair):
                    self.k_empty[x % self.slots].arrive(1 if pair else 2)
                    self.s_full[2 * h + (c & 1)].arrive()
                    if last and not self.bias:
                        self.q_empty[s].arrive(1 if split else 2)
                self.after(0.2, done)

            if n > 0:
                for j in range(min(self.ahead, n)):
                    yield from scores(j)
            elif not self.bias:
                self.q_empty[s].arrive()
            if merged and (n > 0 or not self.o_tie):
                yield self.wait(who + ", O", self.o_free, merges - 1)
            yield self.late()
            for j in range(n):
                x = self.at[k, h, j]
                yield self.wait(f"{who}, V of tile {x}", self.v_ok[x % TILES], x // TILES)
                yield self.wait(who + ", P", self.p_full[2 * h + (pc & 1)], pc >> 1)
                yield self.late()

                def done(x=x, c=pc, pair=pair):
                    self.v_empty[x % self.slots].arrive(1 if pair else 2)
                    self.o_done[2 * h + (c & 1)].arrive()
                self.after(0.2, done)
                pc += 1
                if j + self.ahead < n:
                    yield from scores(j + self.ahead)
            if not self.bias and self.q_tie and not (split and h == 1):
                self.q_empty[s if split else h ^ 1].arrive()
            merged = split
            merges += split
            self.end(k)

    def softmax(self, h):
        c = other = met = bn = 0
        for k, (mode, tiles, _) in enumerate(self.items):
            who, n = f"softmax {h}, item {k}", tiles[h]
            yield self.begin(k, who)
            yield self.late()
            if self.bias and n > 0:
                self.q_full[h].arrive()
            for j in range(n):
                yield self.wait(who + ", S", self.s_full[2 * h + (c & 1)], c >> 1)
                c += 1
                if self.bias:
                    yield self.wait(who + ", bias", self.b_full[h], bn)
                    bn += 1
                yield self.r.uniform(0.2, 0.6) + self.late()
                if self.bias:
                    self.b_empty[h].arrive()
                if j > 0 and self.r.random() < 0.3:
                    yield self.wait(who + ", O to scale", self.o_done[2 * h + (c & 1)], (c - 2) >> 1)
                self.reads(who, self.at[k, h, j])
                self.p_full[2 * h + (c - 1 & 1)].arrive()
            other += tiles[h ^ 1]
            if n > 0:
                yield self.wait(who + ", O", self.o_done[2 * h + (c - 1 & 1)], (c - 1) >> 1)
            yield self.late()
            if mode == "split":
                self.ml.arrive()
                yield self.wait(who + ", maxima", self.ml, met)
                met += 1
                yield self.late()
                if h == 1 or tiles[1] > 0:
                    yield self.wait(who + ", the other O", self.o_done[2 * (h ^ 1) + (other - 1 & 1)], (other - 1) >> 1)
                yield self.late()
                self.o_free.arrive()
            self.end(k)

    def check(self):
        x = 0
        for k in range(len(self.items)):
            yield self.begin(k, "V check")
            yield self.late()
            while x < len(self.row) and self.row[x] == k:
                yield self.wait(f"V check, K of tile {x}", self.k_full[x % TILES], x // TILES)
                if self.v_tie:
                    self.k_empty[x % self.slots].arrive()
                yield self.wait(f"V check, V of tile {x}", self.v_full[x % TILES], x // TILES)
                yield self.late()
                self.reads("V check", x)
                self.v_ok[x % TILES].arrive()
                x += 1
            self.end(k)

    def bias_loads(self, h):
        fills = 0
        for k, (_, tiles, _) in enumerate(self.items):
            yield self.begin(k, f"bias {h}")
            for _ in range(tiles[h]):
                if fills > 0:
                    yield self.wait(f"bias {h}", self.b_empty[h], fills - 1)
                fills += 1
                self.copy(self.b_full[h].arrive)
                yield self.late()
            self.end(k)

    def run(self):
        """What went wrong ('' for nothing)."""
        warps = [self.producer("K", self.k_full, self.k_empty), self.producer("V", self.v_full, self.v_empty), self.scheduler(),
                 self.products(0), self.products(1), self.check(), *(self.softmax(h) for h in (0, 1) for _ in range(4)),
                 *(self.bias_loads(h) for h in (0, 1) if self.bias)]
        waiting = {}

        def step(i):
            waiting.pop(i, None)
            got = next(warps[i], None)
            if callable(got):
                waiting[i] = got
            elif got is not None:
                self.after(got, lambda: step(i))

        for i in range(len(warps)):
            step(i)
        while True:
            ready = [i for i in list(waiting) if waiting[i]()]
            for i in ready:
                step(i)
            if self.wrong:
                return self.wrong[0]
            if ready:
                continue
            if not self.events:
                return "; ".join(f"{w.who} waits" for w in waiting.values())
            t, _, what = heapq.heappop(self.events)
            self.now = (t, self.now[1])
            what()


# K slots, S a chain, with a bias: heads of 64 and of 128
SHAPES = [(8, 2, False), (5, 2, False), (8, 1, True), (4, 1, True)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("short", [False, True])
def test_every_wait_ends_with_its_phase(shape, short):
    for seed in range(300):
        assert Model(seed, *shape, short, TIES).run() == "", seed


@pytest.mark.parametrize("shape,tie", [((8, 2, False), 0), ((8, 1, True), 0), ((5, 2, False), 1), ((8, 2, False), 2), ((4, 1, True), 2)])
def test_a_tie_that_is_missing_is_noticed(shape, tie):
    ties = [t for i, t in enumerate(TIES) if i != tie]
    assert any(Model(seed, *shape, tie == 2, ties).run() for seed in range(1000))
