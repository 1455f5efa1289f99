"""A model of the tree-attention kernel's barrier protocol (csrc/tree_tc.cu) under random
interleavings: two CTAs, each with two loading warps (every second place of the ring each), a fixer
and four softmax warps, and the first CTA's MMA warp. Loads land and MMAs complete after random delays. Checked:
no deadlock, no parity wait that passes on the wrong phase, no stage refilled or buffer
overwritten while a product may still read it, and every product reads what it should."""
import random

import pytest

STAGES, KST = 7, 9


class Barrier:
    """An mbarrier: phases by arrivals and bytes; waits see only the parity."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, expect=0):
        self.tx += expect
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than the phase has"
        self._turn()

    def complete(self, n):
        self.tx -= n
        self._turn()

    def passes(self, parity, want):
        """A parity wait; `want` is the phase that the waiter means."""
        ok = (self.phase & 1) != parity
        if ok:
            assert self.phase > want, "a wait passed before its phase was over"
        assert self.phase <= want + 1, "a wait would miss its phase"
        return ok


class Model:
    def __init__(self, tiles, seed, planted=None):
        self.rng = random.Random(seed)
        self.tiles, self.planted = tiles, planted
        self.bar = [dict(full=[Barrier(2) for _ in range(STAGES)], qfull=Barrier(2),
                         sfree=[Barrier(8), Barrier(8)], pready=Barrier(8),
                         empty=[Barrier(1) for _ in range(STAGES)], qempty=Barrier(1),
                         sfull=[Barrier(1), Barrier(1)], pvdone=Barrier(1), red=Barrier(4),
                         fix=[Barrier(1) for _ in range(STAGES)]) for _ in range(2)]
        self.ring = [[None] * STAGES for _ in range(2)]   # what each stage holds
        self.readers = [0] * STAGES                       # products that may still read a stage
        self.q, self.q_readers = [None, None], 0
        self.s = [[None, None], [None, None]]             # S buffers of each CTA
        self.p, self.p_readers = [[None] * 4, [None] * 4], 0
        self.events = []                                  # landing loads
        self.mma = []                                     # products and commits, in order
        self.done_pv = []

    # -- asynchronous engines
    def load(self, rank, store, key, bar, nbytes):
        def land():
            store(key)
            bar.complete(nbytes)
        self.events.append(land)

    def step_async(self):
        choices = (["load"] if self.events else []) + (["mma"] if self.mma else [])
        if not choices:
            return False
        if self.rng.choice(choices) == "load":
            self.events.pop(self.rng.randrange(len(self.events)))()
        else:
            self.mma.pop(0)()
        return True

    # -- one CTA's loading warps
    def arm(self, rank, bar, n):
        if rank == 0:
            bar.arrive()
            bar.arrive(n)

    def put(self, rank, st, key):
        assert self.readers[st] == 0, "a stage is refilled while a product may read it"
        self.ring[rank][st] = ("landing", key)

        def store(k):
            self.ring[rank][st] = k
        return store

    def loader(self, rank, turn):
        used = 0

        def mine():
            if self.planted == "split":  # one warp for K and one for V instead
                if is_k != (turn == 0):
                    return False
            elif used & 1 != turn:
                return False
            if used >= STAGES:
                st, n = used % STAGES, used // STAGES
                while not self.bar[rank]["empty"][st].passes((n & 1) ^ 1, n - 1):
                    yield
            return True

        def load_k(t):
            nonlocal used, is_k
            tl, is_k = self.tiles[t], True
            if tl["first"] and turn == 0:
                if tl["seg"] > 0:
                    n = tl["seg"] - 1
                    while not self.bar[rank]["qempty"].passes(n & 1, n):
                        yield
                assert self.q_readers == 0
                self.arm(rank, self.bar[0]["qfull"], 2)

                def store_q(k):
                    self.q[rank] = k
                self.load(rank, store_q, tl["seg"], self.bar[0]["qfull"], 1)
            for k in range(KST):
                if (yield from mine()):
                    st = used % STAGES
                    self.arm(rank, self.bar[0]["full"][st], 2)
                    self.load(rank, self.put(rank, st, ("K", t, k)), ("K", t, k),
                              self.bar[0]["full"][st], 1)
                used += 1
                yield

        is_k = True
        yield from load_k(0)
        for t, tl in enumerate(self.tiles):
            if t + 1 < len(self.tiles):
                yield from load_k(t + 1)
            is_k = False
            for j in range(tl["nb"]):
                for dh in range(2):
                    if (yield from mine()):
                        st, key = used % STAGES, ("V", t, j, dh)
                        if tl["fix"][j]:
                            bar = self.bar[rank]["fix"][st]
                            bar.arrive(1)
                            self.load(rank, self.put(rank, st, key), ("raw",) + key, bar, 1)
                        else:
                            self.arm(rank, self.bar[0]["full"][st], 2)
                            self.load(rank, self.put(rank, st, key), key,
                                      self.bar[0]["full"][st], 1)
                    used += 1
                    yield

    def fixer(self, rank):
        used, n_fix = KST, [0] * STAGES
        for t, tl in enumerate(self.tiles):
            used += KST if t + 1 < len(self.tiles) else 0
            for j in range(tl["nb"]):
                for dh in range(2):
                    st = used % STAGES
                    if tl["fix"][j]:
                        while not self.bar[rank]["fix"][st].passes(n_fix[st] & 1, n_fix[st]):
                            yield
                        n_fix[st] += 1
                        assert self.ring[rank][st] == ("raw", "V", t, j, dh)
                        self.ring[rank][st] = ("V", t, j, dh)
                        self.bar[0]["full"][st].arrive()
                        yield
                    used += 1

    # -- the MMA warp
    def mma_warp(self):
        used = 0
        both = lambda name, i=None: [b[name] if i is None else b[name][i] for b in self.bar]  # noqa: E731

        def commit(bars, after=None):
            def done():
                if after:
                    after()
                for b in bars:
                    b.arrive()
            self.mma.append(done)

        def full(key):
            st, n = used % STAGES, used // STAGES
            while not self.bar[0]["full"][st].passes(n & 1, n):
                yield
            assert self.ring[0][st] == key and self.ring[1][st] == key
            self.readers[st] += 1

        def release(st):
            def after():
                self.readers[st] -= 1
            commit(both("empty", st), after)

        def issue_s(t):
            nonlocal used
            tl = self.tiles[t]
            if tl["first"]:
                while not self.bar[0]["qfull"].passes(tl["seg"] & 1, tl["seg"]):
                    yield
            if t >= 2:
                n = (t >> 1) - 1
                while not self.bar[0]["sfree"][t & 1].passes(n & 1, n):
                    yield
            assert self.q == [tl["seg"]] * 2
            self.q_readers += 1
            for k in range(KST):
                yield from full(("K", t, k))
                release(used % STAGES)
                used += 1
                yield

            def s_done():
                for r in range(2):
                    assert self.s[r][t & 1] is None, "S overwritten before it was copied out"
                    self.s[r][t & 1] = (t, 0)
                self.q_readers -= 1
            commit(both("sfull", t & 1), s_done)
            if tl["last"]:
                commit(both("qempty"))

        yield from issue_s(0)
        for t, tl in enumerate(self.tiles):
            if t + 1 < len(self.tiles):
                yield from issue_s(t + 1)
            while not self.bar[0]["pready"].passes(t & 1, t):
                yield
            assert self.p == [[t] * 4] * 2
            self.p_readers += 1
            for j in range(tl["nb"]):
                for dh in range(2):
                    yield from full(("V", t, j, dh))
                    release(used % STAGES)
                    used += 1
                    yield

            def pv_done(t=t):
                self.p_readers -= 1
                self.done_pv.append(t)
            commit(both("pvdone"), pv_done)

    # -- a softmax warp
    def softmax(self, rank, w):
        for t, tl in enumerate(self.tiles):
            n = t >> 1
            while not self.bar[rank]["sfull"][t & 1].passes(n & 1, n):
                yield
            tile, copied = self.s[rank][t & 1]
            assert tile == t
            self.s[rank][t & 1] = (t, copied + 1) if copied < 3 else None
            self.bar[0]["sfree"][t & 1].arrive()
            yield
            self.bar[rank]["red"].arrive()
            while not self.bar[rank]["red"].passes(t & 1, t):
                yield
            if t > 0:
                while not self.bar[rank]["pvdone"].passes((t - 1) & 1, t - 1):
                    yield
            assert self.p_readers == 0, "P overwritten while a product may read it"
            self.p[rank][w] = t
            yield
            self.bar[0]["pready"].arrive()
            if tl["last"]:
                while not self.bar[rank]["pvdone"].passes(t & 1, t):
                    yield
                assert self.done_pv[-1] == t, "O read while the next segment's products run"

    def run(self):
        procs = [self.mma_warp()]
        for r in range(2):
            procs += [self.loader(r, 0), self.loader(r, 1), self.fixer(r)]
            procs += [self.softmax(r, w) for w in range(4)]
        idle = 0
        while procs:
            before = (len(self.events), len(self.mma),
                      tuple(id(x) for x in procs))
            if self.rng.random() < 0.5 and self.step_async():
                idle = 0
                continue
            i = self.rng.randrange(len(procs))
            try:
                next(procs[i])
            except StopIteration:
                procs.pop(i)
                idle = 0
                continue
            idle += 1
            if idle > 4000 and not self.events and not self.mma:
                state = [(x.__name__, x.gi_frame.f_lineno) for x in procs]
                raise AssertionError(f"no progress: {state} {before[:2]}")
            if idle > 200000:
                raise AssertionError("no progress")


def draw_tiles(rng):
    tiles, segs = [], rng.randint(1, 6)
    for s in range(segs):
        left, first = rng.randint(1, 14), True
        while left:
            nb = min(4, left)
            left -= nb
            tiles.append(dict(seg=s, first=first, last=left == 0, nb=nb,
                              fix=[left == 0 and j >= nb - 2 and rng.random() < 0.7
                                   for j in range(nb)]))
            first = False
    return tiles


@pytest.mark.parametrize("seed", range(60))
def test_protocol_under_random_interleavings(seed):
    rng = random.Random(seed)
    Model(draw_tiles(rng), seed).run()


def test_a_wait_too_far_ahead_is_found():
    """Negative control: with one loading warp for K and one for V a parity wait passes on the
    wrong phase."""
    found = 0
    for seed in range(60):
        try:
            Model(draw_tiles(random.Random(seed)), seed, planted="split").run()
        except AssertionError:
            found += 1
    assert found
