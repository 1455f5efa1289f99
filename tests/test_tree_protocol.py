"""A model of the tree-attention kernel's barrier protocol (csrc/tree_tc.cu) under random
interleavings: two CTAs, each with a loading warp for Q and K, one for V, four softmax and four
finishing warps, and the first CTA's two MMA warps (scores; P . V). Loads land and MMAs complete after random delays. Checked:
no deadlock, no parity wait that passes on the wrong phase, no stage refilled or buffer
overwritten while a product may still read it, and every product reads what it should."""
import random

import pytest

K_RING, V_RING, KST = 4, 3, 9


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
        many = lambda n, c: [Barrier(c) for _ in range(n)]  # noqa: E731
        self.bar = [dict(kfull=many(K_RING, 1), vfull=many(V_RING, 8), qfull=Barrier(1),
                         sfree=many(2, 8), pready=[Barrier(8), Barrier(4)], kempty=many(K_RING, 1),
                         vempty=many(V_RING, 1), qempty=Barrier(1), sfull=many(2, 1),
                         pvdone=many(2, 1), red=Barrier(4), sum=Barrier(4), fix=many(V_RING, 1),
                         ofree=Barrier(8), lready=many(2, 2), segdone=Barrier(1))
                    for _ in range(2)]
        self.ring = [dict(k=[None] * K_RING, v=[None] * V_RING) for _ in range(2)]
        self.readers = dict(k=[0] * K_RING, v=[0] * V_RING)  # products that may still read
        self.q, self.q_readers = [None, None], 0
        self.s = [[None, None], [None, None]]             # S buffers of each CTA
        self.p, self.p_readers = [[None] * 4, [None] * 4], [0, 0]
        self.rescaled = [[None] * 4, [None] * 4]
        self.inv, self.o_readers = [[None, None], [None, None]], 0
        self.events = []                                  # landing loads
        self.mma = [[], []]                               # each MMA warp's products, in order
        self.done_pv = []

    # -- asynchronous engines
    def load(self, store, key, bar):
        def land():
            store(key)
            bar.complete(1)
        self.events.append(land)

    def step_async(self):
        choices = [q for q in ([self.events] if self.events else []) + self.mma if q]
        if not choices:
            return False
        q = self.rng.choice(choices)
        q.pop(self.rng.randrange(len(q)) if q is self.events else 0)()
        return True

    def wait(self, bar, phase):
        while not bar.passes(phase & 1, phase):
            yield

    def put(self, rank, ring, st, key):
        assert self.readers[ring][st] == 0, "a stage is refilled while a product may read it"
        self.ring[rank][ring][st] = ("landing", key)

        def store(k):
            self.ring[rank][ring][st] = k
        return store

    # -- one CTA's loading warps
    def load_k(self, rank):
        used = 0
        for t, tl in enumerate(self.tiles):
            if tl["first"]:
                if tl["seg"] > 0 and self.planted != "q":
                    yield from self.wait(self.bar[rank]["qempty"], tl["seg"] - 1)
                assert self.q_readers == 0, "Q is replaced while a product may read it"
                if rank == 0:
                    self.bar[0]["qfull"].arrive(2)

                def store_q(k):
                    self.q[rank] = k
                self.load(store_q, tl["seg"], self.bar[0]["qfull"])
            for k in range(KST):
                st, n = used % K_RING, used // K_RING
                if n > 0:
                    yield from self.wait(self.bar[rank]["kempty"][st], n - 1)
                if rank == 0:
                    self.bar[0]["kfull"][st].arrive(2)
                self.load(self.put(rank, "k", st, (t, k)), (t, k), self.bar[0]["kfull"][st])
                used += 1
                yield

    def load_v(self, rank):
        used = 0
        for t, tl in enumerate(self.tiles):
            for j in range(tl["nb"]):
                for dh in range(2):
                    st, n = used % V_RING, used // V_RING
                    if n > 0:
                        yield from self.wait(self.bar[rank]["vempty"][st], n - 1)
                    key, bar = (t, j, dh), self.bar[0]["vfull"][st]
                    if tl["fix"][j]:
                        bar = self.bar[rank]["fix"][st]
                        bar.arrive(1)
                        key = ("raw",) + key
                    elif rank == 0:
                        for _ in range(7):
                            bar.arrive()
                        bar.arrive(2)
                    self.load(self.put(rank, "v", st, key), key, bar)
                    used += 1
                    yield

    def finisher(self, rank, w):
        used, n_fix = 0, [0] * V_RING
        for t, tl in enumerate(self.tiles):
            for j in range(tl["nb"]):
                for dh in range(2):
                    st, key = used % V_RING, (t, j, dh)
                    if tl["fix"][j]:
                        yield from self.wait(self.bar[rank]["fix"][st], n_fix[st])
                        n_fix[st] += 1
                        held = self.ring[rank]["v"][st]
                        part = 1 if held == ("raw",) + key else held[1] + 1
                        assert part == 1 or held == ("fixed", part - 1) + key
                        self.ring[rank]["v"][st] = key if part == 4 else ("fixed", part) + key
                        self.bar[0]["vfull"][st].arrive()
                        yield
                    used += 1
            if tl["last"]:
                yield from self.wait(self.bar[rank]["lready"][tl["seg"] & 1], tl["seg"] >> 1)
                yield from self.wait(self.bar[rank]["segdone"], tl["seg"])
                assert self.done_pv[-1] == t, "O read while the next segment's products run"
                assert self.inv[rank][tl["seg"] & 1] == tl["seg"]
                yield
                assert self.done_pv[-1] == t and self.o_readers == 0
                self.bar[0]["ofree"].arrive()

    # -- the MMA warps
    def commit(self, w, name, i=None, after=None):
        bars = [b[name] if i is None else b[name][i] for b in self.bar]

        def done():
            if after:
                after()
            for b in bars:
                b.arrive()
        self.mma[w].append(done)

    def use(self, w, ring, used, key):
        size = K_RING if ring == "k" else V_RING
        st, n = used % size, used // size
        yield from self.wait(self.bar[0][ring + "full"][st], n)
        assert self.ring[0][ring][st] == key and self.ring[1][ring][st] == key
        self.readers[ring][st] += 1

        def after():
            self.readers[ring][st] -= 1
        self.commit(w, ring + "empty", st, after)
        yield

    def mma_s(self):
        used = 0
        for t, tl in enumerate(self.tiles):
            if tl["first"]:
                yield from self.wait(self.bar[0]["qfull"], tl["seg"])
            if t >= 2:
                yield from self.wait(self.bar[0]["sfree"][t & 1], (t >> 1) - 1)
            assert self.q == [tl["seg"]] * 2
            self.q_readers += 1
            for k in range(KST):
                yield from self.use(0, "k", used, (t, k))
                used += 1

            def s_done(t=t):
                for r in range(2):
                    assert self.s[r][t & 1] is None, "S overwritten before it was copied out"
                    self.s[r][t & 1] = (t, 0)
                self.q_readers -= 1
            self.commit(0, "sfull", t & 1, s_done)
            if tl["last"]:
                self.commit(0, "qempty")

    def mma_pv(self):
        used = 0
        for t, tl in enumerate(self.tiles):
            hb = 2 if tl["nb"] > 2 else 1
            if tl["first"] and tl["seg"] > 0 and self.planted != "o":
                yield from self.wait(self.bar[0]["ofree"], tl["seg"] - 1)
            for half in range(2):
                yield from self.wait(self.bar[0]["pready"][half], t)
                assert [p[2 * half:2 * half + 2] for p in self.p] == [[t] * 2] * 2
                assert min(map(min, self.rescaled)) >= t, "O used before it was rescaled"
                self.p_readers[half] += 1
                self.o_readers += 1
                for j in range(half * hb, min(hb, tl["nb"]) if half == 0 else tl["nb"]):
                    for dh in range(2):
                        yield from self.use(1, "v", used, (t, j, dh))
                        used += 1

                def pv_done(t=t, half=half):
                    self.p_readers[half] -= 1
                    self.o_readers -= 1
                    if half:
                        self.done_pv.append(t)
                self.commit(1, "pvdone", half, pv_done)
                if half and tl["last"]:
                    self.commit(1, "segdone")

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
            yield from self.wait(self.bar[rank]["red"], t)
            half = w // 2
            rescale = not tl["first"] and tl["rescale"]
            if t > 0 and self.planted != "p":
                yield from self.wait(self.bar[rank]["pvdone"][0], t - 1)
                if rescale:
                    yield from self.wait(self.bar[rank]["pvdone"][1], t - 1)
            if rescale and self.planted != "p":
                assert self.done_pv[-1] == t - 1 and self.p_readers == [0, 0]
            self.rescaled[rank][w] = t
            if half == 1:
                self.bar[0]["pready"][0].arrive()
                yield
                if t > 0 and self.planted != "p":
                    yield from self.wait(self.bar[rank]["pvdone"][1], t - 1)
            assert self.p_readers[half] == 0, "P overwritten while a product may read it"
            self.p[rank][w] = t
            yield
            self.bar[0]["pready"][half].arrive()
            if tl["last"]:
                self.bar[rank]["sum"].arrive()
                yield from self.wait(self.bar[rank]["sum"], tl["seg"])
                if half == 0:
                    self.inv[rank][tl["seg"] & 1] = tl["seg"]
                    self.bar[rank]["lready"][tl["seg"] & 1].arrive()

    def run(self):
        procs = [self.mma_s(), self.mma_pv()]
        for r in range(2):
            procs += [self.load_k(r), self.load_v(r)]
            procs += [self.finisher(r, w) for w in range(4)]
            procs += [self.softmax(r, w) for w in range(4)]
        # some warps, and the loads, may be much slower than others
        pace = {id(x): self.rng.choice([1.0, 1.0, 0.3, 0.03]) for x in procs}
        engines = self.rng.choice([0.5, 0.9, 0.05])
        idle = 0
        while procs:
            if self.rng.random() < engines and self.step_async():
                idle = 0
                continue
            i = self.rng.randrange(len(procs))
            if self.rng.random() > pace[id(procs[i])]:
                continue
            try:
                next(procs[i])
            except StopIteration:
                procs.pop(i)
                idle = 0
                continue
            idle += 1
            if idle > 60000 and not self.events and not any(self.mma):
                state = [(x.__name__, x.gi_frame.f_lineno) for x in procs]
                raise AssertionError(f"no progress: {state}")
            if idle > 2000000:
                raise AssertionError("no progress")


def draw_tiles(rng):
    tiles, segs = [], rng.randint(1, 6)
    for s in range(segs):
        left, first = rng.randint(1, 14), True
        while left:
            nb = min(4, left)
            left -= nb
            tiles.append(dict(seg=s, first=first, rescale=rng.random() < 0.3, last=left == 0, nb=nb,
                              fix=[left == 0 and j >= nb - 2 and rng.random() < 0.7
                                   for j in range(nb)]))
            first = False
    return tiles


@pytest.mark.parametrize("seed", range(60))
def test_protocol_under_random_interleavings(seed):
    rng = random.Random(seed)
    Model(draw_tiles(rng), seed).run()


@pytest.mark.parametrize("planted", ["q", "p", "o"])
def test_a_missing_wait_is_found(planted):
    """Negative controls: Q replaced, P written and O begun anew without their waits."""
    found = 0
    for seed in range(40):
        try:
            Model(draw_tiles(random.Random(seed)), seed, planted=planted).run()
        except AssertionError:
            found += 1
    assert found
