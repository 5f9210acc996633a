"""The barriers of the prefix attention's pair of CTAs, run on the host.

Every role of the kernel is a generator that arrives and waits as the kernel does, and the scheduler picks who goes
on: at random, with warps that lag for long stretches. Arrivals at the other CTA, TMA loads and the tensor cores' commits
are under way for any length of time (the commits of one warp reach a CTA in their order). What is checked:

- a wait by parity passes in its phase, neither one phase early nor after the barrier went on;
- what a role reads (places, operands, S, P, O, maxima) is what it was meant to read, and stays until it has been read;
- every run ends;
- nothing arrives at a CTA that has left.

What the model takes from the source are its constants and its end; the roles are written down here.
"""

import random
import re
from pathlib import Path

import pytest

import deepseek_sparse_attention_ragged_gb300 as ds

SOURCE = (Path(ds.__file__).parent / "csrc" / "prefix_attn.cu").read_text()


class Fault(AssertionError):
    pass


def check(ok, what):
    if not ok:
        raise Fault(what)


def constants():
    """What the source says: ring units, buffers, and how a CTA leaves."""
    number = lambda name: int(re.search(rf"constexpr (?:uint32_t|int) {name} = (\d+);", SOURCE)[1])  # noqa: E731
    by_form = lambda name: tuple(map(int, re.search(  # noqa: E731
        rf"{name} = kByTma<kFormat> \? (\d+) : (\d+);", SOURCE).groups()))
    end = SOURCE[:SOURCE.index("tcgen05.dealloc")]
    end = end[end.rindex("__syncthreads();"):]
    return dict(k_units=number("kKUnits"), v_units=by_form("kVUnits"), p_bufs=by_form("kPBufs"), s_bufs=number("kSBufs"),
                place_bufs=number("kPlaceBufs"), red_bufs=number("kRedBufs") if "kRedBufs =" in SOURCE else 1,
                release="cluster_arrive_release();" in end, both_drained="bar->drained" in end)


class Bar:
    def __init__(self, cta, count):
        self.cta, self.count, self.pending, self.tx, self.phase, self.name = cta, count, count, 0, 0, None

    def arrive(self, expect=0):
        check(not self.cta.left, "an arrival at a CTA that has left")
        self.tx += expect
        self.pending -= 1
        check(self.pending >= 0, "more arrivals than the phase has")
        self._turn()

    def loaded(self):
        check(not self.cta.left, "a load that ends at a CTA that has left")
        self.tx -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def seems_over(self, phase):
        """What a wait by parity sees."""
        return self.phase & 1 != phase & 1

    def over(self, phase):
        """The same for a wait that has to be exact."""
        if self.seems_over(phase):
            check(self.phase == phase + 1, f"a wait for phase {phase} passes in {self.phase}")
            return True
        check(self.phase <= phase, f"a wait for phase {phase}, but the barrier is in {self.phase}")
        return False


class Cta:
    def __init__(self, w, rank):
        self.rank, self.left, self.ended, self.under_way = rank, False, 0, 0
        b = lambda count: Bar(self, count)  # noqa: E731
        units = w.k_units + w.v_units
        tma = w.tma
        self.full = [b(2 if tma else 16) for _ in range(units)]
        self.empty = [b(1) for _ in range(units)]
        self.q_full, self.o_read, self.q_free, self.drained = b(2), b(16), b(1), b(2)
        self.p_full, self.pv_done, self.m_ready = ([b(n) for _ in range(2)] for n in (8, 1, 4))
        self.s_free, self.s_full = ([b(n) for _ in range(w.s_bufs)] for n in (8, 1))
        readers = 4 if tma else 16
        self.place_full = [b(1) for _ in range(w.place_bufs)]
        self.place_free = [b(2 * readers + 4) for _ in range(w.place_bufs)]
        self.met = [Bar(self, 4) for _ in range(2)]  # the named barriers of the softmax sets
        for name, bars in list(vars(self).items()):
            for bar in bars if isinstance(bars, list) else [bars]:
                if isinstance(bar, Bar):
                    bar.name = name
        self.ring, self.place, self.q = [{} for _ in range(units)], [None] * w.place_bufs, None
        self.p = [{} for _ in range(w.p_bufs)]
        self.s = [None] * w.s_bufs
        self.maxima = [{} for _ in range(2)]
        self.red = [[{} for _ in range(w.red_bufs)] for _ in range(2)]


class World:
    """A pair with parts of `parts` tiles each. Waits on the barriers named in `skip` are left out."""

    def __init__(self, parts, tma, rng, skip=(), **kw):
        self.__dict__.update(kw)
        self.skip = skip
        self.v_units, self.p_bufs = self.v_units[not tma], self.p_bufs[not tma]
        self.parts, self.tma, self.rng, self.n = parts, tma, rng, sum(parts)
        self.ctas = [Cta(self, rank) for rank in range(2)]
        self.pool = []           # what is under way: (priority, action)
        self.queues = [[], []]   # the issuing warps' MMAs and commits
        self.commits = {}        # commits under way to a CTA, in order, by (queue, rank)
        self.pv_running = 0
        self.pv_tile, self.o_reads = -1, 16
        self.tiles = [(k, i, at) for at, (k, i) in enumerate((k, i) for k, p in enumerate(parts) for i in range(p))]
        self.by_threads = [rng.random() < 0.3 for _ in range(self.n)]

    # ---- asynchronous parts
    def later(self, action):
        self.pool.append([self.rng.random(), action])

    def remote(self, cta, bar, expect=0):
        """An arrival at the first CTA from a thread of `cta`: its own, or under way."""
        if cta.rank == 0:
            bar.arrive(expect)
            return
        cta.under_way += 1

        def land():
            bar.arrive(expect)
            cta.under_way -= 1
        self.later(land)

    def commit(self, queue, name, ranks=(0, 1)):
        self.queues[queue].append(("commit", name, ranks))

    def engine(self, queue):
        kind, *rest = self.queues[queue].pop(0)
        if kind == "mma":
            rest[0]()
            return
        name, ranks = rest
        for rank in ranks:
            line = self.commits.setdefault((queue, rank), [])
            line.append(name)

    def land_commit(self, key):
        name = self.commits[key].pop(0)
        bar = getattr(self.ctas[key[1]], name[0])
        (bar if len(name) == 1 else bar[name[1]]).arrive()

    # ---- roles
    def places(self, c):
        for it in range(self.n):
            b, lap = it % self.place_bufs, it // self.place_bufs
            yield c.place_free[b], lap - 1
            c.place[b] = None
            yield
            c.place[b] = it
            c.place_full[b].arrive()

    def queries(self, c):
        for k in range(len(self.parts)):
            if k:
                yield c.q_free, k - 1
            c.q = None
            self.remote(c, self.ctas[0].q_full, 1)
            yield

            def loaded(k=k):
                c.q = k
                self.ctas[0].q_full.loaded()
            self.later(loaded)

    def poll(self, bars, phases, u, units, bits):
        """The lanes' look at all units of a form together: returns the units that are known to be full."""
        for lane in range(4):
            if lane < u + units and bars[lane].seems_over(phases[lane]):
                bits.add(lane)
                if lane >= u:
                    check(bars[lane].phase == phases[lane] + 1, "a unit that is taken for full")
            else:
                bits.discard(lane)

    def issue_s(self):
        first = self.ctas[0]
        for k, i, it in self.tiles:
            if i == 0:
                yield first.q_full, k
            s = it % self.s_bufs
            yield first.s_free[s], it // self.s_bufs - 1
            full = set()
            for u in range(4):
                while u not in full:
                    self.poll(first.full[:4], [it] * 4, u, self.k_units, full)
                    yield "again"
                for c in self.ctas:
                    check(c.ring[u] == {j: ("K", it, u) for j in self.steps}, f"K unit {u} of tile {it}: {c.ring[u]}")
                    check(c.q == k, "the query of another part")
                    c.s[s] = None

                def done(u=u, s=s, it=it, k=k):
                    for c in self.ctas:
                        check(c.ring[u] == {j: ("K", it, u) for j in self.steps} and c.q == k, "an operand of S went away")
                        if u == 3:
                            c.s[s] = it
                self.queues[0].append(("mma", done))
                self.commit(0, ("empty", u))
                if u == 3:
                    self.commit(0, ("s_full", s))
                    if i + 1 == self.parts[k]:
                        self.commit(0, ("q_free",))
                yield
        yield from self.drain(0)

    def issue_pv(self):
        first = self.ctas[0]
        for k, i, it in self.tiles:
            yield first.p_full[it & 1], it >> 1
            if i == 0 and k > 0:
                yield first.o_read, k - 1
            if i == 0:
                check(self.o_reads == 16, "O begins anew before it was read")
                self.o_reads = 0
            in_k = self.tma and it + 1 == self.n
            slots = [v if in_k else self.k_units + (4 * it + v) % self.v_units for v in range(4)]
            phases = [self.n if in_k else (4 * it + v) // self.v_units for v in range(4)]
            full = set()
            for v in range(4):
                while v not in full:
                    self.poll([first.full[x] for x in slots], phases, v, self.k_units if in_k else self.v_units, full)
                    yield "again"
                b = it % self.p_bufs

                def there(v=v, it=it, b=b, slot=slots[v]):
                    return all(c.ring[slot] == {j: ("V", it, v) for j in self.steps} and
                               c.p[b] == {w: it for w in range(4)} for c in self.ctas)
                check(there(), f"V unit {v} or P of tile {it}")
                self.pv_running += 1

                def done(v=v, it=it, there=there):
                    check(there(), "an operand of P G went away")
                    self.pv_running -= 1
                    if v == 3:
                        self.pv_tile = it
                self.queues[1].append(("mma", done))
                self.commit(1, ("empty", slots[v]))
                if v == 3:
                    self.commit(1, ("pv_done", it & 1))
                yield
        yield from self.drain(1)

    def drain(self, queue):
        self.commit(queue, ("drained",))
        yield self.ctas[0].drained, 0

    def softmax(self, c, sm, w):
        first, other = self.ctas[0], sm ^ 1
        for k, count in enumerate(self.parts):
            begin = sum(self.parts[:k])
            last = begin + count - 1
            for it in range(begin, begin + count):
                if it & 1 != sm:
                    continue
                place, s = it % self.place_bufs, it % self.s_bufs
                read = lambda: check(c.s[s] == it and c.place[place] == it, f"S or places of tile {it}")  # noqa: E731
                yield c.place_full[place], it // self.place_bufs
                yield c.s_full[s], it // self.s_bufs
                read()
                yield
                read()
                yield from self.exchange(c, sm, w, it)
                if it > 0:
                    yield c.m_ready[other], (it - 1) >> 1
                    check(c.maxima[other].get(w) == it - 1, "the maximum of another tile")
                c.maxima[sm][w] = it
                yield
                c.m_ready[sm].arrive()
                read()
                yield
                had = it - self.p_bufs
                if had >= 0:
                    yield c.pv_done[had & 1], had >> 1
                read()
                yield
                self.remote(c, first.s_free[s])
                c.place_free[place].arrive()
                b = it % self.p_bufs
                c.p[b][w] = None
                yield
                c.p[b][w] = it
                if it > begin and self.rng.random() < 0.5:
                    yield c.pv_done[other], (it - 1) >> 1
                    check(self.pv_running == 0 and self.pv_tile == it - 1, "O is scaled while it is written")
                    yield
                    check(self.pv_running == 0 and self.pv_tile == it - 1, "O is scaled while it is written")
                yield
                self.remote(c, first.p_full[sm])
            if last & 1 != sm:
                yield c.m_ready[other], last >> 1
                check(c.maxima[other].get(w) == last, "the last maximum")
                if self.p_bufs == 2 and last > 0:
                    yield c.pv_done[sm], (last - 1) >> 1
            yield c.pv_done[last & 1], last >> 1
            for _ in range(2):
                check(self.pv_running == 0 and self.pv_tile == last, "O is read while it is written")
                yield
            self.o_reads += 1
            self.remote(c, first.o_read)

    def exchange(self, c, sm, w, it):
        """The two threads of a head, in warps w and w ^ 2, take the larger maximum."""
        red = c.red[sm][it // 2 % self.red_bufs]
        red[w] = it
        c.met[sm].arrive()
        yield c.met[sm], it >> 1
        check(red[w ^ 2] == it, f"the other half's largest logit is tile {red[w ^ 2]}'s, not {it}'s")

    @property
    def steps(self):
        return range(1 if self.tma else 8)

    def load_by_tma(self, c, slot):
        first, n, kv = self.ctas[0], self.n, self.v_units
        lap = 0
        while True:
            v_unit = slot >= self.k_units
            g = slot - self.k_units + lap * kv if v_unit else 4 * min(lap, n - 1) + slot
            of, u = g // 4, g % 4
            if n == 0 or (of + 1 >= n if v_unit else lap > n):
                return
            v_form = v_unit or lap == n
            yield c.place_full[of % self.place_bufs], of // self.place_bufs
            read = lambda: check(c.place[of % self.place_bufs] == of, "the places of another tile")  # noqa: E731
            read()
            yield c.empty[slot], lap - 1
            tag = ("V" if v_form else "K", of, u)
            c.ring[slot] = {}
            if not self.by_threads[of]:
                self.remote(c, first.full[slot], 1)
                yield
                read()

                def loaded(slot=slot, tag=tag):
                    c.ring[slot] = {0: tag}
                    first.full[slot].loaded()
                self.later(loaded)
                c.place_free[of % self.place_bufs].arrive()
            else:
                yield
                read()
                c.place_free[of % self.place_bufs].arrive()
                yield
                c.ring[slot] = {0: tag}
                self.remote(c, first.full[slot])
            lap += 1

    def load_packed(self, c, team, s):
        first, n = self.ctas[0], self.n
        tile_of = lambda f: 0 if f == 0 else n - 1 if f == 2 * n - 1 else (f + 1) // 2 if f & 1 else f // 2 - 1  # noqa: E731
        v_form_of = lambda f: f == 2 * n - 1 or (f > 0 and not f & 1)  # noqa: E731

        def looked_up(of):
            return c.place_full[of % self.place_bufs], of // self.place_bufs

        def fetch(f):
            check(c.place[tile_of(f) % self.place_bufs] == tile_of(f), "the places of another tile")
        if n == 0:
            return
        yield looked_up(0)
        fetch(0)
        c.place_free[0].arrive()
        for f in range(2 * n):
            then = f + 1 < 2 * n
            if then:
                yield looked_up(tile_of(f + 1))
            for k in range(2):
                u = team + 2 * k
                slot = (self.k_units if v_form_of(f) else 0) + u
                yield c.empty[slot], tile_of(f) - 1
                c.ring[slot][s] = None
                yield
                c.ring[slot][s] = ("V" if v_form_of(f) else "K", tile_of(f), u)
                if then:
                    fetch(f + 1)
                self.remote(c, first.full[slot])
            if then:
                c.place_free[tile_of(f + 1) % self.place_bufs].arrive()

    def leave(self, c):
        """__syncthreads, then the pair's barrier."""
        while c.ended < self.roles:
            yield "again"
        if self.both_drained:
            yield c.drained, 0
        while self.release and c.under_way:
            yield "again"
        c.said = True
        while not all(getattr(x, "said", False) for x in self.ctas):
            yield "again"
        yield
        c.left = True

    def run(self):
        procs = []
        for c in self.ctas:
            mine = [self.places(c), self.queries(c)]
            mine += [self.softmax(c, sm, w) for sm in range(2) for w in range(4)]
            if self.tma:
                mine += [self.load_by_tma(c, slot) for slot in range(self.k_units + self.v_units)]
            else:
                mine += [self.load_packed(c, team, s) for team in range(2) for s in range(8)]
            if c.rank == 0:
                mine += [self.issue_s(), self.issue_pv()]
            else:
                mine += [iter(()), iter(())]
            self.roles = len(mine)
            procs += [[self.rng.random(), p, None, c] for p in mine] + [[self.rng.random(), self.leave(c), None, None]]
        rng, idle, held = self.rng, 0, set()
        while procs or self.pool or any(self.queues) or any(self.commits.values()):
            if rng.random() < 0.02:  # others lag from here on
                for x in procs + self.pool:
                    x[0] = rng.random()
                held = {(q, rank) for q in range(2) for rank in range(2) if rng.random() < 0.3}
            ready = [x for x in procs if not isinstance(x[2], tuple) or x[2][0].name in self.skip or x[2][0].over(x[2][1])]
            running = [x for x in ready if x[2] != "again"]
            events = [(q,) for q in range(2) if self.queues[q]] + [k for k, v in self.commits.items() if v]
            check(ready or self.pool or events, "nothing can go on")
            if running or self.pool:
                events = [e for e in events if e not in held]
            idle = 0 if running or self.pool or events else idle + 1
            check(idle < 1000, "nothing goes on")
            kind = rng.random()
            if self.pool and (kind < 0.2 or not ready):
                x = max(self.pool, key=lambda x: x[0]) if rng.random() < 0.7 else rng.choice(self.pool)
                self.pool = [y for y in self.pool if y is not x]
                x[1]()
            elif events and (kind < 0.4 or not ready):
                e = rng.choice(events)
                self.engine(e[0]) if len(e) == 1 else self.land_commit(e)
            elif ready:
                some = running if running and rng.random() < 0.8 else ready
                x = max(some, key=lambda x: x[0]) if rng.random() < 0.9 else rng.choice(some)
                try:
                    x[2] = next(x[1])
                except StopIteration:
                    procs = [y for y in procs if y is not x]
                    if x[3] is not None:
                        x[3].ended += 1
        check(self.pv_tile == self.n - 1, "not every tile was done")


CASES = [[], [1], [2], [3], [1, 1], [1, 2], [2, 1, 1], [4, 1], [5], [3, 4, 1], [9], [1, 1, 1, 1, 1], [6, 6], [11]]


def many(tma, runs, seed, **changed):
    rng = random.Random(seed)
    for _ in range(runs):
        World(rng.choice(CASES), tma, random.Random(rng.random()), **{**constants(), **changed}).run()


@pytest.mark.parametrize("tma", [True, False])
def test_every_order_of_the_roles_is_sound(tma):
    many(tma, 60, 1)


@pytest.mark.parametrize("changed", [dict(release=False), dict(both_drained=False)])
def test_an_exit_that_leaves_arrivals_behind_is_found(changed):
    with pytest.raises(Fault, match="has left"):
        many(True, 400, 2, **{**dict(release=True, both_drained=True), **changed})


def test_one_copy_of_the_largest_logits_is_overwritten():
    """(With packed rows, which wait for each other's tiles more often, it takes more orders to see it.)"""
    with pytest.raises(Fault, match="other half"):
        many(True, 400, 4, red_bufs=1)


@pytest.mark.parametrize("wait", ["place_full", "place_free", "empty", "q_full", "q_free", "s_full", "p_full", "pv_done", "m_ready",
                                  "o_read"])
@pytest.mark.parametrize("tma", [True, False])
def test_a_wait_that_is_left_out_is_found(tma, wait):
    """(Not s_free: with four places and four S, a tile is not looked up before the S that it takes has been read.)"""
    with pytest.raises(Fault):
        many(tma, 200, 3, skip=(wait,))
