"""CPU model of the shared-prefix attention kernel's handoffs (prefix_attention.cu).

The kernel's roles -- two loading warps, two threads that issue products, the eight
softmax warps -- are run as steps in random order under mbarrier semantics: a barrier
completes a phase when its arrivals (and a copy's bytes) are in, and a wait on a parity
passes when the barrier's phase in progress has the other one. Copies land in any order
and products complete in each thread's order. The model knows what each wait means and
checks, at every step: no wait passes on a phase other than the one it is for, no
barrier gets an arrival more than it expects, no slot, Q tile, S, P or O is written while
it is read, and no interleaving stops. The same model with the second wait of the ring
taken out (planted here, in the model) is found wrong.
"""
import random

import pytest


class Fault(AssertionError):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.phase, self.left, self.copies = count, 0, count, 0

    def arrive(self, n=1, copies=0):
        if self.left < n:
            raise Fault("an arrival more than the barrier expects")
        self.left -= n
        self.copies += copies
        self.turn()

    def landed(self):
        self.copies -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.copies == 0:
            self.phase += 1
            self.left = self.count

    def passes(self, want):
        """Would a wait on the parity of phase `want` pass? It must mean that phase."""
        if self.phase % 2 == want % 2:
            return False
        if self.phase != want + 1:
            raise Fault(f"a wait for phase {want} passes in phase {self.phase}")
        return True


def k_pos(t):
    return 0 if t == 0 else 2 * t - 1


def v_pos(t, n):
    return 2 * n - 1 if t == n - 1 else 2 * t + 2


class Model:
    """jobs: (tiles, pair, tail) each; tail: the last tile is not full."""

    def __init__(self, jobs, slots, rng, second_wait=True):
        self.jobs, self.ks, self.rng, self.second_wait = jobs, slots, rng, second_wait
        self.full = [Barrier(2) for _ in range(slots)]
        self.freed = [Barrier(2) for _ in range(slots)]
        self.s_full, self.p_half, self.p_full = [Barrier(1), Barrier(1)], [Barrier(4), Barrier(4)], [Barrier(4), Barrier(4)]
        self.q_full, self.o_done, self.o_free, self.merged = Barrier(8), Barrier(2), Barrier(8), Barrier(8)
        self.turn = [Barrier(1), Barrier(1)]
        self.holds = [[None, None] for _ in range(slots)]   # (job, "K" or "V", tile) of each half that has landed
        self.flying = []                   # copies that have not landed
        self.queue = [[], []]              # products of each issuing thread, in order
        self.reading = {}                  # what unfinished products read: slot or "q" -> count
        self.q_job, self.o_job = None, [None, None]
        self.clears = {}                   # (stream, warp) -> the last tile whose tail it cleared

    def use(self, what, n):
        self.reading[what] = self.reading.get(what, 0) + n

    def landed_waits(self, pos, pair):
        """The waits for ring position `pos` to have landed."""
        at, use = pos % self.ks, pos // self.ks
        waits = [(self.full[at], use)]
        if not pair and use > 0 and self.second_wait:
            waits.insert(0, (self.freed[at], use - 1))
        return waits

    def has(self, at, what):
        return self.holds[at] == [what, what]

    def cleared(self, j, t, pos):
        """Have all warps of a stream that reads this tile cleared its tail, if it has one?"""
        n, pair, tail = self.jobs[j]
        if t < n - 1 or not tail:
            return True
        return any(all(self.clears.get((s, w)) == (j, t) for w in range(4)) for s in (0, 1))

    def loader(self, half):
        pos = 0
        for j, (n, pair, _) in enumerate(self.jobs):
            order = []
            for t in range(n):
                order.append(("K", t))
                if t:
                    order.append(("V", t - 1))
            if n:
                order.append(("V", n - 1))
            for what, t in order:
                at = pos % self.ks
                if pos >= self.ks:
                    yield (self.freed[at], pos // self.ks - 1)
                if self.reading.get(at):
                    raise Fault("a slot is filled while a product reads it")
                self.holds[at][half] = None
                self.full[at].arrive(1, copies=1)
                self.flying.append((at, half, (j, what, t)))
                pos += 1

    def issuer(self, s):
        pos0 = done = step = turns = 0
        for j, (n, pair, _) in enumerate(self.jobs):
            if n == 0:
                continue
            tiles = list(range(n)) if pair else list(range(s, n, 2))

            def s_product(i):
                t = tiles[i]
                pos = pos0 + k_pos(t)
                if not self.has(pos % self.ks, (j, "K", t)) or self.q_job != j:
                    raise Fault("S reads what is not its tile or its Q")
                self.use(pos % self.ks, 1), self.use("q", 1)
                self.queue[s].append(("S", [pos % self.ks, "q"], self.s_full[s]))

            yield (self.q_full, done)
            if tiles:
                yield from self.landed_waits(pos0 + k_pos(tiles[0]), pair)
                s_product(0)
            for i, t in enumerate(tiles):
                pos = pos0 + v_pos(t, n)
                if i + 1 < len(tiles):
                    yield from self.landed_waits(pos0 + k_pos(tiles[i + 1]), pair)
                yield from self.landed_waits(pos, pair)
                if i == 0 and done:
                    yield (self.o_free, done - 1)
                yield (self.p_half[s], step)
                if not self.has(pos % self.ks, (j, "V", t)) or not self.cleared(j, t, pos):
                    raise Fault("P V reads what is not its tile, or what lies past its keys")
                self.o_job[s] = j
                self.use(pos % self.ks, 1)
                self.queue[s].append(("PV", [pos % self.ks], None))
                if pair:
                    if s == 1 or turns > 0:
                        yield (self.turn[s], turns + s - 1)
                    turns += 1
                yield (self.p_full[s], step)
                step += 1
                self.use(pos % self.ks, 1)
                self.queue[s].append(("PV", [pos % self.ks], None))
                if i + 1 < len(tiles):
                    s_product(i + 1)
                if pair:
                    self.turn[1 - s].arrive()
            self.queue[s].append(("end", [], self.o_done))
            done += 1
            pos0 += 2 * n

    def softmax(self, s, w):
        pos0 = done = step = merges = 0
        live = [j for j, (n, _, _) in enumerate(self.jobs) if n]

        def load_q(j):
            if self.reading.get("q"):
                raise Fault("Q is written while a product reads it")
            self.q_job = j
            self.q_full.arrive()

        if live:
            load_q(live[0])
        for x, j in enumerate(live):
            n, pair, tail = self.jobs[j]
            tiles = list(range(n)) if pair else list(range(s, n, 2))
            arrivals = 1 if pair else 2
            for i, t in enumerate(tiles):
                yield (self.s_full[s], step)
                step += 1
                if w == 0:
                    self.freed[(pos0 + k_pos(t)) % self.ks].arrive(arrivals)
                    if i:
                        self.freed[(pos0 + v_pos(tiles[i - 1], n)) % self.ks].arrive(arrivals)
                if t == n - 1 and tail:
                    pos = pos0 + v_pos(t, n)
                    yield from self.landed_waits(pos, pair)
                    if not self.has(pos % self.ks, (j, "V", t)):
                        raise Fault("the tail of another tile is cleared")
                    self.clears[s, w] = (j, t)
                    yield None
                self.p_half[s].arrive()
                yield None
                self.p_full[s].arrive()
            yield (self.o_done, done)
            done += 1
            if tiles and w == 0:
                self.freed[(pos0 + v_pos(tiles[-1], n)) % self.ks].arrive(arrivals)
            pos0 += 2 * n
            if x + 1 < len(live):
                load_q(live[x + 1])
            if not pair:
                self.merged.arrive()
                yield (self.merged, merges)
                merges += 1
            for k in (s,) if pair else (0,) if n == 1 else (0, 1):   # whose O this warp reads
                if self.o_job[k] != j:
                    raise Fault("O is another job's")
            self.o_free.arrive()

    def run(self):
        roles = {("load", 0): self.loader(0), ("load", 1): self.loader(1), ("issue", 0): self.issuer(0), ("issue", 1): self.issuer(1)}
        roles.update({("softmax", s, w): self.softmax(s, w) for s in (0, 1) for w in range(4)})
        waits = {r: None for r in roles}
        speed = {r: self.rng.choice([1, 1, 4, 20]) for r in list(roles) + ["land", "product"]}
        while roles:
            ready = []
            for r in roles:
                if waits[r] is None or waits[r][0].passes(waits[r][1]):
                    ready += [r] * speed[r]
            if self.flying:
                ready += ["land"] * speed["land"]
            if self.queue[0] or self.queue[1]:
                ready += ["product"] * speed["product"]
            if not ready:
                raise Fault("nothing can go on: " + str(sorted(roles)))
            r = self.rng.choice(ready)
            if r == "land":      # any copy, or mostly the first: one may be very late
                at, half, what = self.flying.pop(0 if self.rng.random() < 0.7 else self.rng.randrange(len(self.flying)))
                self.holds[at][half] = what
                self.full[at].landed()
            elif r == "product":
                q = self.rng.choice([q for q in self.queue if q])
                _, reads, bar = q.pop(0)
                for x in reads:
                    self.use(x, -1)
                if bar is not None:
                    bar.arrive()
            else:
                try:
                    waits[r] = next(roles[r])
                except StopIteration:
                    del roles[r]


def some_jobs(rng, wide):
    jobs = []
    for _ in range(rng.randint(1, 5)):
        n = rng.choice([0, 1, 1, 2, 3, 4, 5, 8, 13])
        jobs.append((n, wide and rng.random() < 0.5, rng.random() < 0.5))
    return jobs


@pytest.mark.parametrize("slots,wide", [(5, True), (6, False), (8, True), (8, False)])
def test_no_interleaving_breaks_the_handoffs(slots, wide):
    rng = random.Random(slots * 2 + wide)
    for _ in range(700):
        Model(some_jobs(rng, wide), slots, rng).run()


@pytest.mark.parametrize("slots,wide", [(5, True), (6, False)])
def test_the_model_finds_a_missing_wait(slots, wide):
    """A stream that waits only for its own tiles can meet a slot whose last copy, the
    other stream's, has not landed: two phases behind, and its wait passes."""
    rng = random.Random(slots)
    with pytest.raises(Fault):
        for _ in range(3000):
            Model(some_jobs(rng, wide), slots, rng, second_wait=False).run()
