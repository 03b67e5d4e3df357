"""Event model of the tensor-core window attention's barrier protocol
(csrc/window_fwd_sm100.cu), on the CPU.

Every role of a CTA -- the loader, the two MMA issuers, the eight softmax warps
-- is a generator that waits on mbarriers (by parity, as the hardware does),
works for a random time and arrives; copies and MMAs finish some random time
after they are issued, an issuer's MMAs in order.  Each access to a buffer
checks that it finds what it should: a ring slot or a Q buffer the tile it
wants, until it is done with it; the S columns the scores or the weights of the
right key tile; O the sum through the right one.  Random timing over many items
must neither trip a check nor stop (a wait for a phase that has gone by never
ends).  Planted mistakes must be caught, one of them the kernel's own first
protocol, in which the last PV signalled on the barrier of S."""
import heapq
import random

import pytest


class Stuck(Exception):
    pass


class Wrong(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase, self.waiters = count, count, 0, []

    def passed(self, parity):  # the phase of that parity is done
        return (self.phase & 1) != parity


class Sim:
    def __init__(self, seed, items, stages, mistake=None):
        self.rng, self.mistake, self.items, self.ST = random.Random(seed), mistake, items, stages
        self.now, self.seq, self.events = 0.0, 0, []
        two = 1 if mistake == "one_free" else 2
        self.bar = {("qfull", x): Bar(1) for x in (0, 1)}
        self.bar.update({("qfree", x): Bar(1) for x in (0, 1)})
        for s in range(stages):
            self.bar["full", s], self.bar["free", s] = Bar(1), Bar(two)
        for x in (0, 1):
            self.bar["s", x], self.bar["o", x] = Bar(1), Bar(1)
            for h in (0, 1):
                self.bar["p", x, h] = Bar(4)
        self.slot = [None] * stages           # what a ring slot holds
        self.users = [0] * stages             # MMAs in flight that read it
        self.q = [None, None]
        self.quse = [0, 0]
        self.s = [None, None]                 # ("S" or "P", item, e)
        self.o = [None, None]                 # (item, number of key tiles summed)
        self.tail = [0.0, 0.0]                # when the issuer's last MMA is done
        self.live = 0

    def at(self, t, f):
        self.seq += 1
        heapq.heappush(self.events, (t, self.seq, f))

    def arrive(self, name):
        b = self.bar[name]
        b.left -= 1
        if b.left == 0:
            b.left = b.count
            b.phase += 1
            ready, b.waiters = b.waiters, []
            for parity, go in ready:
                if b.passed(parity):
                    self.at(self.now + self.rng.expovariate(1 / 50), go)
                else:
                    b.waiters.append((parity, go))

    def spawn(self, gen):
        self.live += 1

        def step():
            try:
                kind, *rest = next(gen)
            except StopIteration:
                self.live -= 1
                return
            if kind == "work":
                self.at(self.now + rest[0], step)
            else:
                name, parity = rest
                b = self.bar[name]
                if b.passed(parity):
                    self.at(self.now + 1, step)
                else:
                    # a waiter looks again only after a while: it may miss a phase
                    b.waiters.append((parity, lambda: self.retry(name, parity, step)))

        self.at(self.now, step)

    def retry(self, name, parity, step):
        b = self.bar[name]
        if b.passed(parity):
            step()
        else:
            b.waiters.append((parity, lambda: self.retry(name, parity, step)))

    def run(self):
        while self.events:
            self.now, _, f = heapq.heappop(self.events)
            f()
        if self.live:
            raise Stuck(f"{self.live} roles wait for ever")

    # ---------------------------------------------------------------- roles
    def rnd(self, mean):
        return ("work", self.rng.expovariate(1 / mean))

    def loader(self):
        issued = items = 0
        for n, _ in self.items:
            if n == 0:
                continue

            def load_q(x, item):
                if items > 0:
                    yield "wait", ("qfree", x), (items - 1) & 1
                if self.quse[x]:
                    raise Wrong("Q overwritten while an MMA reads it")
                self.q[x] = None

                def land():
                    self.q[x] = item
                    self.arrive(("qfull", x))
                self.at(self.now + self.rng.expovariate(1 / 800), land)

            yield from load_q(0, items)
            for e in range(2 * n):
                if e == 1:
                    yield from load_q(1, items)
                is_k = e == 0 or (e & 1 and e < 2 * n - 1)
                blk = (e + 1) // 2 if is_k else (n - 1 if e == 2 * n - 1 else e // 2 - 1)
                st = issued % self.ST
                yield "wait", ("free", st), ((issued // self.ST) & 1) ^ 1
                if self.users[st]:
                    raise Wrong("a ring slot refilled while an MMA reads it")
                self.slot[st] = None

                def land(st=st, what=("K" if is_k else "V", items, blk)):
                    self.slot[st] = what
                    self.arrive(("full", st))
                self.at(self.now + self.rng.expovariate(1 / 900), land)
                issued += 1
                yield self.rnd(20)
            items += 1

    def mma(self, x, time, begin, end):
        """Issues one batch of MMAs on issuer x; begin and end check its buffers."""
        start = max(self.now, self.tail[x])
        self.tail[x] = start + self.rng.expovariate(1 / time)
        self.at(start, begin)
        self.at(self.tail[x], end)

    def commit(self, x, name):
        self.at(max(self.now, self.tail[x]) + 1, lambda: self.arrive(name))

    def use_slot(self, st, what):
        def begin():
            if self.slot[st] != what:
                raise Wrong(f"slot {st} holds {self.slot[st]}, not {what}")
            self.users[st] += 1

        def end():
            if self.slot[st] != what:
                raise Wrong("slot changed under an MMA")
            self.users[st] -= 1
        return begin, end

    def issuer(self, x):
        ring = ring_ph = p_ph = q_ph = 0
        items = -1

        def adv(st, ph, by):
            st += by
            return (st - self.ST, ph ^ 1) if st >= self.ST else (st, ph)

        for n, active in self.items:
            if n == 0:
                continue
            items += 1
            item = items
            mine = [e for e in range(n) if active[x][e]]
            yield "wait", ("qfull", x), q_ph
            q_ph ^= 1
            ks, kph = vs, vph = ring, ring_ph
            pend, summed = False, 0
            for e in range(n + 1):
                if e == 1:
                    ks, kph = adv(ks, kph, 1)
                    vs, vph = adv(vs, vph, 1 if n == 1 else 2)
                elif e > 1:
                    ks, kph = adv(ks, kph, 2)
                    vs, vph = adv(vs, vph, 1 if e == n else 2)
                if e < n:
                    yield "wait", ("full", ks), kph
                if e > 0:
                    yield "wait", ("full", vs), vph
                act = e < n and active[x][e]
                if pend:
                    for h in (0, 1):
                        yield "wait", ("p", x, h), p_ph
                        sb, se = self.use_slot(vs, ("V", item, e - 1))

                        def begin(e=e, h=h, sb=sb, item=item):
                            sb()
                            if self.s[x] != ("P", item, e - 1) and self.s[x] != ("half", item, e - 1):
                                raise Wrong(f"PV reads {self.s[x]}")
                            if h == 1 and self.s[x][0] != "P":
                                raise Wrong("PV reads weights that are not written")

                        def end(e=e, h=h, se=se, k=summed, item=item):
                            se()
                            if h == 1:
                                if k > 0 and self.o[x] != (item, k):
                                    raise Wrong(f"O holds {self.o[x]}, not {k} tiles of item {item}")
                                if k == 0 and self.o[x] is not None and self.o[x][0] == item - 1 and self.o[x][1] > 0:
                                    raise Wrong("O overwritten before it was read out")
                                self.o[x] = (item, k + 1)
                        self.mma(x, 250, begin, end)
                        yield self.rnd(100)
                    p_ph ^= 1
                    summed += 1
                if act:
                    sb, se = self.use_slot(ks, ("K", item, e))

                    def begin(sb=sb, item=item):
                        sb()
                        if self.q[x] != item:
                            raise Wrong("S from the wrong Q")
                        self.quse[x] += 1

                    def end(e=e, se=se, item=item):
                        se()
                        self.quse[x] -= 1
                        self.s[x] = ("S", item, e)
                    self.mma(x, 500, begin, end)
                    self.commit(x, ("s", x))
                elif pend and e > mine[-1]:
                    self.commit(x, ("s", x) if self.mistake == "last_pv_on_s" else ("o", x))
                pend = act
                if e > 0 and not (self.mistake == "free_early" and e > 1):
                    self.commit(x, ("free", vs))
                if e < n:
                    if self.mistake == "free_early":
                        self.arrive(("free", ks))
                        if e > 0:
                            self.arrive(("free", vs))
                    else:
                        self.commit(x, ("free", ks))
                elif self.mistake == "free_early" and e > 1:
                    self.arrive(("free", vs))
                if e == n - 1:
                    self.commit(x, ("qfree", x))
                yield self.rnd(60)
            ring, ring_ph = adv(vs, vph, 1)

    def softmax(self, x, warp):
        seen = o_ph = 0
        items = -1
        for n, active in self.items:
            if n == 0:
                continue
            items += 1
            item = items
            mine = [e for e in range(n) if active[x][e]]
            for k, e in enumerate(mine):
                yield "wait", ("s", x), seen & 1
                seen += 1
                if self.s[x] != ("S", item, e):
                    raise Wrong(f"softmax of item {item} tile {e} finds {self.s[x]}")
                if k > 0 and self.rng.random() < 0.3 and self.o[x] != (item, k):
                    raise Wrong(f"rescale finds O {self.o[x]}, not {k} tiles")
                yield self.rnd(300 * (6 if self.rng.random() < 0.03 else 1))  # now and then a slow warp
                for h in (0, 1):
                    yield self.rnd(600)
                    self.done[x, item, e, h] = self.done.get((x, item, e, h), 0) + 1
                    if self.done[x, item, e, h] == 4:  # the last of the four warps has written
                        self.s[x] = ("half" if h == 0 else "P", item, e)
                    self.arrive(("p", x, h))
                    if h == 0 and self.mistake == "p_once":
                        self.arrive(("p", x, 1))
            if mine:
                name = ("s", x) if self.mistake == "last_pv_on_s" else ("o", x)
                yield "wait", name, (seen & 1) if name[0] == "s" else o_ph
                if name[0] == "s":
                    seen += 1
                o_ph ^= 1
                if self.o[x] != (item, len(mine)):
                    raise Wrong(f"output reads {self.o[x]}")
                yield self.rnd(500)
                if self.o[x] != (item, len(mine)):
                    raise Wrong("O changed while it was read out")
                self.read[x, item] = self.read.get((x, item), 0) + 1
                if self.read[x, item] == 4:
                    self.o[x] = (item, 0)

    def go(self):
        self.done, self.read = {}, {}
        self.spawn(self.loader())
        for x in (0, 1):
            self.spawn(self.issuer(x))
            for w in range(4):
                self.spawn(self.softmax(x, w))
        self.run()


def make_items(rng, count):
    """Key tiles of the items, and which of them each query tile needs: the
    sinks for both, the second tile's window one further on, empty tiles."""
    items = []
    for _ in range(count):
        sinks, width = rng.choice([0, 0, 1, 2]), rng.choice([1, 1, 2, 3, 5, 9])
        a = [True] * sinks + [True] * width + [False]
        b = [True] * sinks + [False] + [True] * width
        kind = rng.random()
        if kind < 0.15:       # a single query tile, or a second one without keys
            a, b = [True] * (sinks + width), [False] * (sinks + width)
        elif kind < 0.25:     # a first tile without keys
            a, b = [False] * (sinks + width), [True] * (sinks + width)
        elif kind < 0.35:     # both alike
            a = b = [True] * (sinks + width)
        elif kind < 0.4:
            items.append((0, ([], [])))
            continue
        items.append((len(a), (a, b)))
    return items


@pytest.mark.parametrize("stages", [5, 10])
@pytest.mark.parametrize("seed", range(12))
def test_protocol_holds_under_random_timing(stages, seed):
    rng = random.Random(1000 + seed)
    Sim(seed, make_items(rng, 40), stages).go()


@pytest.mark.parametrize("mistake", ["last_pv_on_s", "free_early", "one_free", "p_once"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(12):
        rng = random.Random(seed)
        try:
            Sim(seed, make_items(rng, 40), 5, mistake).go()
        except (Stuck, Wrong):
            caught += 1
    assert caught >= 9, caught
