"""Event model of the tensor-core window backward's barrier protocol
(csrc/window_bwd_sm100.cu), on the CPU: the loader, the MMA issuer and the eight
element-wise warps as generators that wait on mbarriers by parity and work for
random times, with a check at every access that a buffer holds what it should.
The layouts of the kernels (two buffers of S, with one or two gradient products
per pair; one buffer, with S and dP half by half behind them) must hold under
random timing;
planted mistakes must be caught, among them the terms of both pairs in flight
signalled on one barrier, as the kernel first had it: a warp that ran ahead
then stood in for one that had not written yet."""
import random

import pytest

from test_window_fwd_protocol_model import Bar, Sim, Stuck, Wrong


LAYOUTS = {  # two buffers of S, gradients per pair, stages of the two rings
    "dq": (True, 1, 3, 2),
    "dkdv64": (True, 2, 3, 3),
    "dkdv128": (False, 2, 2, 2),
}


class Bwd(Sim):
    def __init__(self, seed, n, layout, mistake=None):
        super().__init__(seed, [], 1, None)
        self.n, self.mistake = n, mistake
        self.two, self.ng, self.NA, self.NB = LAYOUTS[layout]
        self.bar = {"fixed": Bar(1)}
        for r, k in (("a", self.NA), ("b", self.NB)):
            for i in range(k):
                self.bar["full", r, i], self.bar["free", r, i] = Bar(1), Bar(1)
        for h in (0, 1):
            self.bar["s", h] = Bar(1)
            for p in (0, 1):
                self.bar["p", p, h] = Bar(8 if self.two else 4)  # two buffers: h = 0 for all
        self.bar["r"] = Bar(8)
        self.hold = {"a": [None] * self.NA, "b": [None] * self.NB}
        self.busy = {"a": [0] * self.NA, "b": [0] * self.NB}
        self.sbuf = {(i, h): None for i in (0, 1) for h in (0, 1)}  # ("S" or "T", pair)
        self.written = {}
        self.dp = [None, None]      # per half: pair, or None once overwritten is allowed
        self.reads = {}             # (pair, half) -> warps that read dP
        self.done_pairs = 0
        self.t = 0.0

    def sb(self, it):
        return it % 2 if self.two else 0

    def loader(self):
        yield self.rnd(100)
        self.at(self.now + 500, lambda: self.arrive("fixed"))
        for it in range(self.n):
            for r, k in (("a", self.NA), ("b", self.NB)):
                i = it % k
                yield "wait", ("free", r, i), ((it // k) & 1) ^ 1
                if self.busy[r][i]:
                    raise Wrong(f"{r} stage {i} refilled while an MMA reads it")
                self.hold[r][i] = None

                def land(r=r, i=i, it=it):
                    self.hold[r][i] = it
                    self.arrive(("full", r, i))
                self.at(self.now + self.rng.expovariate(1 / 1000), land)

    def op(self, time, uses, begin=None, end=None):
        start = max(self.now, self.t)
        self.t = start + self.rng.expovariate(1 / time)

        def b():
            for r, it in uses:
                i = it % (self.NA if r == "a" else self.NB)
                if self.hold[r][i] != it:
                    raise Wrong(f"{r} stage holds {self.hold[r][i]}, not {it}")
                self.busy[r][i] += 1
            if begin:
                begin()

        def e():
            for r, it in uses:
                self.busy[r][it % (self.NA if r == "a" else self.NB)] -= 1
            if end:
                end()
        self.at(start, b)
        self.at(self.t, e)

    def sign(self, name):
        self.at(max(self.now, self.t) + 1, lambda: self.arrive(name))

    def scores(self, it, halves):
        def begin():
            for h in halves:
                old = self.sbuf[self.sb(it), h]
                if old is not None and old[0] == "S":
                    raise Wrong("S overwritten before its terms were used")
                self.sbuf[self.sb(it), h] = None

        def end():
            for h in halves:
                self.sbuf[self.sb(it), h] = ("S", it)
        self.op(300, [("a", it)], begin, end)

    def dprobs(self, it, halves=(0, 1)):
        def begin():
            for h in halves:
                if it > 0 and self.reads.get((it - 1, h), 0) != 4:
                    raise Wrong("dP overwritten before it was read")
                self.dp[h] = None

        def end():
            for h in halves:
                self.dp[h] = it
        self.op(300, [("b", it)], begin, end)

    def grads(self, it, h):
        def begin():
            if self.sbuf[self.sb(it), h] != ("S", it) or self.written.get((it, h), 0) != 4:
                raise Wrong(f"gradient product of pair {it} finds {self.written.get((it, h), 0)} of 4 warps' terms")

        def end():
            self.sbuf[self.sb(it), h] = ("T", it)
            self.done_pairs += h
        self.op(300, [("a", it)] + ([("b", it)] if self.ng == 2 else []), begin, end)

    def mma(self):
        yield "wait", "fixed", 0
        yield "wait", ("full", "a", 0), 0
        yield "wait", ("full", "b", 0), 0
        self.scores(0, (0, 1))
        self.dprobs(0)
        self.sign(("s", 0))
        if not self.two:
            self.sign(("s", 1))
        if self.ng == 1:
            self.sign(("free", "b", 0))
        if self.two and self.n > 1:
            yield "wait", ("full", "a", 1 % self.NA), (1 // self.NA) & 1
            self.scores(1, (0, 1))
        for it in range(self.n):
            more, p, ph = it + 1 < self.n, it & 1, (it >> 1) & 1
            if self.mistake == "one_p":
                p, ph = 0, it & 1
            if self.two:
                if more:
                    yield "wait", ("full", "b", (it + 1) % self.NB), ((it + 1) // self.NB) & 1
                    if self.mistake != "no_read_wait":
                        yield "wait", "r", it & 1
                    self.dprobs(it + 1)
                    self.sign(("s", 0))
                    if self.ng == 1:
                        self.sign(("free", "b", (it + 1) % self.NB))
                    yield self.rnd(100)
                if it + 2 < self.n:
                    yield "wait", ("full", "a", (it + 2) % self.NA), ((it + 2) // self.NA) & 1
                yield "wait", ("p", p, 0), ph
                self.grads(it, 0)
                self.grads(it, 1)
                self.sign(("free", "a", it % self.NA))
                if self.ng == 2:
                    self.sign(("free", "b", it % self.NB))
                if it + 2 < self.n:
                    self.scores(it + 2, (0, 1))
                yield self.rnd(100)
                continue
            for h in (0, 1):
                yield "wait", ("p", p, h), ph
                self.grads(it, h)
                if h == 1:
                    self.sign(("free", "a", it % self.NA))
                    self.sign(("free", "b", it % self.NB))
                yield self.rnd(150)
                if more:
                    if h == 0:
                        yield "wait", ("full", "a", (it + 1) % self.NA), ((it + 1) // self.NA) & 1
                        yield "wait", ("full", "b", (it + 1) % self.NB), ((it + 1) // self.NB) & 1
                    self.scores(it + 1, (h,))
                    self.dprobs(it + 1, (h,))
                    self.sign(("s", h))

    def warp(self, w):
        h = w // 4
        for it in range(self.n):
            yield "wait", ("s", 0 if self.two else h), it & 1
            if self.sbuf[self.sb(it), h] != ("S", it) or self.dp[h] != it:
                raise Wrong(f"warp {w} at pair {it} finds S {self.sbuf[self.sb(it), h]}, dP {self.dp[h]}")
            yield self.rnd(200 * (8 if self.rng.random() < 0.05 else 1))
            if self.dp[h] != it:
                raise Wrong("dP changed while it was read")
            self.reads[it, h] = self.reads.get((it, h), 0) + 1
            if self.two:
                self.arrive("r")
            yield self.rnd(1200 * (4 if self.rng.random() < 0.05 else 1))  # now and then a slow warp
            if self.sbuf[self.sb(it), h] != ("S", it):
                raise Wrong("S gone before its terms were written")
            self.written[it, h] = self.written.get((it, h), 0) + 1
            self.arrive(("p", 0 if self.mistake == "one_p" else it & 1, 0 if self.two else h))
        yield "wait", ("free", "a", (self.n - 1) % self.NA), ((self.n - 1) // self.NA) & 1
        if self.done_pairs != self.n:
            raise Wrong(f"output after {self.done_pairs} of {self.n} pairs")

    def go(self):
        self.spawn(self.loader())
        self.spawn(self.mma())
        for w in range(8):
            self.spawn(self.warp(w))
        self.run()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("seed", range(8))
def test_protocol_holds_under_random_timing(layout, seed):
    for n in (1, 2, 3, 4, 60):
        Bwd(100 * seed + n, n, layout).go()


@pytest.mark.parametrize("mistake", ["one_p", "no_read_wait"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(10):
        try:
            Bwd(seed, 80, "dq", mistake).go()
        except (Stuck, Wrong):
            caught += 1
    assert caught >= 9, caught

