"""CPU model of the attention backward kernel's barrier protocol (no GPU).

attention_backward_kernel holds two kinds of CTA (dK/dV of 128 keys, dQ of one
or two tiles of 128 queries) whose roles -- two producer warps, the MMA
issuing warp, two elementwise warpgroups, and behind them the tensor core,
which runs MMAs in issue order, and the loads in flight -- meet only at
mbarriers.  This module restates every role's sequence of waits, arrivals,
loads and MMAs, with the barriers' parity rule (a wait for parity p passes
while the current phase has the other parity, so a phase too far ahead blocks
it), interleaves them at random and checks that
  * every run ends: no order of events blocks a wait for good;
  * every MMA and every elementwise step finds the operand it is meant to read
    (no ring stage, score or probability tile is overwritten too early);
  * each accumulator gets every tile once, in order.
A protocol with a planted mistake must fail.  The GPU tests check the kernel
itself against the formula."""
import random

import pytest


class Bar:
    def __init__(self, count=1):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        return (self.phase & 1) != parity


class Cta:
    """One CTA: shared state, the tensor core's queue and the loads in flight."""

    def __init__(self, T, is_dq, nt, tiles, mistake=None):
        self.T, self.is_dq, self.nt, self.mistake = T, is_dq, nt, mistake
        self.tiles = tiles     # of scores in tensor memory: 1, or 2 with D = 64
        one = lambda n: [Bar() for _ in range(n)]
        self.own, self.x_full, self.x_empty = one(4), one(3), one(3)
        self.y_full, self.y_empty, self.stat, self.stat_empty = one(2), one(2), one(2), one(2)
        self.s, self.s_free, self.dp, self.acc = one(2), Bar(2), Bar(), Bar()
        self.p, self.ds = [one(2), one(2)], one(2)
        self.mem = {}          # shared and tensor memory: name -> content
        self.queue = []        # the tensor core, in issue order
        self.loads = []        # (slot, content, barrier)
        self.sums = {"A0": [], "A1": []}

    # ------------------------------------------------ what the roles do
    def load(self, slot, content, bar):
        self.loads.append((slot, content, bar))

    def mma(self, reads, write=None, add=None):
        self.queue.append(("mma", reads, write, add))

    def commit(self, bar):
        self.queue.append(("commit", bar))

    def expect(self, slot, content):
        assert self.mem.get(slot) == content, (slot, self.mem.get(slot), content)

    def run_tensor_core(self):
        op = self.queue.pop(0)
        if op[0] == "commit":
            op[1].arrive()
            return
        _, reads, write, add = op
        for slot, content in reads:
            self.expect(slot, content)
        if write:
            self.mem[write[0]] = write[1]
        if add:
            self.sums[add[0]].append(add[1])

    def land(self, i):
        slot, content, bar = self.loads.pop(i)
        self.mem[slot] = content
        bar.arrive()

    # ------------------------------------------------ the roles
    def producer(self, first):
        stages = (1 if self.is_dq else 2) + (1 if first else 0)
        full, empty = (self.x_full, self.x_empty) if first else (self.y_full, self.y_empty)
        ring, own = ("X", 0) if first else ("Y", 1)
        self.load(("own", own), ("own", own), self.own[own])
        rs, rp = 0, 1
        for j in range(self.T):
            yield empty[rs], rp
            self.load((ring, rs), (ring, j), full[rs])
            rs += 1
            if rs == stages:
                rs, rp = 0, rp ^ 1
            if not self.is_dq and first:
                if self.mistake == "statistics wait on dS":   # a phase that can run ahead
                    if j >= 2:
                        yield self.ds[0], j & 1
                        yield self.ds[1], j & 1
                else:
                    yield self.stat_empty[j & 1], ((j >> 1) & 1) ^ 1
                self.load(("stat", j & 1), ("stat", j), self.stat[j & 1])
            if j == 0 and self.nt == 2:
                self.load(("own", 2 + own), ("own", 2 + own), self.own[2 + own])

    def tile(self, i):
        """Item i's score tile: name, barrier index, parity."""
        b = i % self.tiles
        return f"R0.{b}", b, (i // self.tiles) & 1

    def next_scores(self, i, own, xn, j):
        name, b, _ = self.tile(i)
        self.scores(own, "X", xn, j, ("S", i), name)
        self.commit(self.s[b])

    def scores(self, own, ring, stage, j, tile, out):
        self.mma([(("own", own), ("own", own)), ((ring, stage), (ring, j))], write=(out, tile))

    def issue_dkdv(self):
        yield self.own[0], 0
        yield self.x_full[0], 0
        self.next_scores(0, 0, 0, 0)
        yield self.own[1], 0
        yield self.y_full[0], 0
        self.scores(1, "Y", 0, 0, ("dP", 0), "R1")
        self.commit(self.dp)
        xs = xp = 0
        for j in range(self.T):
            par, ys, nxt = j & 1, j & 1, j + 1 < self.T
            xn, xnp = (0, xp ^ 1) if xs == 2 else (xs + 1, xp)
            if nxt:
                yield self.x_full[xn], xnp
            if nxt and (self.tiles == 2 or self.mistake == "S before dV"):
                self.next_scores(j + 1, 0, xn, j + 1)
            for h in range(2):
                name, b, sp = self.tile(j)
                if self.mistake == "one barrier for two tiles":
                    b, sp = 0, par
                yield self.p[b][h], sp
                self.mma([(("P", h, j % self.tiles), ("P", j)), (name, ("S", j)),
                          (("Y", ys), ("Y", j))], add=("A0", (j, h)))
            self.commit(self.y_empty[ys])
            if nxt and self.tiles == 1 and self.mistake != "S before dV":
                self.next_scores(j + 1, 0, xn, j + 1)
            for h in range(2):
                yield self.ds[h], par
                self.mma([(("dS", h), ("dS", j)), ("R1", ("dP", j)), (("X", xs), ("X", j))],
                         add=("A1", (j, h)))
            self.commit(self.x_empty[xs])
            self.stat_empty[ys].arrive()
            if nxt:
                yield self.y_full[ys ^ 1], ((j + 1) >> 1) & 1
                self.scores(1, "Y", ys ^ 1, j + 1, ("dP", j + 1), "R1")
                self.commit(self.dp)
            xs, xp = xn, xnp
        self.commit(self.acc)

    def issue_dq(self):
        nt = self.nt
        yield self.own[0], 0
        yield self.x_full[0], 0
        self.next_scores(0, 0, 0, 0)
        yield self.own[1], 0
        yield self.y_full[0], 0
        self.scores(1, "Y", 0, 0, ("dP", 0), "R1")
        self.commit(self.dp)
        if nt == 1:
            self.commit(self.y_empty[0])
        else:
            yield self.own[2], 0
            yield self.own[3], 0
        j = t = par = i = 0
        while j < self.T:
            jn, tn = (j + 1, 0) if t + 1 == nt else (j, t + 1)
            nxt, xs, xn = jn < self.T, j & 1, jn & 1
            if nxt:
                if tn == 0:
                    yield self.x_full[xn], (jn >> 1) & 1
                if self.tiles == 1 and self.mistake != "S without its reader":
                    yield self.s_free, par
                self.next_scores(i + 1, 2 * tn, xn, jn)
            for h in range(2):
                yield self.ds[h], par
                self.mma([(("dS", h), ("dS", i)), ("R1", ("dP", i)), (("X", xs), ("X", j))],
                         add=(f"A{t}", (j, h)))
            if t == nt - 1:
                self.commit(self.x_empty[xs])
            if nxt:
                if tn == 0:
                    yield self.y_full[0], jn & 1
                self.scores(2 * tn + 1, "Y", 0, jn, ("dP", i + 1), "R1")
                self.commit(self.dp)
                if tn == nt - 1:
                    self.commit(self.y_empty[0])
            j, t, par, i = jn, tn, par ^ 1, i + 1
        self.commit(self.acc)

    def elementwise(self, h):
        for i in range(self.T * (self.nt if self.is_dq else 1)):
            par = i & 1
            if not self.is_dq:
                yield self.stat[par], (i >> 1) & 1
            name, b, sp = self.tile(i)
            yield self.s[b], sp
            self.expect(name, ("S", i))
            yield None                       # (the scores on their way to registers)
            self.expect(name, ("S", i))
            if self.is_dq and self.tiles == 1:
                self.s_free.arrive()
            if not self.is_dq:
                self.expect(("stat", par), ("stat", i))
                self.mem[("P", h, b)] = ("P", i)
                self.p[0 if self.mistake == "one barrier for two tiles" else b][h].arrive()
            yield self.dp, par
            self.expect("R1", ("dP", i))
            if not self.is_dq:
                self.expect(("stat", par), ("stat", i))
            yield None
            self.expect("R1", ("dP", i))
            self.mem[("dS", h)] = ("dS", i)
            self.ds[h].arrive()
        yield self.acc, 0


def simulate(T, is_dq, nt, tiles, rng, mistake=None):
    c = Cta(T, is_dq, nt, tiles, mistake)
    roles = [c.producer(True), c.producer(False), c.issue_dq() if is_dq else c.issue_dkdv(),
             c.elementwise(0), c.elementwise(1)]
    waiting = [next(r, "end") for r in roles]
    # some runs favour one actor, so that it runs as far ahead as it can
    weight = [rng.choice([1, 1, 1, 20]) for _ in range(7)]
    while True:
        ready = [i for i, w in enumerate(waiting)
                 if w != "end" and (w is None or w[0].passes(w[1]))]
        if c.queue:
            ready.append(5)
        if c.loads:
            ready.append(6)
        if not ready:
            break
        i = rng.choices(ready, [weight[k] for k in ready])[0]
        if i == 5:
            c.run_tensor_core()
        elif i == 6:
            c.land(rng.randrange(len(c.loads)))
        else:
            waiting[i] = next(roles[i], "end")
    assert all(w == "end" for w in waiting), "blocked"
    every = [(j, h) for j in range(T) for h in range(2)]
    assert c.sums["A0"] == every
    assert c.sums["A1"] == (every if not is_dq or nt == 2 else [])


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("is_dq,nt", [(False, 1), (True, 1), (True, 2)])
def test_every_interleaving_ends_with_the_right_operands(is_dq, nt, tiles):
    for T in (1, 2, 3, 4, 5, 8, 13):
        for seed in range(60):
            simulate(T, is_dq, nt, tiles, random.Random(1000 * T + seed))


@pytest.mark.parametrize("is_dq,nt,tiles,mistake", [
    (False, 1, 1, "statistics wait on dS"), (False, 1, 2, "statistics wait on dS"),
    (False, 1, 1, "S before dV"), (True, 2, 1, "S without its reader"),
    (False, 1, 2, "one barrier for two tiles")])
def test_planted_mistakes_are_found(is_dq, nt, tiles, mistake):
    failed = 0
    for seed in range(300):
        try:
            simulate(9, is_dq, nt, tiles, random.Random(seed), mistake)
        except AssertionError:
            failed += 1
    assert failed > 0, mistake
