"""All mbarriers of the tree attention's tensor-core kernel in one CPU model, the
error path's aside: those of test_attn_tree_protocol.py and, besides,
  q_full    the run's queries are written (the MMA warp waits for it once a run;
            a convert warp writes its queries before its first tile, so op_ready
            alone would give the same order);
  op_full   bf16 caches: a tile's copies have landed (the convert warps and the
            MMA warp wait for it; there are no raw tiles);
  pv_done   a product with the weights b is complete.  It is the one barrier that
            is waited on now and then: by a softmax warp before it rescales the
            output, when a row's reference has moved, so whole phases pass
            without a poll.
Checked at every poll: the barrier has completed the phases before the one meant,
or one more.  Checked besides: no operand, score, weight or query is overwritten
before its last use, no product adds to an output that is being rescaled, and it
is rescaled after exactly the products before.  Roles run in random order, copies
land and MMA groups complete (in the order of issue) after random delays.
Protocols with one wait wrong or missing are shown to fail."""
import random

import pytest

from tests.test_attn_tree_protocol import RUNS, Bar, item

WARPS = 2                                        # convert warps, softmax warps of a row half


class Model:
    def __init__(self, runs, rng, rings, fault=None, moves=0.4):
        """runs: [(tiles, row halves)]; rings: operand and raw tiles (no raw ones: a bf16 cache)."""
        self.runs, self.rng, self.fault, self.moves = runs, rng, fault, moves
        self.n_ops, self.n_raw = rings
        self.k8 = self.n_raw > 0

        def bars(n, need):
            return [Bar(None, need) for _ in range(n)]
        self.op_full, self.op_ready, self.op_empty = bars(self.n_ops, 1), bars(self.n_ops, WARPS), bars(self.n_ops, 1)
        self.raw_full, self.raw_empty = bars(self.n_raw, 1), bars(self.n_raw, WARPS)
        self.q_full = Bar("q_full", WARPS)
        self.s_full, self.p_full, self.pv_done, self.o_full = bars(2, 1), bars(2, WARPS), bars(2, 1), bars(2, 1)
        for name in ("op_full", "op_ready", "op_empty", "raw_full", "raw_empty", "s_full", "p_full", "pv_done", "o_full"):
            for i, b in enumerate(getattr(self, name)):
                b.name = f"{name}[{i}]"
        self.bad, self.copies, self.mma = [], [], []
        self.raw_holds, self.op_holds, self.op_done = {}, {}, {}
        self.q_parts, self.s_holds, self.p_parts, self.products, self.moved = {}, {}, {}, {}, {}
        self.at, self.gen = {}, {}
        self.polls = {}

    # ---- waits
    def wait(self, bar, phase):
        while True:
            if phase < 0:
                return
            if bar.done not in (phase, phase + 1):
                self.bad.append((bar.name, phase, bar.done))
            self.polls[bar.name] = self.polls.get(bar.name, 0) + 1
            if (bar.done & 1) != (phase & 1):
                return
            yield

    def meet(self, key, n):
        self.at[key] = self.at.get(key, 0) + 1
        if self.at[key] == n:
            self.at[key], self.gen[key] = 0, self.gen.get(key, 0) + 1
            return
        gen = self.gen.get(key, 0)
        while self.gen.get(key, 0) == gen:
            yield

    def run_end(self):
        yield from self.meet("run", 2 + 3 * WARPS)

    def expect(self, ok, *what):
        if not ok:
            self.bad.append(what)

    def held_after(self, held, nt, nm):
        return [held[b] + (nt if nm == 2 else (nt + 1 - b) // 2) for b in range(2)]

    # ---- roles
    def copy(self):
        n = 0
        for r, (nt, _) in enumerate(self.runs):
            for i in range(2 * nt):
                size = self.n_raw if self.k8 else self.n_ops
                slot, use = n % size, n // size
                if self.fault != "copy does not wait":
                    yield from self.wait((self.raw_empty if self.k8 else self.op_empty)[slot], use - 1)
                self.copies.append((slot, (r, i)))
                n += 1
                yield
            yield from self.run_end()

    def convert(self):
        n = 0
        for r, (nt, _) in enumerate(self.runs):
            self.expect(not any(m[0] == "S" for m in self.mma), "queries written under the scores", r)
            yield
            self.q_parts[r] = self.q_parts.get(r, 0) + 1
            self.q_full.arrive()
            for i in range(2 * nt):
                os_, ou = n % self.n_ops, n // self.n_ops
                if self.k8:
                    rs, ru = n % self.n_raw, n // self.n_raw
                    yield from self.wait(self.raw_full[rs], ru)
                    yield from self.wait(self.op_empty[os_], ou - 1)
                    self.expect(self.raw_holds.get(rs) == (r, i), "raw tile", rs, (r, i))
                else:
                    yield from self.wait(self.op_full[os_], ou)
                    self.expect(self.op_holds.get(os_) == (r, i), "tile", os_, (r, i))
                n += 1
                yield
                self.op_done[(r, i)] = self.op_done.get((r, i), 0) + 1
                if self.k8:
                    if self.op_done[(r, i)] == WARPS:
                        self.op_holds[os_] = (r, i)
                    self.raw_empty[rs].arrive()
                self.op_ready[os_].arrive()
                yield
            yield from self.run_end()

    def mma_role(self):
        n, held = 0, [0, 0]
        for r, (nt, nm) in enumerate(self.runs):
            index = {item(j, nt): j for j in range(2 * nt)}

            def ready(j):
                slot, use = (n + j) % self.n_ops, (n + j) // self.n_ops
                if not self.k8:
                    yield from self.wait(self.op_full[slot], use)
                yield from self.wait(self.op_ready[slot], use)
                return slot

            def scores(t, m):
                slot = yield from ready(index[(t, False)])
                b = m if nm == 2 else t & 1
                self.expect(self.q_parts.get(r) == WARPS, "queries", r)
                self.mma.append(("S", slot, (r, index[(t, False)]), b, (r, t, m),
                                 [self.s_full[b]] + ([self.op_empty[slot]] if m == nm - 1 else [])))

            def product(t, m):
                b, k = (m, t) if nm == 2 else (t & 1, t >> 1)
                yield from self.wait(self.p_full[b], held[b] + k)
                slot = yield from ready(index[(t, True)])
                self.mma.append(("P", slot, (r, index[(t, True)]), b, (r, t, m),
                                 [self.pv_done[b]] + ([self.o_full[m]] if t == nt - 1 else []) +
                                 ([self.op_empty[slot]] if m == nm - 1 else [])))
            yield from self.wait(self.q_full, r)
            for t in range(-1, nt):
                steps = [(f, u, m) for m in range(nm) for f, u in ((product, t), (scores, t + 1))]
                if nm == 1:
                    steps.reverse()
                for f, u, m in steps:
                    if 0 <= u < nt:
                        yield from f(u, m)
                        yield
            n += 2 * nt
            held = self.held_after(held, nt, nm)
            yield from self.run_end()

    def softmax(self, m, w):
        held, outputs = [0, 0], 0
        for r, (nt, nm) in enumerate(self.runs):
            if m < nm:
                half = ("half", m)
                for t in range(nt):
                    b, k = (m, t) if nm == 2 else (t & 1, t >> 1)
                    yield from self.wait(self.s_full[b], held[b] + k)
                    self.expect(self.s_holds.get(b) == (r, t, m), "scores", b, (r, t, m), self.s_holds.get(b))
                    yield
                    moves = self.moved.setdefault((r, t, m), self.rng.random() < self.moves)
                    yield from self.meet(half, WARPS)
                    if moves:
                        yield from self.meet(half, WARPS)
                        yield from self.meet(half, WARPS)
                        if t > 0:
                            if nm == 1 and self.fault != "no pv_done":
                                late = 1 if self.fault == "pv_done of the next tile" else 0
                                yield from self.wait(self.pv_done[b ^ 1], held[b ^ 1] + ((t - 1) >> 1) + late)
                            for _ in range(2):         # the output is read, then written
                                done = self.products.get((r, m), 0)
                                flying = [x[4] for x in self.mma if x[0] == "P" and x[4][0] == r and x[4][2] == m]
                                self.expect(done == t and not flying, "output rescaled", (r, t, m), done, flying)
                                yield
                        self.expect(self.s_holds.get(b) == (r, t, m), "scores gone", b, (r, t, m))
                        yield from self.meet(half, WARPS)
                    self.expect(nm == 2 or t < 2 or self.products.get((r, m), 0) >= t - 1, "weights in use", (r, t, m))
                    self.p_parts[(r, t, m)] = self.p_parts.get((r, t, m), 0) + 1
                    self.p_full[b].arrive()
                    yield
                yield from self.wait(self.o_full[m], outputs)
                outputs += 1
                self.expect(self.products.get((r, m)) == nt, "output", (r, m), self.products.get((r, m)))
                yield from self.meet(half, WARPS)
            held = self.held_after(held, nt, nm)
            yield from self.run_end()

    def step_async(self):
        """Something in flight completes: any copy, or the oldest MMA group."""
        if self.rng.randrange(2) == 0 and self.copies:
            slot, what = self.copies.pop(self.rng.randrange(len(self.copies)))
            held = (self.raw_holds if self.k8 else self.op_holds)
            held[slot] = what
            (self.raw_full if self.k8 else self.op_full)[slot].arrive()
        elif self.mma:
            kind, slot, tile, b, who, commits = self.mma.pop(0)
            self.expect(self.op_holds.get(slot) == tile, "operand", slot, tile, self.op_holds.get(slot))
            if kind == "S":
                self.s_holds[b] = who
            else:
                self.expect(self.p_parts.get(who) == WARPS, "weights", who)
                self.products[(who[0], who[2])] = self.products.get((who[0], who[2]), 0) + 1
            for c in commits:
                c.arrive()

    def go(self, steps=200000):
        live = [self.copy(), self.mma_role()] + [self.convert() for _ in range(WARPS)] + \
            [self.softmax(m, w) for m in range(2) for w in range(WARPS)]
        for _ in range(steps):
            if self.bad or not live:
                break
            if self.rng.random() < 0.3:
                self.step_async()
                continue
            c = self.rng.choice(live)
            try:
                for _ in range(self.rng.choice((1, 1, 1, 12))):
                    next(c)
            except StopIteration:
                live.remove(c)
        return not live


# 8 bits and bf16, with up to 128 rows a run and with up to 256
RINGS = [(3, 5), (3, 3), (5, 0), (4, 0)]


@pytest.mark.parametrize("rings", RINGS)
@pytest.mark.parametrize("runs", RUNS + [[(9, 1)], [(8, 1), (5, 1), (9, 1)]])
def test_every_poll_of_every_barrier(runs, rings):
    polled = set()
    for seed in range(40):
        m = Model(runs, random.Random(seed), rings, moves=(0.0, 0.1, 0.5, 1.0)[seed % 4])
        assert m.go(), ("does not end", seed, m.bad)
        assert not m.bad, (seed, m.bad[:3])
        polled |= {name.split("[")[0] for name in m.polls}
    want = {"q_full", "op_ready", "op_empty", "s_full", "p_full", "o_full"}
    want |= {"raw_full", "raw_empty"} if rings[1] else {"op_full"}
    if any(nt > 1 and nm == 1 for nt, nm in runs):
        want.add("pv_done")
    want -= {name for name, n in zip(("op_empty", "raw_empty"), rings)
             if sum(2 * nt for nt, _ in runs) <= n}            # a ring that is not used twice
    assert polled >= want, want - polled


@pytest.mark.parametrize("rings", RINGS)
@pytest.mark.parametrize("fault", ["no pv_done", "pv_done of the next tile", "copy does not wait"])
def test_a_wait_wrong_or_missing_fails(fault, rings):
    assert any(not (m := Model([(7, 1), (4, 1)], random.Random(s), rings, fault)).go(20000) or m.bad
               for s in range(200))
