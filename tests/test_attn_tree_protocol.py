"""The barrier protocol of the tree attention's tensor-core kernel, modelled on
the CPU.

The kernel (csrc/attn_tree_tc.cu) hands operand tiles and scores from copy to
convert to MMA to softmax warps through mbarriers, waited on by phase parity.
That is sound only if, at every poll for a phase, the barrier has completed
either exactly the phases before it or one more: one fewer reads as done (a
false pass, and the next arrivals come out of turn), two more as not done (a
wait that never ends).  This model runs the roles' program order as coroutines
under random interleavings, with copies landing and MMA groups completing after
random delays (MMAs in the order of issue), and checks every poll, that no tile,
scores or weights are overwritten before their last use, and that every run
ends.  Two protocols that the kernel must not use are shown to fail: one barrier
for the weights of both tiles in turn (a softmax warp a tile ahead arrives for
one that has not), and a ring of an odd number of slots shared by two groups of
convert warps that take tiles in turn."""
import random

import pytest


class Bar:
    def __init__(self, name, need):
        self.name, self.need, self.got, self.done = name, need, 0, 0

    def arrive(self):
        self.got += 1
        if self.got == self.need:
            self.got, self.done = 0, self.done + 1


def item(i, nt):
    """Operand tile i in the order of use: (tile, values?)."""
    if i == 0:
        return 0, False
    if i == 2 * nt - 1:
        return nt - 1, True
    return ((i + 1) // 2, False) if i & 1 else (i // 2 - 1, True)


class Model:
    WARPS = 2                                     # of a softmax group, and of a convert group

    def __init__(self, runs, rng, ops=3, raw=5, groups=1, one_p=False):
        """runs: [(tiles, row halves)]."""
        self.runs, self.rng, self.ops, self.raw, self.groups = runs, rng, ops, raw, groups
        self.op_ready = [Bar(f"op_ready{i}", self.WARPS) for i in range(ops)]
        self.op_empty = [Bar(f"op_empty{i}", 1) for i in range(ops)]
        self.raw_full = [Bar(f"raw_full{i}", 1) for i in range(raw)]
        self.raw_empty = [Bar(f"raw_empty{i}", self.WARPS) for i in range(raw)]
        self.s_full = [Bar("s0", 1), Bar("s1", 1)]
        self.p_full = [Bar("p0", self.WARPS), Bar("p1", self.WARPS)]
        if one_p:
            self.p_full[1] = self.p_full[0]
        self.one_p = one_p
        self.o_full = [Bar("o0", 1), Bar("o1", 1)]
        self.bad, self.copies, self.mma = [], [], []
        self.raw_holds, self.op_holds, self.op_parts = {}, {}, {}
        self.s_holds, self.p_holds = {}, {}
        self.meet = 0                             # roles at the run's end
        self.n_roles = 2 + groups * self.WARPS + 2 * self.WARPS
        self.run_no = 0

    def poll(self, bar, phase):
        if bar.done not in (phase, phase + 1) and phase >= 0:
            self.bad.append((bar.name, phase, bar.done))
        return phase < 0 or (bar.done & 1) != (phase & 1)

    def wait(self, bar, phase):
        while not self.poll(bar, phase):
            yield

    def expect(self, ok, what):
        if not ok:
            self.bad.append(what)

    def ring(self, n, size):
        return n % size, n // size

    # ---- roles (each yields where another may run)
    def end_run(self):
        self.meet += 1
        if self.meet == self.n_roles:
            self.meet, self.run_no = 0, self.run_no + 1
            return
        at = self.run_no
        while self.run_no == at:
            yield

    def copy(self):
        n = 0
        for r, (nt, _) in enumerate(self.runs):
            for i in range(2 * nt):
                slot, use = self.ring(n, self.raw)
                yield from self.wait(self.raw_empty[slot], use - 1)
                self.copies.append((slot, (r, i)))
                n += 1
                yield
            yield from self.end_run()

    def convert(self, group):
        n = 0
        for r, (nt, _) in enumerate(self.runs):
            for i in range(2 * nt):
                mine = self.groups == 1 or (i & 1) == group
                rs, ru = self.ring(n, self.raw)
                os_, ou = self.ring(n, self.ops)
                n += 1
                if not mine:
                    continue
                yield from self.wait(self.raw_full[rs], ru)
                yield from self.wait(self.op_empty[os_], ou - 1)
                self.expect(self.raw_holds.get(rs) == (r, i), ("raw tile", rs, (r, i)))
                yield
                parts = self.op_parts.setdefault((r, i), 0) + 1
                self.op_parts[(r, i)] = parts
                if parts == self.WARPS:
                    self.op_holds[os_] = (r, i)
                self.raw_empty[rs].arrive()
                self.op_ready[os_].arrive()
                yield
            yield from self.end_run()

    def issue(self, kind, slot, tile, b, m, commits):
        self.mma.append((kind, slot, tile, b, m, commits))

    def mma_role(self):
        n, held = 0, [0, 0]
        for r, (nt, nm) in enumerate(self.runs):
            def ready(i):
                slot, use = self.ring(n0 + i, self.ops)
                yield from self.wait(self.op_ready[slot], use)
            n0, i = n, 0
            index = {item(j, nt): j for j in range(2 * nt)}
            for t in range(-1, nt):
                for m in range(nm):
                    def scores():
                        j = index[(t + 1, False)]
                        yield from ready(j)
                        b = m if nm == 2 else (t + 1) & 1
                        slot = self.ring(n0 + j, self.ops)[0]
                        self.issue("S", slot, (r, j), b, (r, t + 1, m),
                                   [self.s_full[b]] + ([self.op_empty[slot]] if m == nm - 1 else []))

                    def product():
                        b = m if nm == 2 else t & 1
                        k = t if nm == 2 else t >> 1
                        if self.one_p and nm == 1:
                            yield from self.wait(self.p_full[0], held[0] + held[1] + t)
                        else:
                            yield from self.wait(self.p_full[b], held[b] + k)
                        j = index[(t, True)]
                        yield from ready(j)
                        slot = self.ring(n0 + j, self.ops)[0]
                        self.issue("P", slot, (r, j), b, (r, t, m),
                                   ([self.o_full[m]] if t == nt - 1 else []) +
                                   ([self.op_empty[slot]] if m == nm - 1 else []))
                    if nm == 2:                   # in order after the product that reads the weights
                        if t >= 0:
                            yield from product()
                        if t + 1 < nt:
                            yield from scores()
                    else:
                        if t + 1 < nt:
                            yield from scores()
                        if t >= 0:
                            yield from product()
                    yield
            n += 2 * nt
            for b in range(2):
                held[b] += nt if nm == 2 else (nt + 1 - b) // 2
            yield from self.end_run()

    def softmax(self, m, w):
        held, o = [0, 0], 0
        for r, (nt, nm) in enumerate(self.runs):
            if m < nm:
                for t in range(nt):
                    b, k = (m, t) if nm == 2 else (t & 1, t >> 1)
                    yield from self.wait(self.s_full[b], held[b] + k)
                    self.expect(self.s_holds.get(b) == (r, t, m), ("scores", b, (r, t, m), self.s_holds.get(b)))
                    yield
                    self.expect(self.s_holds.get(b) == (r, t, m), ("scores overwritten", b, (r, t, m)))
                    self.p_holds.setdefault((r, t, m), set()).add(w)
                    self.p_full[b].arrive()
                    yield
                yield from self.wait(self.o_full[m], o)
                o += 1
            for b in range(2):
                held[b] += nt if nm == 2 else (nt + 1 - b) // 2
            yield from self.end_run()

    def step_async(self):
        """Something in flight completes: any copy, or the oldest MMA group."""
        pick = self.rng.randrange(2)
        if pick == 0 and self.copies:
            slot, what = self.copies.pop(self.rng.randrange(len(self.copies)))
            self.raw_holds[slot] = what
            self.raw_full[slot].arrive()
        elif self.mma:
            kind, slot, tile, b, who, commits = self.mma.pop(0)
            self.expect(self.op_holds.get(slot) == tile, ("operand", slot, tile, self.op_holds.get(slot)))
            if kind == "S":
                self.s_holds[b] = who
            else:
                self.expect(len(self.p_holds.get(who, ())) == self.WARPS, ("weights", who))
            for c in commits:
                c.arrive()

    def go(self, steps=200000):
        roles = [self.copy(), self.mma_role()]
        roles += [self.convert(g) for g in range(self.groups) for _ in range(self.WARPS)]
        roles += [self.softmax(m, w) for m in range(2) for w in range(self.WARPS)]
        live = list(roles)
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


RUNS = [[(1, 1)], [(2, 1)], [(7, 1)], [(1, 2)], [(5, 2)], [(3, 1), (1, 1), (4, 1), (2, 1)],
        [(2, 2), (3, 1), (1, 2), (6, 1), (1, 1)], [(1, 1)] * 5]


@pytest.mark.parametrize("runs", RUNS)
@pytest.mark.parametrize("raw", [3, 5])
def test_every_poll_is_for_the_phase_it_means(runs, raw):
    for seed in range(40):
        m = Model(runs, random.Random(seed), raw=raw)
        assert m.go(), ("does not end", seed, m.bad)
        assert not m.bad, (seed, m.bad[:3])


def test_one_barrier_for_both_weights_fails():
    assert any(not (m := Model([(9, 1)], random.Random(s), one_p=True)).go() or m.bad for s in range(200))


def test_odd_rings_shared_by_two_groups_fail():
    assert any(not (m := Model([(12, 1)], random.Random(s), ops=4, raw=3, groups=2)).go() or m.bad
               for s in range(300))
    for s in range(40):
        m = Model([(12, 1), (3, 1)], random.Random(s), ops=4, raw=4, groups=2)
        assert m.go() and not m.bad, (s, m.bad[:3])
