"""The order of waits in the dQ kernel of differential attention, on a model of its roles.

A wait on an mbarrier knows its phase by parity alone: it is only sound while the phase after the awaited one cannot
complete before the waiting thread has passed.  The model runs the kernel's roles (loader, issuer, two of the compute
warps) with its rings, barriers and products in random orders, one compute warp far behind the others, and compares what
every test of a parity answers with what has happened.
"""
import random

import pytest


class Bar:
    """An mbarrier: phases complete one after the other, each after ``count`` arrivals."""

    def __init__(self, count=1):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.count

    def passes(self, phase):
        answer, truth = (self.done & 1) != (phase & 1), self.done > phase
        if answer != truth:
            raise AssertionError(f"a wait for phase {phase} reads {answer} with {self.done} phases complete")
        return truth


class Dq:
    """One block of the dQ kernel.  ``v_at_end``: the compute warps also wait for V behind an item's last tile."""

    COMPUTE = 2

    def __init__(self, items, kr, vr, v_at_end):
        self.items, self.kr, self.vr, self.v_at_end = items, kr, vr, v_at_end
        self.q_full, self.q_empty = Bar(), Bar()
        self.k_full, self.k_empty = [Bar() for _ in range(kr)], [Bar() for _ in range(kr)]
        self.v_full, self.v_empty = [Bar() for _ in range(vr)], [Bar() for _ in range(vr)]
        self.s_full, self.dp_full = [Bar(), Bar()], Bar()
        self.dq_done, self.dq_free = Bar(), Bar(self.COMPUTE)
        self.arrived = {"P": 0, "DS": 0}  # of the named barriers between the compute warps and the issuer
        self.copies, self.products = [], []  # in flight: barriers; per product the barriers it completes

    def loader(self):
        G = 0
        for it, n in enumerate(self.items):
            if it:
                yield lambda: self.q_empty.passes(it - 1)
            self.copies.append(self.q_full)
            for _ in range(n):
                k, v = G % self.kr, G % self.vr
                if G >= self.kr:
                    yield lambda: self.k_empty[k].passes(G // self.kr - 1)
                self.copies.append(self.k_full[k])
                if G >= self.vr:
                    yield lambda: self.v_empty[v].passes(G // self.vr - 1)
                self.copies.append(self.v_full[v])
                G += 1

    def met(self, name):
        if self.arrived[name] < self.COMPUTE:
            return False
        self.arrived[name] -= self.COMPUTE
        return True

    def issuer(self):
        G0 = 0
        for it, n in enumerate(self.items):
            yield lambda: self.q_full.passes(it)
            yield lambda: self.k_full[G0 % self.kr].passes(G0 // self.kr)
            self.products.append([self.s_full[0]])
            yield lambda: self.v_full[G0 % self.vr].passes(G0 // self.vr)
            self.products.append([self.dp_full, self.v_empty[G0 % self.vr]])
            self.products.append([self.s_full[1]] + ([self.q_empty] if n == 1 else []))
            for g in range(n):
                G, more = G0 + g, g + 1 < n
                yield lambda: self.met("P")
                if g == 0 and it:
                    yield lambda: self.dq_free.passes(it - 1)
                if more:
                    self.products.append([self.s_full[0]])
                    self.products.append([self.dp_full, self.v_empty[(G + 1) % self.vr]])
                yield lambda: self.met("DS")
                self.products.append([self.k_empty[G % self.kr]])
                if more:
                    self.products.append([self.s_full[1]] + ([self.q_empty] if g + 2 == n else []))
            self.products.append([self.dq_done])
            G0 += n

    def compute(self):
        G = 0
        for it, n in enumerate(self.items):
            for g in range(n):
                more = g + 1 < n
                k = G + 1 if more else G
                yield lambda: self.s_full[0].passes(G)
                yield lambda: self.k_full[k % self.kr].passes(k // self.kr)
                yield lambda: self.dp_full.passes(G)
                if more or self.v_at_end:
                    yield lambda: self.v_full[k % self.vr].passes(k // self.vr)
                self.arrived["P"] += 1
                yield lambda: self.s_full[1].passes(G)
                self.arrived["DS"] += 1
                G += 1
            yield lambda: self.dq_done.passes(it)
            self.dq_free.arrive()

    def run(self, rng):
        # the engines take their turns like the roles; products end in order, copies in any
        def copy_ends():
            if self.copies:
                self.copies.pop(rng.randrange(len(self.copies))).arrive()

        def product_ends():
            if self.products:
                for bar in self.products.pop(0):
                    bar.arrive()

        roles = [self.loader(), self.issuer(), *(self.compute() for _ in range(self.COMPUTE))]
        waits = [next(r, None) for r in roles]
        idle = 0
        while any(w is not None for w in waits):
            late = len(roles) - 1  # this compute warp moves in one turn of fifty
            who = rng.choice([*range(len(roles) + 2)])
            if who == late and rng.random() < 0.98:
                continue
            before = sum(w is None for w in waits), len(self.copies), len(self.products)
            if who == len(roles):
                copy_ends()
            elif who > len(roles):
                product_ends()
            elif waits[who] is not None and waits[who]():
                waits[who] = next(roles[who], None)
                idle = 0
            idle = idle + 1 if before == (sum(w is None for w in waits), len(self.copies), len(self.products)) else 0
            assert idle < 100000, "nothing moves"
        assert self.dq_done.done == len(self.items)


CASES = [([2, 3, 1, 4, 2], 3, 2), ([1, 2, 1, 1, 3], 3, 2), ([7, 1, 8, 6], 6, 5)]


@pytest.mark.parametrize("items,kr,vr", CASES)
def test_every_wait_names_its_phase(items, kr, vr):
    for seed in range(60):
        Dq(items, kr, vr, v_at_end=False).run(random.Random(seed))


@pytest.mark.parametrize("items,kr,vr", CASES)
def test_the_model_finds_a_phase_that_runs_ahead(items, kr, vr):
    """Behind the last tile dA has freed the slot of V, so V's barrier may have gone on: the model sees a wait for it."""
    with pytest.raises(AssertionError, match="a wait for phase"):
        for seed in range(200):
            Dq(items, kr, vr, v_at_end=True).run(random.Random(seed))
