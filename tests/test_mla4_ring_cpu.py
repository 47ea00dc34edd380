"""The barriers of the 4-bit attention kernel, followed step by step on the CPU.

The kernel's roles (decode warps, the two issuing warps, softmax warps) and its tensor-core queues are walked in many
orders.  A wait on an mbarrier sees one bit of its phase, so a role that is two phases behind passes a wait at once; each
wait here says which phase it means, and passing before that phase is complete is the fault looked for.  Whether the
decode warps wait for a slot of the ring that a row's query takes is read off the kernel's source.
"""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SLOTS = 3


def skip_query_waits():
    src = open(os.path.join(ROOT, "long_context_sparse_11_b200", "csrc", "mla4.cuh")).read()
    body = re.search(r"auto skip_query = \[&\] \{(.*?)\n    \};", src, re.S).group(1)
    assert "mbar_arrive(bar(B_FULL + ring.slot))" in body
    wait = body.find("wait(B_EMPTY + ring.slot, ring.phase ^ 1)")
    return 0 <= wait < body.find("mbar_arrive")


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):
        return (self.done & 1) != parity


class Ring:
    """Uses of the slots in order; use u of a slot ends with phase u of its barriers."""

    def __init__(self):
        self.n = 0

    def take(self):
        slot, use = self.n % SLOTS, self.n // SLOTS
        self.n += 1
        return slot, use


def roles(rows, skip_waits, queues):
    """Generators of ("wait", barrier, phase) and ("arrive", barrier), and the issuers' pushes to their queues, for rows
    of these numbers of tiles."""
    n = sum(rows)
    item = {sum(rows[:r]): r for r in range(len(rows))}  # a row's first tile

    def last(i):
        return i + 1 in item or i + 1 == n

    def decode():
        ring = Ring()

        def query():
            slot, use = ring.take()
            if skip_waits:
                yield "wait", ("empty", slot), use - 1
            yield "arrive", ("full", slot), None
        yield from query()
        for i in range(n):
            slot, use = ring.take()
            yield "wait", ("empty", slot), use - 1
            if i:
                yield "wait", ("rfree",), i - 1
            yield "arrive", ("full", slot), None
            if last(i) and i + 1 < n:
                yield from query()

    def issue_s():
        ring = Ring()
        for i in range(n):
            if i in item:
                slot, use = ring.take()
                yield "wait", ("full", slot), use
                yield "wait", ("qfull",), item[i]
                if i:
                    yield "wait", ("sfull",), i - 1
                queues[0].append(("empty", slot))
            if i:
                yield "wait", ("sread",), i - 1
            slot, use = ring.take()
            yield "wait", ("full", slot), use
            queues[0].extend([("rfree",), ("sfull",)])
            yield "arrive", ("sfull",), None

    def issue_pv():
        ring = Ring()
        for i in range(n):
            if i in item:
                ring.take()
            slot, _ = ring.take()
            yield "wait", ("pfull",), i
            queues[1].extend([("empty", slot), ("pvdone",)])

    def softmax():
        ring = Ring()
        ring.take()
        yield "arrive", ("qfull",), None
        for i in range(n):
            yield "wait", ("sfull",), i
            yield "arrive", ("sread",), None
            if i:
                yield "wait", ("pvdone",), i - 1
            yield "arrive", ("pfull",), None
            ring.take()
            if last(i):
                if i + 1 < n:
                    slot, use = ring.take()
                    yield "wait", ("empty", slot), use - 1
                    yield "arrive", ("qfull",), None
                yield "wait", ("pvdone",), i

    return [decode(), decode(), issue_s(), issue_pv(), softmax(), softmax()]


def walk(rows, skip_waits, rng):
    """One order of steps to the end.  Returns the first wait that passed too early, or None."""
    bars = {("empty", s): Barrier(1) for s in range(SLOTS)}
    bars.update({("full", s): Barrier(2) for s in range(SLOTS)})
    bars.update({("rfree",): Barrier(1), ("sfull",): Barrier(2), ("qfull",): Barrier(2), ("sread",): Barrier(2),
                 ("pfull",): Barrier(2), ("pvdone",): Barrier(1)})
    queues = ([], [])
    gens = roles(rows, skip_waits, queues)
    todo = [next(g) for g in gens]
    weight = [rng.choice([1, 1, 8, 64]) for _ in range(len(gens) + 2)]  # some actors are slow in this order
    while True:
        ready = [i for i, t in enumerate(todo)
                 if t and (t[0] == "arrive" or bars[t[1]].passes(t[2] & 1))]
        ready += [len(gens) + q for q in range(2) if queues[q]]
        if not ready:
            assert not any(todo) and not any(queues), ("nothing can go on", todo)
            return None
        i = rng.choices(ready, [weight[r] for r in ready])[0]
        if i >= len(gens):
            bars[queues[i - len(gens)].pop(0)].arrive()
            continue
        kind, bar, phase = todo[i]
        if kind == "arrive":
            bars[bar].arrive()
        elif bars[bar].done <= phase:
            return i, bar, phase
        todo[i] = next(gens[i], None)


def early(rows, skip_waits, orders=800):
    rng = random.Random(sum(rows))
    found = (walk(rows, skip_waits, rng) for _ in range(orders))
    return next((f for f in found if f), None)


def test_the_walk_finds_a_wait_that_passes_early():
    """Rows of one tile, the decode not waiting for the slots of queries: a tile's slot is taken while its values are
    still read, two phases back."""
    assert early([1] * 8, False, 5000)


@pytest.mark.parametrize("rows", [[1] * 8, [2] * 6, [3] * 5, [4, 4, 1], [4, 4, 2], [5] * 4, [16, 16]], ids=str)
def test_no_wait_of_the_ring_passes_a_phase_early(rows):
    assert early(rows, skip_query_waits()) is None
