"""The steps of the attention kernel of many rows (csrc/attn_chunk.cu, watch and issue_products), on the host.

The watcher lets the issuer go from step to step through eight hardware barriers in turn: it arrives
and goes on, the issuer waits.  Here both are generators over the same items, run in any order, and
the watcher's waits may run out at any place: both have to end, whatever the order."""

import random

import pytest

BARRIERS = 8


class Block:
    def __init__(self, items, start, units, streams):
        self.items, self.start, self.units, self.streams = items, start, units, streams  # items: units each
        self.arrived, self.dead, self.scores = [0] * BARRIERS, False, set()


def watch(b, stop):
    """Yields where it waits: what has to hold before it goes on."""
    step, needs, alive = 0, 0, True

    def need(ready):
        nonlocal needs, alive
        if alive:
            if needs == stop:
                b.dead, alive = True, False
                return
            needs += 1
            while not ready():
                if b.dead:
                    alive = False
                    return
                yield

    def go():
        nonlocal step
        b.arrived[step % BARRIERS] += 1
        step += 1
        return alive

    item, unit = 0, b.start
    yield from need(lambda: True)
    if not go():
        return
    for u in range(b.units):
        more, last = u + 1 < b.units, unit + 1 == b.items[item]
        if more:
            if last:
                yield from need(lambda: True)  # the next item is known
                if alive:
                    item, unit = item + 1, 0
            else:
                unit += 1
        if b.streams == 2:
            for s in range(2):
                yield from need(lambda: (u, s) in b.scores)  # weights follow scores
                if not go():
                    return
                if more and last:
                    yield from need(lambda: True)
                    if not go():
                        return
        else:
            if more and not last:
                yield from need(lambda: True)
                if not go():
                    return
            yield from need(lambda: (u, 0) in b.scores)
            if not go():
                return
            if more and last:
                yield from need(lambda: True)
                if not go():
                    return


def issue(b):
    step, gone = 0, False

    def come():
        nonlocal step, gone
        if b.dead:
            gone = True
            return
        i = step % BARRIERS
        while b.arrived[i] == 0:
            yield
        b.arrived[i] -= 1
        step += 1

    yield from come()
    if gone or b.dead:
        return
    item, unit = 0, b.start
    for s in range(b.streams):
        b.scores.add((0, s))
    for u in range(b.units):
        more, last = u + 1 < b.units, unit + 1 == b.items[item]
        unit = 0 if last else unit + 1

        def following():
            nonlocal item
            yield from come()
            if not gone:
                if last:
                    item += 1
                b.scores.add((u + 1, 0))

        if b.streams == 2:
            for s in range(2):
                yield from come()
                if gone:
                    return
                if more:
                    if last:
                        yield from come()
                        if gone:
                            return
                        if s == 0:
                            item += 1
                    b.scores.add((u + 1, s))
        else:
            if more and not last:
                yield from following()
                if gone:
                    return
            yield from come()
            if gone:
                return
            if more and last:
                yield from following()
                if gone:
                    return


def run(b, stop, rng, elsewhere=None):
    """Whether both end; `elsewhere`: the turn in which a wait of another task runs out."""
    tasks = [watch(b, stop), issue(b)]
    for turn in range(4000):
        if not tasks:
            return True
        if turn == elsewhere:
            b.dead = True
        t = rng.choice(tasks)
        try:
            next(t)
        except StopIteration:
            tasks.remove(t)
        assert max(b.arrived) <= 1  # two arrivals would let a barrier go without the issuer
    return not tasks


WORK = [([1], 0, 1), ([1, 1, 1, 1], 0, 4), ([5, 3], 2, 6), ([2, 1, 4, 1, 1, 3], 1, 10), ([30], 3, 20)]


@pytest.mark.parametrize("streams", [1, 2])
@pytest.mark.parametrize("items,start,units", WORK)
def test_both_end_wherever_a_wait_runs_out(items, start, units, streams):
    rng = random.Random(units)
    most = 8 * units + 8
    for stop in range(most):
        for _ in range(6):
            assert run(Block(items, start, units, streams), stop, rng), stop
    for elsewhere in range(0, 6 * most, 3):
        assert run(Block(items, start, units, streams), -1, rng, elsewhere), elsewhere


@pytest.mark.parametrize("streams", [1, 2])
@pytest.mark.parametrize("items,start,units", WORK)
def test_every_unit_is_issued_where_no_wait_runs_out(items, start, units, streams):
    rng = random.Random(units)
    for _ in range(20):
        b = Block(items, start, units, streams)
        assert run(b, -1, rng)
        assert b.scores == {(u, s) for u in range(units) for s in range(streams)} and max(b.arrived) == 0
