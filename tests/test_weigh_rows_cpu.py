"""The ring of what belongs to the rows (-L, exponents) in the key weights (csrc/fa_weigh.cuh): eight slots, written when
the products of the tile four (or two) before are done, read by two warpgroups, of which the second has no part in units
of one key tile. A model of the roles in which that warpgroup is as slow as the waits let it be and the writer as fast:
with the kernel's waits nothing is written that is still to be read; with waits that know of the scores only, there
is."""
import random

import pytest

SLOTS = 8


class Late(Exception):
    pass


class Barrier:
    """Phases as mbarrier has them: a wait for a parity passes while the phase under way has the other one."""

    def __init__(self):
        self.phase = 0

    def passes(self, parity):
        return (self.phase & 1) != parity


class SecondGroup:
    """What it does, in order: of every product the scores read (s_empty) and what belongs to the rows read, and after a
    unit that one of one key tile follows, `paused`."""

    def __init__(self):
        self.todo, self.step, self.products = [], 0, 0
        self.s_empty, self.paused = [Barrier(), Barrier()], Barrier()

    def product(self, tile):
        self.todo += [("scores", self.products & 1), ("read", tile)]
        self.products += 1

    def wait(self, barrier, parity):
        while not barrier.passes(parity):
            assert self.step < len(self.todo), "nothing left that could end this wait"
            what, x = self.todo[self.step]
            self.step += 1
            if what == "scores":
                self.s_empty[x].phase += 1
            elif what == "pause":
                self.paused.phase += 1

    def unread(self):
        return [x for what, x in self.todo[self.step:] if what == "read"]


def run(units, q_slots, kernel):
    """units: (two key tiles, tiles of rows, the rows are those of before)."""
    group, tile, written, pause, pauses, before = SecondGroup(), -1, 0, False, 0, False

    def write_up_to(t):
        nonlocal written
        while written <= t:
            if any(r % SLOTS == written % SLOTS and r != written for r in group.unread()):
                raise Late
            written += 1

    def end_pause():
        nonlocal pause, pauses
        if pause and kernel:
            group.wait(group.paused, pauses & 1)
            pauses += 1
        pause = False

    for i, (two, rows, same) in enumerate(units):
        if two:
            end_pause()
        pause = pause or (before and not two)
        before = two
        for _ in range(rows):
            if not same:
                write_up_to(tile + q_slots)  # q_empty of the tile before: its products are done as soon as they please
                end_pause()
                if not kernel and not two:
                    for n in (group.products - 1, group.products - 2):
                        if n >= 0:
                            group.wait(group.s_empty[n & 1], (n >> 1) & 1)
                tile += 1
                write_up_to(tile)
            if two:
                n = group.products
                group.wait(group.s_empty[n & 1], ((n >> 1) & 1) ^ 1)
                group.product(tile)
        if two and i + 1 < len(units) and not units[i + 1][0]:
            group.todo.append(("pause", None))
    return group, pauses


def some_units(rng):
    units = []
    while len(units) < 120:
        two, rows = rng.random() < 0.5, rng.choice([1, 1, 1, 2, 5])
        for _ in range(rng.choice([1, 2, 3, 12])):
            units.append((two, rows, rows == 1 and bool(units) and units[-1][1] == 1 and rng.random() < 0.4))
    return units


@pytest.mark.parametrize("q_slots", [2, 4])
def test_nothing_is_written_that_is_still_to_be_read(q_slots):
    rng = random.Random(q_slots)
    for _ in range(400):
        group, pauses = run(some_units(rng), q_slots, True)
        # no pause is passed over: every wait was for the phase that it meant
        assert pauses <= sum(what == "pause" for what, _ in group.todo) <= pauses + 1 and group.paused.phase >= pauses


@pytest.mark.parametrize("q_slots", [2, 4])
def test_scores_read_are_not_enough(q_slots):
    """One product of the second warpgroup, then a run of units of one key tile."""
    units = [(True, 1, False)] + [(False, 1, False)] * 12
    run(units, q_slots, True)
    with pytest.raises(Late):
        run(units, q_slots, False)
