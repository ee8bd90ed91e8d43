"""The ring of K and V stages in the tcgen05 attention kernel
(csrc/k_attn_chunk.cuh), checked as a model under random interleavings on the
CPU.

Stage i of an item's steps is K (even) or V (odd), in slot i % ST:
  loads     wait EMPTY(slot) of the use before; start the copy -> FULL(slot)
  products  wait FULL in order; for V of a partial step also FIX(slot); the
            product's commit -> one arrival at EMPTY(slot)
  V warp    waits FULL of every stage in order; in a partial step looks at V,
            then -> FIX(slot)
A wait names a phase by its parity alone: it passes while the barrier has
completed as many phases, modulo two, as the waiter expects. A waiter that
falls two phases behind waits for what is over, and one that falls further
behind takes a later phase for its own. In steps that are not partial nothing
but the ring itself ties the V warp to the others, so its own arrival has to
be one of those that free a stage. How many arrivals free one is read from
the source.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_lm_gen_b200", "csrc",
                      "k_attn_chunk.cuh")


def releases():
    """Arrivals that free a stage: CH_RELEASES, and that the V warp makes its own, for K and on both ways for V."""
    with open(SOURCE) as f:
        text = f.read()
    m = re.search(r"constexpr int CH_RELEASES = (\d+);", text)
    if not m:
        return 1
    assert re.search(r"i >= B::EMPTY && i < B::EMPTY \+ ST \? CH_RELEASES", text)
    v_warp = text[text.index("V at the ends of the range", text.index("loads: lane e issues")):]
    assert [v_warp.count(f"mbar_arrive(&bars[B::EMPTY + {x}])") for x in ("kv % ST", "slot")] == [1, 2]
    return int(m.group(1))


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "more arrivals than the phase has"
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, phase):
        """As try_wait.parity does: by the parity of the phases that are complete."""
        return (self.done & 1) != (phase & 1)


def run(stages, steps, partial, seed, free, starve):
    """One interleaving of `steps` steps. `starve`: rounds in which the V warp does not get to run."""
    rng = random.Random(seed)
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(free) for _ in range(stages)]
    fix = [Barrier(1) for _ in range(stages)]
    late = []                                   # copies and products under way: [rounds, barrier]

    def loads():
        for i in range(2 * steps):
            if i >= stages:
                yield empty[i % stages], i // stages - 1
            late.append([rng.randint(1, 4), full[i % stages]])

    def products():
        fixed = [0] * stages
        for i in range(2 * steps):
            yield full[i % stages], i // stages
            if i & 1 and partial(i // 2):
                yield fix[i % stages], fixed[i % stages]
                fixed[i % stages] += 1
            late.append([rng.randint(1, 3), empty[i % stages]])

    def v_warp():
        for i in range(2 * steps):
            yield full[i % stages], i // stages
            assert full[i % stages].done == i // stages + 1, "the V warp took a later phase for its own"
            if i & 1 and partial(i // 2):
                fix[i % stages].arrive()
            if free == 2:
                empty[i % stages].arrive()

    roles = {"loads": loads(), "products": products(), "v": v_warp()}
    at = {k: next(g, None) for k, g in roles.items()}
    idle = rounds = 0
    while any(w is not None for w in at.values()) or late:
        rounds += 1
        moved = False
        for x in list(late):
            x[0] -= 1
            if x[0] <= 0:
                late.remove(x)
                x[1].arrive()
            moved = True
        names = list(roles)
        rng.shuffle(names)
        for k in names:
            if at[k] is None or (k == "v" and rounds % (starve + 1)):
                continue
            bar, phase = at[k]
            if bar.passes(phase):
                at[k] = next(roles[k], None)
                moved = True
        idle = 0 if moved else idle + 1
        assert idle <= 2 * (starve + 1), f"nothing moves: {[k for k, w in at.items() if w]} wait"
    assert all(b.left == b.count for b in full + empty + fix)


PARTIAL = {"none": lambda s: False, "ends": lambda s: s in (0, 38, 39), "all": lambda s: True}


@pytest.mark.parametrize("stages", [4, 8])
@pytest.mark.parametrize("partial", list(PARTIAL))
@pytest.mark.parametrize("starve", [0, 3, 17, 200])
def test_the_v_warp_keeps_up_however_late_it_runs(stages, partial, starve):
    for seed in range(10):
        run(stages, 40, PARTIAL[partial], seed, releases(), starve)


@pytest.mark.parametrize("stages", [4, 8])
def test_the_model_sees_a_ring_that_does_not_wait_for_it(stages):
    with pytest.raises(AssertionError):
        for seed in range(10):
            run(stages, 40, PARTIAL["ends"], seed, 1, 17)
