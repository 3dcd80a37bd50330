"""CPU model of the pair kernel's accumulator hand-over (MXFP4 product).

Tiles alternate between two accumulators that share columns. The MMAs of tile
t + 1 may start once (1) every epilogue warp has read tile t - 1 (the same
accumulator) and (2) the warps that hold tile t's shared columns have read
them. Warps of the half that holds the shared columns (they alternate with the
tiles) arrive after reading them, the others when they come to the tile.
The model runs the warps with random durations and checks (1) and (2) at
every start, with one arrival barrier per accumulator (the kernel's), and
shows that a single barrier for all tiles lets an early arrival for tile
t + 2 stand in for a late one for tile t + 1.
"""
import heapq
import random

import pytest

WARPS = 8   # per half: four of each CTA of the pair


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1


def simulate(seed, tiles, barriers):
    """Returns (violations, finished). Warp states advance by events; the MMA
    starts tile t when its barrier has completed often enough."""
    rng = random.Random(seed)
    slow = [rng.choice([0.2, 1.0, 1.0, 6.0]) for _ in range(2 * WARPS)]
    tnext = [Barrier(2 * WARPS) for _ in range(barriers)]
    mma_done = [None] * tiles
    shared_read = [0] * tiles                     # warps that have read tile t's shared columns
    read = [[False] * tiles for _ in range(2 * WARPS)]
    waiting = {}                                  # warp -> tile it waits for
    violations, started, now = 0, 0, 0.0
    events = []

    def bar(t):
        return tnext[t % barriers]

    def may_start(t):
        # completions of tile t - 1's barrier that tile t needs
        return t == 0 or bar(t - 1).done >= ((t - 1) // barriers) + 1

    def come_to(w, t):
        if t == tiles:
            return
        if (w // WARPS) != (1 - t % 2):           # not the half with the shared columns
            bar(t).arrive()
        waiting[w] = t

    for w in range(2 * WARPS):
        come_to(w, 0)
    mma_free = True
    while True:
        progressed = False
        if mma_free and started < tiles and may_start(started):
            t = started
            if t >= 2 and not all(read[w][t - 2] for w in range(2 * WARPS)):
                violations += 1
            if t >= 1 and shared_read[t - 1] < WARPS:
                violations += 1
            heapq.heappush(events, (now + rng.uniform(0.1, 1.0), "mma", t, 0))
            mma_free, started, progressed = False, started + 1, True
        for w, t in list(waiting.items()):
            if mma_done[t] is not None:
                del waiting[w]
                heapq.heappush(events, (now + slow[w] * rng.uniform(0.1, 1.0), "shared", t, w))
                progressed = True
        if progressed:
            continue
        if not events:
            break
        now, what, t, w = heapq.heappop(events)
        if what == "mma":
            mma_done[t], mma_free = now, True
        elif what == "shared":
            if (w // WARPS) == (1 - t % 2):
                shared_read[t] += 1
                bar(t).arrive()
            heapq.heappush(events, (now + slow[w] * rng.uniform(0.1, 3.0), "rest", t, w))
        else:
            read[w][t] = True
            come_to(w, t + 1)
    return violations, all(all(r) for r in read)


@pytest.mark.parametrize("seed", range(40))
def test_one_barrier_per_accumulator_is_safe_and_never_stalls(seed):
    assert simulate(seed, 30, 2) == (0, True)


def test_a_single_barrier_is_not():
    results = [simulate(seed, 30, 1) for seed in range(40)]
    assert sum(v > 0 or not done for v, done in results) > 20
