"""CPU model of the MXFP4 pair kernel's end after a wait has run out.

The two CTAs of a pair stop at any moment: some loads are on their way to
shared memory, some stages are half announced. Nobody may leave before every
load has landed. The leader's barrier of a stage counts its own producer's
arrival, the bytes of both CTAs' loads (all announced by the leader) and the
scale warps of both CTAs, so that it need not complete by itself any more.

The model runs the roles in random order, stops each CTA at a random time and
then applies the kernel's rule (put in place what will not come, wait). It
checks that every stage's barrier completes, once, and that no load is in
flight then. The plain rule (the leader waits for the stages it has loaded
itself) leaves loads in flight or waits for good.
"""
import random

import pytest

WARPS, BOXES = 4, 2      # scale warps per CTA; boxes that a CTA loads per stage
AHEAD = 4                # scale buffers


class Stage:
    def __init__(self):
        self.pending, self.tx, self.done = 1 + 2 * WARPS, 0, 0

    def change(self, arrivals=0, tx=0):
        self.pending -= arrivals
        self.tx += tx
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.pending, self.done = 1 + 2 * WARPS, self.done + 1


class Pair:
    """One use of a stage per step; use u has stage u % stages."""

    def __init__(self, seed, stages, uses):
        self.rng, self.k, self.uses = random.Random(seed), stages, uses
        self.full = [Stage() for _ in range(stages)]
        self.issued, self.scaled, self.mma = [0, 0], [[0] * WARPS, [0] * WARPS], 0
        self.empty = [0, 0]            # uses whose MMAs are known to be done, per CTA
        self.flight = []               # (use, CTA) of boxes on their way
        self.stopped = [False, False]
        self.speed = {r: self.rng.choice([1, 1, 4]) for r in ("p0", "p1", "s0", "s1", "mma", "land", "e0", "e1")}
        self.speed["land"] = self.rng.choice([0.02, 0.3, 4])       # loads may be slow

    def steps(self):
        out = []
        for r in (0, 1):
            if self.empty[r] < self.mma:
                out.append(("e%d" % r, ("empty", r)))
            if self.stopped[r]:
                continue
            u = self.issued[r]
            if u < self.uses and self.empty[r] > u - self.k:
                out.append(("p%d" % r, ("load", r)))
            for w in range(WARPS):
                u = self.scaled[r][w]
                if u < self.uses and self.empty[r] > u - AHEAD:
                    out.append(("s%d" % r, ("scale", r, w)))
        u = self.mma
        if not self.stopped[0] and u < self.uses and self.full[u % self.k].done > u // self.k:
            out.append(("mma", ("mma",)))
        out += [("land", ("land", i)) for i in range(len(self.flight))]
        return out

    def step(self, what):
        if what[0] == "empty":
            self.empty[what[1]] += 1
        elif what[0] == "load":
            r, u = what[1], self.issued[what[1]]
            if r == 0:
                self.full[u % self.k].change(1, 2 * BOXES)
            self.flight += [(u, r)] * BOXES
            self.issued[r] += 1
        elif what[0] == "scale":
            _, r, w = what
            self.full[self.scaled[r][w] % self.k].change(1)
            self.scaled[r][w] += 1
        elif what[0] == "mma":
            self.mma += 1
        else:
            u, _ = self.flight.pop(what[1])
            self.full[u % self.k].change(0, -1)

    def run(self):
        """Until both CTAs have stopped (or all work is done)."""
        stops = [self.rng.randrange(30 * self.uses) for _ in (0, 1)]
        if self.rng.random() < 0.5:
            stops[1] = stops[0] + self.rng.randrange(10)      # both at nearly the same time
        elif self.rng.random() < 0.4:
            stops[self.rng.randrange(2)] = 10 ** 9        # one CTA notices last: it runs until nothing is left
        for now in range(10 ** 6):
            for r in (0, 1):
                self.stopped[r] = self.stopped[r] or now >= stops[r]
            ready = self.steps()
            if all(self.stopped) or not [s for s in ready]:
                self.stopped = [True, True]
                return
            self.step(self.rng.choices([s[1] for s in ready], [self.speed[s[0]] for s in ready])[0])

    def land_all(self):
        while self.flight:
            self.step(("land", self.rng.randrange(len(self.flight))))

    def last(self, issued, s):
        return issued - 1 - (issued - 1 - s) % self.k if issued > s else -1


def finish(pair):
    """The kernel's rule; the waits of its last line as a list of (stage, completions wanted)."""
    waits = []
    for s in range(pair.k):
        u0, u1 = (pair.last(n, s) for n in pair.issued)
        u = max(u0, u1)
        if u < 0 or pair.full[s].done > u // pair.k:
            continue
        if u0 < u:
            pair.full[s].change(1, BOXES)
        if u1 < u:
            pair.full[s].change(0, -BOXES)
        for n in pair.scaled[0] + pair.scaled[1]:
            if n <= u:
                pair.full[s].change(1)
        waits.append((s, u // pair.k + 1))
    return waits


@pytest.mark.parametrize("stages", [4, 5])
def test_every_load_has_landed(stages):
    for seed in range(400):
        pair = Pair(seed, stages, random.Random(seed).choice([1, 3, 7, 20]))
        pair.run()
        waits = finish(pair)
        while any(pair.full[s].done < n for s, n in waits):
            assert pair.flight, (seed, "waits for good")
            pair.step(("land", pair.rng.randrange(len(pair.flight))))
        assert not pair.flight, (seed, "leaves loads in flight")
        assert all(pair.full[s].done == n for s, n in waits)


def test_the_plain_rule_leaves_loads_behind():
    unwatched = stalled = 0
    for seed in range(400):
        pair = Pair(seed, 5, 20)
        pair.run()
        unwatched += any(u >= pair.issued[0] for u, _ in pair.flight)   # no barrier that the leader waits for
        waits = [(s, pair.last(pair.issued[0], s) // 5 + 1) for s in range(5) if pair.last(pair.issued[0], s) >= 0]
        pair.land_all()
        stalled += any(pair.full[s].done < n for s, n in waits)
    assert unwatched > 20 and stalled > 50, (unwatched, stalled)


def _signals(stages, tiles, per_tile):
    """Signals that cross between the CTAs of a pair where nothing goes wrong, as (receiver, barrier, completion)."""
    out = set()
    for u in range(tiles * per_tile):
        out |= {(0, "full", u), (1, "empty", u)}          # scale warps of CTA 1; MMA commits of CTA 0
    for t in range(tiles):
        out |= {(0, "tnext", t), (1, "tfull", t)}         # epilogue warps of CTA 1; MMA commits
    return out | {(1, "done", 0)}


def _awaited(stages, tiles, per_tile, tails):
    """Those that some thread of the receiver waits for before it leaves. tails: the producers wait for their
    last stages to be used, and the MMA warp for the last tile's hand-over."""
    uses = tiles * per_tile
    out = {(0, "full", u) for u in range(uses)} | {(1, "tfull", t) for t in range(tiles)} | {(1, "done", 0)}
    out |= {(1, "empty", u) for u in range(uses if tails else max(0, uses - AHEAD))}   # producer, scale warps
    return out | {(0, "tnext", t) for t in range(tiles if tails else tiles - 1)}


@pytest.mark.parametrize("stages", [4, 5])
@pytest.mark.parametrize("tiles,per_tile", [(1, 1), (1, 9), (5, 1), (7, 10)])
def test_no_signal_is_on_its_way_to_a_cta_that_leaves(stages, tiles, per_tile):
    """The cluster barrier at the kernel's end does not order signals: each is waited for."""
    assert _signals(stages, tiles, per_tile) <= _awaited(stages, tiles, per_tile, True)
    assert not _signals(stages, tiles, per_tile) <= _awaited(stages, tiles, per_tile, False)


def test_the_kernel_waits_for_its_tails():
    """The two waits in the source, behind the loops over the tiles."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "muon_newton_schulz_05_b200", "csrc", "mxfp4_gemm.cu")).read()
    pair = src[src.index("mx_gemm_pair_kernel(const"):src.index("mx_reduce_kernel(const")]
    producer = pair[pair.index("record->issued = issued;"):pair.index("MMA issuer")]
    assert "mbar_wait(&empty[" in producer
    mma = pair[pair.index("umma_commit_pair(done);"):pair.index("scale producer")]
    assert re.search(r"if \(ok\) mbar_wait\(&tnext\[\(tile - 1\) & 1u\]", mma)
