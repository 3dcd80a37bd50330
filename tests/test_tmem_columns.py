"""CPU model of tensor-memory columns in the few-row MXFP4 product.

An SM has 512 columns; a CTA of the few-row kernel takes 128 by an allocation
that waits until they are free. With a short K more than four of its CTAs fit
an SM's shared memory and registers, so that some wait. The K parts of a tile
are the CTAs of a cluster, which wait for each other once all of them have
their columns. A CTA that kept its columns during that wait could hold up
another cluster's CTA, whose own cluster holds up this one's.

The model lets CTAs of many clusters, spread over few SMs in random order, run
to their end in random order, and reports the ones that can never go on.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "muon_newton_schulz_05_b200", "csrc")
COLUMNS, TAKEN = 512, 128


def stuck(seed, clusters, split, sms, resident, free_first):
    """CTAs that never end. resident: CTAs that an SM takes at once (what is left
    of a cluster that does not fit starts when there is room for all of it)."""
    rng = random.Random(seed)
    free = [COLUMNS] * sms
    room = [resident] * sms
    waiting = list(range(clusters))
    live = {}                                      # (cluster, rank) -> [sm, state]
    arrived = [0] * clusters

    def place():
        while waiting:
            spots = [s for s in range(sms) for _ in range(room[s])]
            if len(spots) < split:
                return
            rng.shuffle(spots)
            c = waiting.pop(0)
            for r in range(split):
                room[spots[r]] -= 1
                live[c, r] = [spots[r], "alloc"]

    while True:
        place()
        ready = [k for k, (sm, state) in live.items()
                 if (state == "alloc" and free[sm] >= TAKEN) or (state == "cluster" and arrived[k[0]] == split) or
                 state == "work"]
        if not ready:
            return len(live)
        k = rng.choice(ready)
        sm, state = live[k]
        if state == "alloc":
            free[sm] -= TAKEN
            arrived[k[0]] += 1                     # the arrival follows the allocation
            live[k][1] = "work"
        elif state == "work":                      # its loads and MMAs, which need nobody
            if free_first:
                free[sm] += TAKEN
            live[k][1] = "cluster"
        else:
            if not free_first:
                free[sm] += TAKEN
            room[sm] += 1
            del live[k]


@pytest.mark.parametrize("split", [2, 3, 8])
@pytest.mark.parametrize("resident", [4, 5, 7])
def test_columns_freed_before_the_cluster_barrier_never_stall(split, resident):
    assert all(stuck(seed, 40, split, 4, resident, True) == 0 for seed in range(30))


def test_columns_held_across_it_can():
    assert sum(stuck(seed, 40, 3, 4, 7, False) > 0 for seed in range(30)) > 5
    assert all(stuck(seed, 40, 3, 4, 4, False) == 0 for seed in range(30))   # where all columns fit


def test_the_kernel_frees_before_it_waits():
    """The order in the source: in the split branch, columns go before the first cluster barrier."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mxfp4_gemm.cu")).read())
    body = src[src.index("mx_gemm_few_kernel(const"):]
    body = body[:body.index("\nMxGemmPlan ")]
    assert body.count("tmem_alloc(") == body.count("tmem_dealloc(") == 1
    free = re.search(r"auto (\w+) = \[&\] \{[^}]*tmem_dealloc", body)
    before = body[free.end():body.index("cluster_wait()")] if free else ""
    assert "} else {" in before and free.group(1) + "();" in before[before.rindex("} else {"):]
