"""No two passes of a training run share random numbers: layers and steps (and
micro-batches) through the offset that `advance` moves. Host side, on the plain
form of the generator."""
import itertools
import os
import re

import numpy as np
import pytest
import torch

import _lowbit_reference as ref
import muon_newton_schulz_05_b200 as mb
from muon_newton_schulz_05_b200 import fourbit

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _layers(sites):
    return [fourbit.Mxfp4Linear((1, 8, 40), 3, p=0.1, site=s, device="cpu") for s in sites]


def test_a_step_of_one_repeats_a_neighbours_numbers():
    """The counter holds offset + site: this is what `advance` has to avoid."""
    a = ref.numbers16(7, 5, 2, 0, 4, 40)
    assert np.array_equal(a, ref.numbers16(7, 6, 1, 0, 4, 40)) and np.array_equal(a, ref.numbers16(7, 7, 0, 0, 4, 40))


@pytest.mark.parametrize("sites", [[0], [0, 1], [0, 1, 2, 3], [3, 0, 7], [5]])
def test_layers_and_steps_share_no_numbers(sites):
    layers, rng = _layers(sites), torch.tensor([7, 2 ** 33 - 3])
    drawn = {}
    for step in range(6):
        for lin in layers:
            for domain in range(3):
                drawn[step, lin.site, domain] = ref.numbers16(7, int(rng[1]), lin.site, domain, 3, 40)
        fourbit.advance(rng, layers)
    assert rng[0] == 7 and rng[1] == 2 ** 33 - 3 + 6 * (max(sites) + 1)
    for a, b in itertools.combinations(drawn.values(), 2):
        assert np.mean(a == b) < 0.1                 # 120 numbers of 16 bits: equal ones are chance


def test_advance_refusals():
    rng = torch.tensor([1, 2])
    with pytest.raises(ValueError, match="different sites"):
        fourbit.advance(rng, _layers([0, 1, 1]))
    for bad in (0, -1, 1.5, True, None):
        with pytest.raises(ValueError):
            mb.advance_rng(rng, bad)
    for bad in (rng.int(), torch.tensor([1, 2, 3])):
        with pytest.raises(ValueError):
            mb.advance_rng(bad, 1)
    assert rng.tolist() == [1, 2]
    for site in (-1, 1 << 62):
        with pytest.raises(ValueError, match="site"):
            _layers([site])
    mb.advance_rng(rng, 3)
    assert rng.tolist() == [1, 5]


def test_the_documents_advance_past_the_sites():
    text = open(os.path.join(ROOT, "README.md")).read()
    example = text[text.index("fourbit import"):]
    example = example[:example.index("```")]
    assert "advance(rng, [lin])" in example and not re.search(r"rng\[1\]\s*\+=", text)
