"""The sharing out of latent tree calls, modelled on the CPU and checked by
brute force, and what the calls of test_gpu_latent_cuts.py are there for (no GPU)."""
import random

import numpy as np
import pytest

from _latent_counts import CASES, GROUP, expected, tolerance
from _latent_plan import FEW, PAIRS, check, plan
from tree_speculative_decoding_attn_gb300 import _build
from tree_speculative_decoding_attn_gb300 import specverify as sv


@pytest.mark.parametrize("name", CASES)
def test_cases_are_shared_out_as_they_say(name):
    lengths, nodes, heads, latent, _, kernel, mode, form = CASES[name]
    p = plan(lengths, nodes, heads, latent)
    assert (p.kernel, p.mode, p.form) == (kernel, mode, form), p
    check(p, lengths, nodes, heads)
    assert mode == "whole" or len(p.cuts) > 0


@pytest.mark.parametrize("name", CASES)
def test_the_library_plans_as_the_model(name):
    """Which kernel takes a call, and its parts, from the workspace that it asks for."""
    _build.build()
    lengths, nodes, heads, latent, *_ = CASES[name]
    p = plan(lengths, nodes, heads, latent)
    k = FEW if p.kernel == "few" else PAIRS
    size = sv.tree_attn_latent_workspace_bytes(sv.BF16, len(lengths), nodes, heads, latent, 64, max(x or 0 for x in lengths))
    assert size == 16 * k["most"] + 2 * p.parts * k["rows"] * (latent + 2) * 4


def test_cases_reach_every_join_of_either_kernel():
    cut = {(c[5], c[3], c[7]) for c in CASES.values() if c[6] != "whole"}
    assert {("pairs", l, f) for l in (256, 512) for f in (0, 1, 8)} <= cut
    assert {("few", l, f) for l in (256, 512) for f in (1, 8)} <= cut
    full = 0
    for lengths, nodes, heads, latent, *_ in CASES.values():
        for mine in plan(lengths, nodes, heads, latent).segments:
            # a piece of a unit, whole ones, and a piece of another
            full += len(mine) > 2 and mine[0][2] > 0 and mine[-1][3] < mine[-1][4]
    assert full > 10


def test_random_calls():
    rng = random.Random(7)
    seen = set()
    for _ in range(2500):
        batch = rng.choice([1, 2, 3, 4, 8, 31, 32, 33, 64, 100, 153, 200])
        top = rng.choice([0, 1, 64, 129, 1000, 5000, 40000, 100000]) if batch <= 64 else rng.choice([0, 200, 1500])
        equal = rng.random() < 0.5
        lengths = [top if equal else rng.randint(0, top) for _ in range(batch)]
        if rng.random() < 0.3:
            lengths = [None if rng.random() < 0.2 else x for x in lengths]
        nodes, heads = rng.choice([1, 1, 2, 5, 32, 60, 129, 256]), rng.choice([1, 3, 16, 16, 40, 64, 128])
        if batch * nodes * heads > 40000:
            continue
        latent = rng.choice([256, 512])
        p = plan(lengths, nodes, heads, latent, max(1, top * rng.choice([1, 1, 1, 3])))
        check(p, lengths, nodes, heads)
        assert p.parts <= 152 and all(n <= p.parts for _, _, n in p.cuts.values())
        seen.add((p.kernel, p.mode, p.form))
    assert {m for _, m, _ in seen} == {"whole", "cut", "halves"} and len(seen) >= 8


@pytest.mark.parametrize("name", CASES)
def test_a_lost_or_doubled_group_shows(name):
    """What the GPU results are compared with moves far past the tolerance where
    one group of keys is left out or taken twice."""
    lengths, nodes, heads, latent, *_ = CASES[name]
    rng = random.Random(len(name))
    mask = np.ones((1, 1), bool)
    every = sorted({x for x in lengths if x})
    for length in rng.sample(every, min(5, len(every))):
        good = expected(length, 1, 2, latent, mask)
        n = -(-length // GROUP)
        for at in {0, n - 1, rng.randrange(n)}:
            for times in (0, 2):
                groups = np.ones(n)
                groups[at] = times
                bad = expected(length, 1, 2, latent, mask, groups)
                for h in range(2):
                    if h == 1 and at % 2 == 1:
                        continue                    # odd rows do without odd groups
                    moved = np.abs(bad[0, h] - good[0, h])
                    tol = tolerance(good[0, h], 2.0 ** -8)
                    assert (moved > 4 * tol + 1e-12).any(), (length, at, times, h)
