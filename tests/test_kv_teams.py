"""The paged attention's split as the kernel makes it, without a GPU: teams, walks, slots of parts and groups of joins."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sim(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv") / "kv_teams_sim")
    subprocess.check_call(["g++", "-O1", "-std=c++17", os.path.join(ROOT, "tests", "kv_teams_sim.cpp"), "-o", exe])
    return exe


def run(sim, n_sm, per_sm, row, units, lens):
    tile = 16 if row >= 256 else 4096 // row
    args = [sim] + [str(int(x)) for x in (n_sm, per_sm, row, tile, units, *lens)]
    r = subprocess.run(args, capture_output=True, text=True)
    assert r.returncode == 0, (args[1:], r.stdout)
    tiles, teams, solo, parts = map(int, r.stdout.split())
    assert tiles == sum(-(-n // tile) for n in lens) * units
    return teams, solo, parts


@pytest.mark.parametrize("n_sm", [148, 7])
@pytest.mark.parametrize("row", [64, 128, 256, 512])
def test_every_tile_once(sim, n_sm, row):
    for lens in ([1], [517], [0, 0, 0], [0, 5, 0, 0, 4096, 1, 0], range(0, 900, 7), [131071], [73306], [900] * 7, [4096] * 64, [16] * 5,
                 [700] * 40, [30000] * 8):
        for units in (1, 2, 8, 5):
            run(sim, n_sm, 1 if row == 512 else 2, row, units, list(lens))


def test_random_lengths(sim):
    rng = np.random.default_rng(7)
    seen = set()
    for _ in range(250):
        B = int(np.exp(rng.uniform(0, np.log(300))))
        top = 10 ** rng.uniform(0.3, 5.1)
        lens = (np.full(B, top) if rng.random() < 0.3 else rng.uniform(0, top, B) if rng.random() < 0.5 else top ** rng.uniform(0, 1, B)).astype(int)
        row = int(rng.choice([64, 128, 256, 512]))
        teams, solo, parts = run(sim, int(rng.choice([148, 148, 3, 20])), 1 if row == 512 else 2, row, int(rng.integers(1, 20)), lens)
        seen.add((solo, min(parts, 17) > 1, parts > 16))
    assert {(1, True, False), (0, True, False), (0, True, True)} <= seen  # teams of both kinds, joins of parts and by groups


def test_many_parts_are_joined_by_groups(sim):
    for units, want in ((1, 200), (2, 100)):
        teams, solo, parts = run(sim, 148, 2, 256, units, [73306])
        assert not solo and parts >= want and teams <= 296
