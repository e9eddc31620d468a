"""The eviction's search for the border key, without a GPU: a host simulation with the kernel's range arithmetic against the
oracle's sort, over weights that reach the ends of the key range (NaN is the heaviest weight, -inf the lightest)."""
import os
import subprocess

import numpy as np
import pytest

from oracle import paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOG_BINS = {9: 4, 11: 3}  # of CTAs of 128 and of 512 threads, and the passes that 32 bits take at most


@pytest.fixture(scope="module")
def sim(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv") / "kv_border_sim")
    subprocess.check_call(["g++", "-O1", "-std=c++17", os.path.join(ROOT, "tests", "kv_border_sim.cpp"), "-o", exe])
    return exe


def check(sim, cases):
    """cases: (weights, budget, n_recent, n_sink)."""
    runs = [(b,) + c for c in cases for b in LOG_BINS]
    text = "\n".join("%d %d %d %d %d %s" % (b, len(w), budget, recent, sink, " ".join(map(str, w.view(np.uint32))))
                     for b, w, budget, recent, sink in runs)
    r = subprocess.run([sim], input=text, capture_output=True, text=True, timeout=100)
    lines = r.stdout.splitlines()
    assert r.returncode == 0 and len(lines) == len(runs), r.stdout[-200:]
    for line, (b, w, budget, recent, sink) in zip(lines, runs):
        assert line != "endless", (b, len(w), budget, recent, sink)
        passes, *kept = map(int, line.split())
        assert passes <= LOG_BINS[b]
        assert kept == paged.evict_choice(w, len(w), budget, recent, sink), (b, len(w), budget, recent, sink)


def with_nans(rng, n, count, low=None, base=None):
    w = (rng.exponential(size=n) if base is None else base).astype(np.float32)
    w[rng.permutation(n)[:count]] = np.nan
    if low is not None:  # the smallest weight, by its low mantissa bits the grid that the bins start from
        w[~np.isnan(w)] = np.maximum(w[~np.isnan(w)], np.float32(low))
        w[rng.permutation(np.flatnonzero(~np.isnan(w)))[:1]] = low
    return w


@pytest.mark.parametrize("recent,sink", [(20, 4), (60, 4), (0, 0), (0, 100), (100, 0), (3, 1)])
def test_more_nans_than_places(sim, recent, sink):
    rng = np.random.default_rng(recent)
    check(sim, [(with_nans(rng, 300, k, low), 100, recent, sink) for k in (1, 75, 76, 77, 120, 150, 299, 300)
                for low in (None, 0.30078125, 0.3, 1e-30)])


def test_keys_at_the_ends_of_the_range(sim):
    rng = np.random.default_rng(1)
    cases = []
    for _ in range(150):
        n = int(rng.integers(2, 200))
        parts = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-42, 3e38, -3e38, 0.30078125, 0.3], np.float32)
        w = rng.choice(parts[rng.permutation(len(parts))[: int(rng.integers(1, 6))]], n)
        some = rng.random(n) < rng.choice([0.0, 0.3])
        w[some] = rng.standard_normal(int(some.sum())).astype(np.float32) * np.float32(10.0) ** rng.integers(-20, 20)
        budget = int(rng.integers(1, n))
        recent = int(rng.integers(0, budget + 1)) if rng.random() < 0.7 else 0
        cases.append((w, budget, recent, int(rng.integers(0, budget - recent + 1)) if rng.random() < 0.7 else 0))
    check(sim, cases)


def test_ordinary_weights(sim):
    rng = np.random.default_rng(2)
    cases = []
    for _ in range(60):
        n = int(rng.integers(2, 1500))
        budget = int(rng.integers(1, n))
        recent = int(rng.integers(0, budget + 1))
        cases.append((rng.exponential(size=n).astype(np.float32) ** 3 / n, budget, recent, int(rng.integers(0, budget - recent + 1))))
    check(sim, cases)


def test_random_bit_patterns(sim):
    rng = np.random.default_rng(3)
    cases = []
    for _ in range(100):
        n = int(rng.integers(2, 400))
        top = int(rng.choice([0, 0x7F000000, 0xFF000000, 0x7F800000]))
        w = ((rng.integers(0, 1 << 32, n, dtype=np.uint64).astype(np.uint32) & np.uint32(0xFFFFFFFF if top == 0 else 0x00FFFFFF)) | np.uint32(top)).view(np.float32)
        budget = int(rng.integers(1, n))
        cases.append((w, budget, 0, int(rng.integers(0, budget + 1))))
    check(sim, cases)
