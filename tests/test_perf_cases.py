"""The cases of perf/operators.py on the CPU: every seed's draw ends, and stays
within the sizes that the file states."""

import random
import signal

import pytest

from perf import operators

SEEDS = 6000


@pytest.fixture
def limit():
    def late(*_):
        raise TimeoutError("draw() does not return")

    before = signal.signal(signal.SIGALRM, late)
    signal.alarm(60)
    yield
    signal.alarm(0)
    signal.signal(signal.SIGALRM, before)


def test_every_draw_ends_within_its_bounds(limit):
    for seed in range(SEEDS):  # 1152: one sequence with too many rows of queries to begin with
        c = operators.draw(random.Random(seed))
        d = c["d"]
        if c["op"] == "rope":
            assert c["B"] * c["H"] * c["N"] * d <= 4 * 16 * 8192 * 128, (seed, c)
        elif c["op"] == "append":
            assert 1 <= c["N"] <= 4096 and c["Lmin"] <= c["Lmax"] <= 8192, (seed, c)
        elif c["op"] == "prefix":
            assert c["B"] >= 1 and c["Nq"] >= 1 and c["B"] * c["Hq"] * c["Nq"] <= 16384, (seed, c)
            assert c["P"] % c["page"] == 0 and c["P"] <= 32768 and c["Lmin"] == c["Nq"] <= c["Lmax"], (seed, c)
        else:
            assert 1 <= c["Nq"] <= 1000 and c["Lmin"] <= c["Lmax"], (seed, c)
        if c["op"] != "rope":
            assert c["Hq"] % c["Hkv"] == 0 and c["page"] % 16 == 0, (seed, c)


def test_listed_cases_are_named_apart_and_have_work():
    names = [c["name"] for c in operators.listed()]
    assert 4 <= len(names) <= 12 and len(set(names)) == len(names)
    for c in operators.listed():
        w = operators.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0
