"""The cases of perf/more_operators.py on the CPU: every seed's draw ends and
stays within the sizes that the file states."""

import random

from perf import more_operators as operators

SEEDS = 6000


def test_every_draw_ends_within_its_bounds():
    kinds = set()
    for seed in range(SEEDS):
        c = operators.draw(random.Random(seed))
        kinds.add(c["op"])
        assert c["page"] % 16 == 0 and c["d"] in (64, 128), (seed, c)
        assert 1 <= c["Lmin"] <= c["Lmax"], (seed, c)
        assert all(1 <= n <= c["Lmax"] for n in operators._spread(c)), (seed, c)
        w = operators.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0
        if c["op"] in ("fork", "compact"):
            pages = sum((n + c["page"] - 1) // c["page"] for n in operators._spread(c)) + c.get("spare", 0)
            values = max(pages, c.get("pages", 0)) * c["layers"] * c["Hkv"] * c["page"] * c["d"]
            assert values <= 2 ** 30, (seed, c, values)
        else:
            assert c["Hq"] % c["Hkv"] == 0, (seed, c)
        if c["op"] == "append":
            assert 1 <= c["N"] <= 4096 and c["Lmax"] <= 8192, (seed, c)
        if c["op"] == "prefix":
            assert c["B"] * c["Hq"] * c["Nq"] <= 16384 and c["P"] % c["page"] == 0 and c["P"] <= 32768, (seed, c)
    assert kinds == {"append", "paged", "prefix", "fork", "compact"}


def test_listed_cases_are_named_apart_and_have_work():
    names = [c["name"] for c in operators.listed()]
    assert 4 <= len(names) <= 12 and len(set(names)) == len(names)
    for c in operators.listed():
        w = operators.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0
