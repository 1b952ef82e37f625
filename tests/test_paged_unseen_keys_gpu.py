"""Infinite scores in keys that a row does not see: whatever stands there, the
row's O and LSE are those of the keys that it sees."""

import numpy as np
import pytest
import torch

from tests.helpers import scale_for
from tests.test_paged_gpu import check, make_batch, reference, run

pytestmark = pytest.mark.gpu

# Queries near a border of 128 keys, so that some end in front of a key tile that
# others reach: in pieces that the row tiles share and in pieces of their own.
CASES = [
    # what, B, Hq, Hkv, Nq, d, page, lens_k, lens_q
    ("64 rows", 1, 4, 1, 16, 128, 64, [136], None),
    ("64 rows, d = 64", 2, 8, 2, 16, 64, 32, [136, 130], None),
    ("100 rows, several sequences", 5, 8, 8, 100, 128, 128, [200, 228, 100, 300, 391], None),
    ("128 rows", 2, 8, 2, 32, 128, 256, [150, 661], None),
    ("rows that are padding", 3, 6, 2, 40, 64, 16, [140, 131, 133], [40, 7, 0]),
    ("both row tiles of 300 rows", 2, 3, 1, 100, 128, 128, [210, 140], None),
    ("a chunk", 1, 4, 2, 300, 64, 64, [400], None),
    ("24 rows", 2, 4, 1, 6, 128, 64, [132, 67], None),
    ("single tokens", 3, 8, 2, 1, 128, 128, [129, 127, 64], None),
]


def fill_stale(pages, table, lens, page, value, column):
    """Rows behind the last key: zeros but for one column."""
    for b, n in enumerate(lens):
        if n % page:
            rows = pages[table[b, n // page], :, n % page:]
            rows.zero_()
            rows[..., column] = value


@pytest.mark.parametrize("stale", [float("inf"), 3e38])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c[0].replace(" ", "-"))
def test_rows_behind_the_last_key(case, stale):
    """They hold an infinity, or finite values whose score overflows, in a
    component that is positive in every query."""
    what, B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    q[..., 7] = 1.5
    ref = reference(q, kp, vp, table, lens_k, lens_q, True)
    filled = kp.clone()
    fill_stale(filled, table, lens_k, page, stale, 7)
    fill_stale(vp, table, lens_k, page, stale, 3)
    for o_dtype in (torch.float32, torch.bfloat16):
        o, lse = run(q, filled, vp, table, lens_k, lens_q, o_dtype=o_dtype)
        check(o, lse, ref, q, kp, scale_for(d), 16 if Hq // Hkv * Nq <= 16 else 8, what)


@pytest.mark.parametrize("case", [c for c in CASES if c[4] > 1], ids=lambda c: c[0].replace(" ", "-"))
def test_later_keys_of_the_sequence(case):
    """Each sequence's last key has a score of +inf with every query: its last
    queries are NaN, the others do not depend on it."""
    what, B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    q[..., 7] = 1.5
    ref = reference(q, kp, vp, table, lens_k, lens_q, True)
    inf = kp.clone()
    hit = torch.zeros(B, Hq, Nq, dtype=torch.bool)
    for b, n in enumerate(lens_k):
        inf[table[b, (n - 1) // page], :, (n - 1) % page, 7] = float("inf")
        queries = lens_q[b] if lens_q else Nq
        if queries:
            hit[b, :, queries - 1] = True
    o, lse = (t.cpu() for t in run(q, inf, vp, table, lens_k, lens_q))
    assert torch.equal(torch.isnan(lse), hit) and torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
    o[hit], lse[hit] = torch.tensor(ref[0]).float()[hit], torch.tensor(ref[1]).float()[hit]
    check(o, lse, ref, q, kp, scale_for(d), 16 if Hq // Hkv * Nq <= 16 else 8, what)


@pytest.mark.parametrize("Nq,B", [(1, 20), (4, 8), (60, 3)])
def test_a_key_of_the_prefix_that_shorter_sequences_do_not_reach(Nq, B):
    """A key of the shared prefix with scores of +inf: the sequences that end in
    front of it do not depend on it, those behind it are NaN."""
    Hq, Hkv, d, page, prefix = 4, 1, 128, 64, 512
    lens = [100 + 13 * b if b % 2 else 560 + 7 * b for b in range(B)]
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=Nq)
    prefix_table = table[int(np.argmax(lens)), :prefix // page].clone()
    table[:, :prefix // page] = prefix_table
    q[..., 7] = 1.5
    ref = reference(q, kp, vp, table, lens, None, True)
    inf = kp.clone()
    inf[prefix_table[500 // page], :, 500 % page, 7] = float("inf")
    hit = torch.zeros(B, Hq, Nq, dtype=torch.bool)
    for b, n in enumerate(lens):
        hit[b, :, :] = n > 500
        for i in range(Nq):
            hit[b, :, i] &= n - Nq + i >= 500
    assert hit.any() and not hit.all()
    o, lse = (t.cpu() for t in run(q, inf, vp, table, lens, prefix=prefix, prefix_table=prefix_table))
    assert torch.equal(torch.isnan(lse), hit) and torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
    o[hit], lse[hit] = torch.tensor(ref[0]).float()[hit], torch.tensor(ref[1]).float()[hit]
    check(o, lse, ref, q, kp, scale_for(d), 8)
