"""Scores at the edges of what the paged attention takes: NaN in keys and
queries that are seen, in every division of the work, and infinite scores."""

import numpy as np
import pytest
import torch

from tests.helpers import scale_for
from tests.test_paged_gpu import check, make_batch, reference, run

pytestmark = pytest.mark.gpu

WAYS = [
    # what, B, Hq, Hkv, Nq, d, page, prefix, lens_k, bits
    ("steps, a unit a CTA", 3, 8, 2, 1, 128, 16, 0, [40, 64, 17], 16),
    ("steps, pieces, eight warps a row", 2, 8, 2, 2, 128, 64, 0, [3000, 700], 16),
    ("steps, pieces, four warps a row", 24, 32, 8, 1, 64, 32, 0, [300 + i for i in range(24)], 16),
    ("steps, pieces, a warp for two rows", 50, 32, 8, 1, 64, 32, 0, [300 + i for i in range(50)], 16),
    ("steps of 24 rows", 2, 4, 1, 6, 128, 64, 0, [900, 40], 8),
    ("steps of 32 rows", 3, 8, 2, 8, 64, 16, 0, [2000, 64, 333], 8),
    ("tiles, two row tiles on the same rows", 2, 4, 1, 16, 128, 64, 0, [700, 5000], 8),
    ("tiles, cut", 2, 4, 2, 200, 64, 32, 0, [1500, 300], 8),
    ("tiles, cut, d = 128", 1, 3, 1, 300, 128, 48, 0, [4000], 8),
    ("tiles, dealt out whole", 1, 64, 64, 1024, 64, 64, 0, [1024], 8),
    ("tiles, drawn", 32, 10, 10, 300, 64, 64, 0, [300 + i for i in range(32)], 8),
    ("prefix and steps", 20, 8, 2, 1, 128, 64, 1024, [1025 + 17 * i for i in range(20)], 8),
    ("prefix and steps, many rows", 70, 8, 1, 1, 64, 16, 512, [513 + 5 * i for i in range(70)], 8),
    ("prefix and tiles", 3, 4, 2, 90, 64, 16, 640, [730, 1000, 800], 8),
]


@pytest.mark.parametrize("way", WAYS, ids=lambda w: w[0].replace(" ", "-"))
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_nan_of_a_seen_key_or_query_reaches_its_rows_and_no_others(way, place):
    """A NaN in one key of one head and in one query: the rows that have a
    score with it are NaN in O and LSE, in whichever piece it lies; all others
    are what they are without it."""
    _, B, Hq, Hkv, Nq, d, page, prefix, lens, bits = way
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=Nq + d + B)
    n = prefix // page
    prefix_table = table[int(np.argmax(lens)), :n].clone()
    table[:, :n] = prefix_table  # (of no prefix: nothing)
    some = sorted({0, 1 % B, B // 2, B - 1})  # the oracle takes its time
    lens_some = [lens[b] for b in some]
    ref = reference(q[some], kp, vp, table[some], lens_some, None, True)
    G, sick, head = Hq // Hkv, some[-1], Hkv - 1
    at = {"first": 0, "middle": lens[sick] // 2, "last": lens[sick] - 1}[place]
    kq, kk = q.clone(), kp.clone()
    kk[table[sick, at // page], head, at % page, 5] = float("nan")
    kq[some[0], 0, Nq // 2, 3] = float("nan")
    hit = torch.zeros(len(some), Hq, Nq, dtype=torch.bool)
    for i, b in enumerate(some):
        if b == sick or at < prefix:
            first = max(0, at - lens[b] + Nq)  # the first query at or behind the key
            hit[i, head * G:(head + 1) * G, first:] = True
    hit[0, 0, Nq // 2] = True
    kw = dict(prefix=prefix, prefix_table=prefix_table) if prefix else {}
    for o_dtype in (torch.float32, torch.bfloat16):
        o, lse = (t.cpu()[some] for t in run(kq, kk, vp, table, lens, o_dtype=o_dtype, **kw))
        assert torch.equal(torch.isnan(lse), hit), (torch.isnan(lse) ^ hit).nonzero()[:5]
        assert torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
        o[hit], lse[hit] = torch.tensor(ref[0]).to(o_dtype)[hit], torch.tensor(ref[1]).float()[hit]
        check(o, lse, ref, q[some], kp, scale_for(d), bits, way[0])


@pytest.mark.parametrize("way", [w for w in WAYS if min(w[8]) - w[4] > 200 or w[0].startswith("prefix")],
                         ids=lambda w: w[0].replace(" ", "-"))
def test_keys_of_score_minus_infinity_have_no_weight(way):
    """The first 200 keys score -inf and the others about -512: rows are the
    softmax over the others."""
    _, B, Hq, Hkv, Nq, d, page, prefix, lens, bits = way
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=Nq + d + B)
    n = prefix // page
    prefix_table = table[int(np.argmax(lens)), :n].clone()
    table[:, :n] = prefix_table
    q[..., 0], q[..., 1] = 1.0, 64.0
    kp[..., 1] -= 512 / 64 * d ** 0.5  # (NaN where no key is)
    clean = kp.clone()
    for b in range(B):
        for p in range(200):
            kp[table[b, p // page], :, p % page, 0] = -float("inf")
    some = sorted({0, B // 2, B - 1})
    ref = reference(q[some], kp, vp, table[some], [lens[b] for b in some], None, True)
    assert np.all(np.isfinite(ref[1])) and ref[1].max() < -300
    kw = dict(prefix=prefix, prefix_table=prefix_table) if prefix else {}
    o, lse = run(q, kp, vp, table, lens, **kw)
    check(o[some], lse[some], ref, q[some], clean, scale_for(d), bits, way[0])


@pytest.mark.parametrize("way", WAYS, ids=lambda w: w[0].replace(" ", "-"))
def test_an_infinite_key_is_nan_or_nothing(way):
    """One key with +inf in a component that is 1 in some queries and -1 in the
    others: the first have a score of +inf and are NaN, for the others the key
    has no weight."""
    _, B, Hq, Hkv, Nq, d, page, prefix, lens, bits = way
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=Nq + d + B)
    n = prefix // page
    prefix_table = table[int(np.argmax(lens)), :n].clone()
    table[:, :n] = prefix_table
    g = torch.Generator().manual_seed(7)
    up = torch.rand(B, Hq, Nq, generator=g) < 0.4
    q[..., 7] = torch.where(up, 1.0, -1.0).to(q.dtype)
    some = sorted({0, B // 2, B - 1})
    G, sick, head = Hq // Hkv, some[-1], Hkv - 1
    at = lens[sick] // 3
    row = table[sick, at // page], head, at % page, 7
    far, inf = kp.clone(), kp.clone()
    far[row], inf[row] = 2e4, float("inf")  # 2e4: a weight of exp(-1700) and less, 0 in 64 bits
    ref = reference(q[some], far, vp, table[some], [lens[b] for b in some], None, True)
    hit = torch.zeros(len(some), Hq, Nq, dtype=torch.bool)
    for i, b in enumerate(some):
        if b == sick or at < prefix:
            hit[i, head * G:(head + 1) * G, max(0, at - lens[b] + Nq):] = True
    hit &= up[some]
    kw = dict(prefix=prefix, prefix_table=prefix_table) if prefix else {}
    o, lse = (t.cpu()[some] for t in run(q, inf, vp, table, lens, **kw))
    assert torch.equal(torch.isnan(lse), hit) and torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
    o[hit], lse[hit] = torch.tensor(ref[0]).float()[hit], torch.tensor(ref[1]).float()[hit]
    check(o, lse, ref, q[some], kp, scale_for(d), bits, way[0])
