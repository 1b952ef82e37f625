"""Scores and lengths at the edges of the paged attention: NaN in keys and
queries that are seen, in every division of the work."""

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
