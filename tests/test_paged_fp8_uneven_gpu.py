"""The paged attention over a cache in E4M3 where many of a key head's row tiles
have no query, because the sequences have fewer new tokens than the longest: a
row tile then passes over long runs of key tiles and their scales."""

import pytest
import torch

from tests.test_paged_fp8_edges_gpu import Some
from tests.test_paged_fp8_gpu import check, make_batch, reference, run, with_prefix

pytestmark = pytest.mark.gpu

CASES = [
    # B, Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q
    (8, 16, 8, 384, 64, 64, 0, [5000] * 8, [100] * 8),                      # rows 256 to 511 of 768: the second tile only
    (16, 32, 16, 384, 64, 128, 0, [2500 + 100 * i for i in range(16)], [100 + i for i in range(16)]),  # units are drawn
    (6, 9, 3, 512, 128, 16, 0, [4000, 300, 4000, 2600, 64, 3500], [128, 300, 1, 130, 64, 500]),
    (3, 4, 2, 640, 64, 64, 2048, [4500, 3000, 2148], [100, 128, 100]),      # behind a prefix
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(x) for x in c[:7]))
def test_few_queries_of_many_rows(case, causal):
    B, Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B, spread=1.0)
    kw = with_prefix(c, prefix, lens_k) if prefix else {}
    some = sorted({0, B // 2, B - 1})  # the oracle takes its time
    ref = reference(q[some], Some(c, some), [lens_k[b] for b in some], [lens_q[b] for b in some], causal)
    first = run(q, c, lens_k, lens_q, causal=causal, **kw)
    check(first[0][some], first[1][some], ref, q[some], c, "tiles", case)
    for _ in range(5):
        o, lse = run(q, c, lens_k, lens_q, causal=causal, **kw)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    for b in range(B):
        assert not first[0][b, :, lens_q[b]:].any() and torch.isneginf(first[1][b, :, lens_q[b]:]).all()
