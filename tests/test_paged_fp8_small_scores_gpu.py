"""The paged attention over a cache in E4M3 where scores are zero or next to it:
queries of zeros and tiny ones, cells of the smallest scales, next to masked keys."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from tests.test_paged_fp8_gpu import check, make_batch, reference, run, way_of, with_prefix

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

CASES = [
    # Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q
    (4, 2, 1, 128, 64, 0, [200, 33], None),                  # single tokens
    (8, 2, 6, 64, 16, 0, [150, 77], None),                   # 24 rows
    (4, 1, 16, 128, 64, 0, [200, 141], None),                # 64 rows
    (8, 2, 25, 64, 32, 0, [333, 50], [25, 3]),               # 100 rows, some of them padding
    (4, 2, 100, 128, 128, 0, [300, 110], None),              # a chunk
    (6, 2, 90, 64, 48, 0, [1000, 90], None),
    (8, 2, 2, 128, 64, 256, [300, 150], None),               # behind a prefix, one ends inside it
    (4, 2, 80, 64, 64, 128, [250, 129], None),
]


def ids(c):
    return "x".join(str(x) for x in c[:6])


def check_both(o, lse, ref, q, c, way, what=""):
    """check, whose bound of a log-sum-exp leans on that of the scores, with one
    of its own: the logarithm that the kernels take is off by 2^-22 of itself, and
    is one of a sum that has 1 / scale in it: at most 2^(logs + 14) a key; as much
    again for the merge of partial results."""
    check(o, torch.tensor(ref[1]).float(), ref, q, c, way, what)
    logs = np.abs(np.log2(c.scales[1][torch.isfinite(c.scales[1])].double().numpy())).max()
    top = np.abs(ref[1][np.isfinite(ref[1])]).max()
    keys = np.log2(c.table.numel() * c.page)
    d = q.shape[-1]
    qn, kn = (np.nan_to_num(np.abs(x)).reshape(-1, d) for x in (q.double().numpy(), c.values[0]))
    scores = (d + 8) * 2.0 ** -24 * d ** -0.5 * np.sqrt((qn ** 2).sum(1).max() * (kn ** 2).sum(1).max())
    scores += d ** -0.5 * 2.0 ** (-17 if way == "tiles" else -39) * qn.max() * kn.sum(1).max()  # (see check)
    bound = 2 * 2.0 ** -22 * (logs + 14 + keys) + scores + 2.0 ** -21 * (1 + top)
    got = lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(ref[1])), what
    fin = np.isfinite(ref[1])
    assert np.abs(got[fin] - ref[1][fin]).max() <= bound, what


def go(q, c, case, causal=True):
    Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    kw = with_prefix(c, prefix, lens_k) if prefix else {}
    ref = reference(q, c, lens_k, lens_q, causal)
    for o_dtype in (F32, BF16):
        o, lse = run(q, c, lens_k, lens_q, causal=causal, o_dtype=o_dtype, **kw)
        check_both(o, lse, ref, q, c, way_of(Hq, Hkv, Nq, prefix), case)


@pytest.mark.parametrize("key_scale", [2.0 ** -32, 2.0 ** -22, 1.0])
@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -126, 2.0 ** -110, 2.0 ** -60, 1.0])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_small_queries_and_small_scales(case, q_scale, key_scale):
    """Scores of 0 or next to it: the mean of the values and the logarithm of
    their number.  (Values in cells of 2^-32 that are all zeros are what the
    append makes of zero keys; here the numbers are not zeros.)"""
    Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, c = make_batch(len(lens_k), Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d, q_scale=q_scale)
    live = torch.isfinite(c.scales[0])
    c.scales[0] = torch.where(live, torch.full_like(c.scales[0], key_scale), c.scales[0])
    c.update()
    go(q, c, case, causal=Nq > 1)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_a_batch_of_zeros(case):
    """Zeros appended and attended to, as in a program's first, empty run: O is 0
    and LSE the logarithm of the number of keys that a row sees."""
    Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    B, longest = len(lens_k), max(lens_k)
    pages = B * -(-longest // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
    c = [torch.full((pages, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + [
        torch.full((pages, Hkv, page // 16), float("nan"), device="cuda") for _ in range(2)]
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    zeros = torch.zeros(B, Hkv, longest, d, dtype=BF16, device="cuda")
    fa.kv_append_fp8(zeros, zeros, *c, table, lk, lk)
    q = torch.zeros(B, Hq, Nq, d, dtype=BF16, device="cuda")
    lq = torch.tensor(lens_q if lens_q else [Nq] * B, dtype=torch.int32, device="cuda")
    if prefix:
        table[:, :prefix // page] = table[int(np.argmax(lens_k)), :prefix // page]
        o, lse = fa.forward_shared_prefix_fp8(q, *c, table[0, :prefix // page].clone(), prefix, table, lk, lq)
    else:
        o, lse = fa.forward_paged_fp8(q, *c, table, lk, lq)
    fa.sync_status()
    assert not o.any()
    for b in range(B):
        n = int(lq[b])
        seen = lens_k[b] - n + 1 + torch.arange(n, dtype=torch.float64)
        want = torch.log(seen)
        # 2^-22 of the logarithm of at most 2^(32 + 14 + 11), and as much for a merge
        assert ((lse[b, :, :n].cpu().double() - want).abs() <= 2.0 ** -21 * (57 + want)).all()
        assert torch.isneginf(lse[b, :, n:]).all()


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -60, 1.0, 100.0])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_keys_of_scale_zero(case, q_scale):
    """Keys whose scales are 0 have scores of 0 whatever their numbers are."""
    Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, c = make_batch(len(lens_k), Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d, q_scale=q_scale)
    live = torch.isfinite(c.scales[0])
    c.scales[0] = torch.where(live, torch.zeros_like(c.scales[0]), c.scales[0])
    c.update()
    go(q, c, case, causal=Nq > 1)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_cells_of_scale_zero_beside_others(case):
    """Every third cell of keys has the scale 0, or the smallest that the append
    gives; every fifth query is zeros."""
    Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, c = make_batch(len(lens_k), Hq, Hkv, Nq, d, page, lens_k, seed=3 + Nq + d)
    q.view(-1, d)[::5] = 0.0
    flat = c.scales[0].view(-1)
    live = torch.isfinite(flat)
    some = torch.arange(flat.numel())
    flat[live & (some % 3 == 0)] = 0.0
    flat[live & (some % 3 == 1)] = 2.0 ** -32
    c.update()
    go(q, c, case)


@pytest.mark.parametrize("Hq,Hkv,Nq,prefix", [(4, 2, 1, 0), (8, 2, 4, 0), (8, 2, 8, 0), (4, 2, 40, 0), (4, 2, 100, 0),
                                              (4, 2, 2, 128)])
@pytest.mark.parametrize("high", [30, 45, 60])
@pytest.mark.parametrize("q_scale", [0.0, 1.0, 10.0])
def test_values_of_the_smallest_scale_beside_large_ones(Hq, Hkv, Nq, prefix, high, q_scale):
    """Values' cells of 2^-32, which the append gives to zeros, in turn with cells
    of up to 2^60, one or eight of the small ones at a time."""
    d, page, lens = 128, 64, [1500, 200 + Nq]
    for group in (1, 8):
        q, c = make_batch(2, Hq, Hkv, Nq, d, page, lens, seed=8, q_scale=q_scale)
        kw = with_prefix(c, prefix, lens) if prefix else {}
        cells = torch.arange(c.scales[1].numel()).view(c.scales[1].shape)
        small = cells // group % 2 == 0
        live = torch.isfinite(c.scales[1])
        c.scales[1] = torch.where(live, torch.where(small, 2.0 ** -32, 2.0 ** high), c.scales[1])
        c.update()
        o, lse = run(q, c, lens, **kw)
        check_both(o, lse, reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq, prefix))
