"""The paged attention over a cache in E4M3 at the edges of what it takes: NaN in
keys and queries, padding, scales far apart, weights far apart, bad pages and
lengths, streams, graphs, and offsets past 32 bits."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from oracle import serving
from tests.helpers import scale_for, to64
from tests.test_paged_edges_gpu import WAYS
from tests.test_paged_fp8_gpu import Cache, check, make_batch, reference, run, way_of, with_prefix

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Some:
    """Some of a batch's sequences, for the oracle."""

    def __init__(self, c, some):
        self.table, self.values, self.scales, self.page = c.table[some], c.values, c.scales, c.page


@pytest.mark.parametrize("way", WAYS, ids=lambda w: w[0].replace(" ", "-"))
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_nan_of_a_seen_key_or_query_reaches_its_rows_and_no_others(way, place):
    """A NaN in one key of one head, a NaN in one query and an infinity in
    another: the rows that have a score with them are NaN in O and LSE, in
    whichever piece they lie; all others are what they are without."""
    _, B, Hq, Hkv, Nq, d, page, prefix, lens, _ = way
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=Nq + d + B)
    kw = with_prefix(c, prefix, lens) if prefix else {}
    some = sorted({0, 1 % B, B // 2, B - 1})  # the oracle takes its time
    lens_some = [lens[b] for b in some]
    ref = reference(q[some], Some(c, some), lens_some, None, True)
    G, sick, head = Hq // Hkv, some[-1], Hkv - 1
    at = {"first": 0, "middle": lens[sick] // 2, "last": lens[sick] - 1}[place]
    kq = q.clone()
    c.pages[0].view(torch.uint8)[c.table[sick, at // page], head, at % page, 5] = 0x7F
    kq[some[0], 0, Nq // 2, 3] = float("nan")
    kq[some[0], Hq - 1, 0, 7] = -float("inf")
    hit = torch.zeros(len(some), Hq, Nq, dtype=torch.bool)
    for i, b in enumerate(some):
        if b == sick or at < prefix:
            first = max(0, at - lens[b] + Nq)  # the first query at or behind the key
            hit[i, head * G:(head + 1) * G, first:] = True
    hit[0, 0, Nq // 2] = True
    hit[0, Hq - 1, 0] = True  # (sees its own key at least)
    for o_dtype in (F32, BF16):
        o, lse = (t.cpu()[some] for t in run(kq, c, lens, o_dtype=o_dtype, **kw))
        assert torch.equal(torch.isnan(lse), hit), (torch.isnan(lse) ^ hit).nonzero()[:5]
        assert torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
        o[hit], lse[hit] = torch.tensor(ref[0]).to(o_dtype)[hit], torch.tensor(ref[1]).float()[hit]
        check(o, lse, ref, q[some], c, way_of(Hq, Hkv, Nq, prefix), way[0])


@pytest.mark.parametrize("Hq,Hkv,Nq,prefix", [(8, 2, 3, 0), (4, 1, 7, 0), (4, 2, 100, 0), (4, 1, 16, 0), (8, 2, 3, 64)])
def test_padding_rows_are_empty_whatever_they_hold(Hq, Hkv, Nq, prefix):
    """Rows behind a sequence's queries, and queries that see no key, are 0 and
    -inf although they hold NaN and infinities."""
    B, d, page = 4, 128, 32
    lens_k, lens_q = [200, 90, 0, 70 + prefix], [Nq, 2, Nq, 0]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq)
    kw = with_prefix(c, prefix, lens_k) if prefix else {}
    ref = reference(q, c, lens_k, lens_q, True)
    empty = torch.tensor(np.isneginf(ref[1]))
    assert empty.any() and not empty.all()
    dirty = q.clone()
    dirty[empty] = torch.tensor([float("nan"), float("inf")] * (d // 2)).to(BF16)
    o, lse = run(dirty, c, lens_k, lens_q, **kw)
    check(o, lse, ref, q, c, way_of(Hq, Hkv, Nq, prefix))
    assert not o.cpu()[empty].any()


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 2, 1), (8, 1, 2), (6, 1, 4), (8, 2, 8), (4, 2, 64), (4, 2, 200)])
def test_scales_far_apart(Hq, Hkv, Nq):
    """Cells' scales from 2^-20 to 2^20 of one another, in keys (the queries
    smaller for it) and values."""
    B, d, page = 2, 64, 16
    lens = [777, 300 + Nq]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=3)
    g = torch.Generator().manual_seed(1)
    for i, span in ((0, 3), (1, 10)):
        e = torch.randint(-span, span + 1, c.scales[i].shape, generator=g)
        c.scales[i] = c.scales[i] * torch.exp2(e.float())
    c.update()
    o, lse = run(q, c, lens)
    check(o, lse, reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq))


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 2, 1), (8, 2, 4), (8, 2, 8), (4, 2, 64)])
@pytest.mark.parametrize("low,high,q_scale", [(-32, 28, 1.0), (0, 60, 1.0), (-32, -32, 1.0), (60, 60, 1.0), (-32, -32, 10.0)])
def test_scales_of_values_at_their_limits(Hq, Hkv, Nq, low, high, q_scale):
    """Values' scales of 2^low and 2^high, cells in turn, with scores of +-2 and of
    +-20 (in units of ln 2 times 10)."""
    B, d, page = 2, 128, 64
    lens = [1500, 200 + Nq]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=8, q_scale=q_scale)
    live = torch.isfinite(c.scales[1])
    at = torch.arange(page // 16) % 2 == 0
    c.scales[1] = torch.where(live, torch.where(at, 2.0 ** low, 2.0 ** high).float().expand_as(live), c.scales[1])
    c.update()
    o, lse = run(q, c, lens)
    check(o, lse, reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq))


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 2, 1), (8, 2, 8), (4, 2, 64), (2, 1, 300)])
def test_one_large_weight_and_many_small_ones(Hq, Hkv, Nq):
    """The first key takes about half of every row's weight, thousands of others
    the rest, each 2^-12 of it and less: none of them is lost."""
    B, d, page = 1, 128, 64
    lens = [6000]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=5)
    q[:] = 0.0
    q[..., 0] = 1.0
    raw = c.pages[0].view(torch.uint8)
    keys = torch.zeros_like(raw)
    dead = raw == 0x7F
    keys[c.table[0, 0], :, 0, 0] = torch.tensor([96.0]).to(E4M3).view(torch.uint8).item()
    keys[dead] = 0x7F
    raw.copy_(keys)
    c.scales[0][torch.isfinite(c.scales[0])] = 1.0  # scores 96 / sqrt(128) = 8.5 and 0: e^8.5 = 4900
    c.update()
    ref = reference(q, c, lens, None, True)
    o, lse = run(q, c, lens)
    check(o, lse, ref, q, c, way_of(Hq, Hkv, Nq))


def test_peaked_scores_large_values_and_outliers_in_queries():
    """Scores of +-200, values of 1e6, queries with one element a thousand
    times the others."""
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 16
    lens = [500, 77]
    for Nq in (1, 6, 20):
        q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=4, q_scale=10.0)
        c.scales[1] *= 1e6
        c.update()
        o, lse = run(q, c, lens)
        check(o, lse, reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq), Nq)
        q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=5, q_scale=0.02)
        q[..., 17] = 20.0
        o, lse = run(q, c, lens)
        check(o, lse, reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq), Nq)


@pytest.mark.parametrize("Nq", [1, 5, 40])
def test_agrees_with_the_bf16_cache_of_the_same_values(Nq):
    """With scales that are powers of two the stored values are bf16 numbers:
    forward_paged over those gives the same to the sum of both bounds."""
    B, Hq, Hkv, d, page = 3, 8, 2, 128, 32
    lens = [900, 33 + Nq, 5 + Nq]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=7)
    for i in (0, 1):
        c.scales[i] = torch.exp2(torch.floor(torch.log2(c.scales[i])))
    c.update()
    o, lse = run(q, c, lens)
    kp, vp = (torch.tensor(x).to(BF16).cuda() for x in c.values)
    assert np.array_equal(np.nan_to_num(to64(kp)), np.nan_to_num(c.values[0]))
    o2, lse2 = fa.forward_paged(q.cuda(), kp, vp, c.table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    fa.sync_status()
    # weights of 8 bits at most on either side, |v| below 4: 2 * 2 * 2^-8 * 4 / 2
    assert (o - o2).abs().max() <= 2 * 2.0 ** -8 * 4 and (lse - lse2).abs().max() <= 1e-4


@pytest.mark.parametrize("Nq", [1, 40])
def test_bad_pages_are_reported_and_read_nothing(Nq):
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    lens = [100, 90, 80]
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=2)
    ref = reference(q, c, lens, None, True)
    good = c.table.clone()
    for entry in (c.pages[0].shape[0], -1, -2 ** 31, 2 ** 31 - 1):
        c.table = good.clone()
        c.table[1, 2] = entry
        o, lse = fa.forward_paged_fp8(q.cuda(), *c.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        with pytest.raises(fa.FAError) as e:
            fa.sync_status()
        assert e.value.status == fa.FA_ERR_BAD_PAGE
        assert fa.fa_last_failure()[2:] == [1, entry]
        fa.sync_status()
        keep = [0, 2]
        check(o[keep], lse[keep], [r[keep] for r in ref], q, c, way_of(Hq, Hkv, Nq))


def test_lengths_are_clamped_and_workspace_is_bounded():
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    lens = [96, 96, 96]
    for Nq in (1, 30):
        q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=3)
        c.table = c.table[:, :6].contiguous()  # six pages: 96 keys
        ref = reference(q, c, [96, 0, 96], None, True)
        need = fa.fa_fwd_paged_workspace_bytes(B, Hq, Hkv, Nq, d) // 4
        ws = torch.full((need + 64,), 123.0, device="cuda")
        o = torch.full((B * Hq * Nq * d + 64,), 55.0, device="cuda")
        lse = torch.full((B * Hq * Nq + 64,), 55.0, device="cuda")
        out = (o[:-64].view(B, Hq, Nq, d), lse[:-64].view(B, Hq, Nq))
        fa.forward_paged_fp8(q.cuda(), *c.cuda(), torch.tensor([10 ** 6, -5, 96], dtype=torch.int32, device="cuda"),
                             workspace=ws[:need], out=out)
        fa.sync_status()
        assert torch.all(ws[need:] == 123.0) and torch.all(o[-64:] == 55.0) and torch.all(lse[-64:] == 55.0)
        check(out[0], out[1], ref, q, c, way_of(Hq, Hkv, Nq))
    full = run(q, c, [96] * 3)
    o2, l2 = fa.forward_paged_fp8(q.cuda(), *c.cuda())  # no lengths: every sequence fills its table
    fa.sync_status()
    assert torch.equal(full[0], o2) and torch.equal(full[1], l2)


@pytest.mark.parametrize("Nq,prefix", [(1, 0), (24, 0), (300, 0), (2, 128)])
def test_repeats_are_bit_equal_on_streams_and_in_graphs(Nq, prefix):
    """Calls on two streams at once with their own workspaces, and two captured
    calls replayed at once beside eager ones: the same bits."""
    lens = [3000, 317, 1024]
    q, c = make_batch(3, 8, 2, Nq, 128, 64, lens, seed=8)
    kw = with_prefix(c, prefix, lens) if prefix else {}
    first = run(q, c, lens, **kw)
    dev, lk = [q.cuda(), *c.cuda()], torch.tensor(lens, dtype=torch.int32, device="cuda")
    pt = kw["prefix_table"].cuda() if prefix else None

    def call():
        if prefix:
            return fa.forward_shared_prefix_fp8(*dev[:5], pt, prefix, dev[5], lk)
        return fa.forward_paged_fp8(*dev, lk)

    call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, graphs = [], []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(call())
    torch.cuda.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        outs.append(call())
    torch.cuda.synchronize()
    fa.sync_status()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_decoding_loop_in_a_graph():
    """Append and attention of a step captured once and replayed while the
    sequences grow over cell and page borders, against the oracle on what the
    cache holds."""
    B, Hq, Hkv, d, page, prefix = 4, 8, 2, 128, 16, 64
    start, grown = [64, 70, 90, 79], [110] * 4
    g = torch.Generator().manual_seed(1)
    _, c = make_batch(B, Hq, Hkv, 1, d, page, grown, seed=12)
    kw = with_prefix(c, prefix, grown)
    for b in range(B):  # rows behind the start are stale: the loop has to write them
        for p in range(start[b], 110):
            for x in c.pages:
                x.view(torch.uint8)[c.table[b, p // page], :, p % page] = 0x7F
            if p % 16 == 0:
                for x in c.scales:
                    x[c.table[b, p // page], :, p % page // 16] = float("nan")
    k, v, ks, vs, dt = c.cuda()
    pt = kw["prefix_table"].cuda()
    turns = fa.rope_turns(d, device="cuda")
    lk = torch.tensor(start, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, 1, Hq + 2 * Hkv, d, dtype=BF16, device="cuda")
    xq, xk, xv = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    rq = torch.zeros(B, Hq, 1, d, dtype=BF16, device="cuda")

    def step():
        lk.add_(1)
        fa.kv_append_fp8(xk, xv, k, v, ks, vs, dt, lk, turns=turns, q=xq, q_out=rq)
        return (fa.forward_paged_fp8(rq, k, v, ks, vs, dt, lk),
                fa.forward_shared_prefix_fp8(rq, k, v, ks, vs, pt, prefix, dt, lk))

    keep = [t.clone() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t, was in zip((k.view(torch.uint8), v.view(torch.uint8), ks, vs), keep):
        t.copy_(was)
    lk.copy_(torch.tensor(start, dtype=torch.int32))
    for n in range(20):
        x.copy_((torch.randn(B, 1, Hq + 2 * Hkv, d, generator=g) * (0.5 + n)).to(BF16))  # scales are raised on the way
        graph.replay()
        fa.sync_status()
        if n % 6 and n != 19:
            continue
        lens = [m + n + 1 for m in start]
        c.pages, c.scales = [t.cpu() for t in (k, v)], [t.cpu() for t in (ks, vs)]
        c.update()
        ref = reference(rq.cpu(), c, lens, None, True)
        check(*outs[0], ref, rq.cpu(), c, "steps", n)
        check(*outs[1], ref, rq.cpu(), c, "tiles", n)
        # and the last token's values are what was given, to half a step of its cell's scale
        for b in range(B):
            p = lens[b] - 1
            there = c.values[1][c.table[b, p // page], :, p % page]
            scale = to64(c.scales[1])[c.table[b, p // page], :, p % page // 16]
            want = to64(xv[b, :, 0])
            assert np.all(np.abs(there - want) <= np.maximum(np.abs(want) * 2.0 ** -4, scale[:, None] * 2.0 ** -10))


def test_prompt_in_chunks_equals_prompt_at_once():
    """A prompt appended in ragged chunks stands for the same values as one
    appended at once but for what raised scales make subnormal, and the
    attention over it is the rotated rows' to the rounding of the cache."""
    B, H, d, page, N = 1, 2, 64, 16, 300
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, N, 3 * H, d, generator=g).to(BF16).cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([H, H, H], 2))
    turns = fa.rope_turns(d, device="cuda")
    table = torch.randperm(20, generator=g).to(torch.int32)[None].cuda()

    def cache():
        return [torch.zeros(20, H, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + [
            torch.zeros(20, H, page // 16, device="cuda") for _ in range(2)]

    def values(c):
        x = torch.stack([c[i].float() * c[2 + i].repeat_interleave(16, 2)[..., None] for i in range(2)])
        return x[:, table[0].long()].transpose(1, 2).flatten(2, 3)[:, :, :N]

    one, parts = cache(), cache()
    whole = torch.tensor([N], dtype=torch.int32, device="cuda")
    rq = fa.kv_append_fp8(k, v, *one, table, whole, turns=turns, q=q)
    o1, lse1 = fa.forward_paged_fp8(rq, *one, table, whole)
    at = 0
    for n in (100, 1, 7, 128, 64):
        cut = slice(at, at + n)
        at += n
        lk = torch.tensor([at], dtype=torch.int32, device="cuda")
        rq = fa.kv_append_fp8(k[:, :, cut], v[:, :, cut], *parts, table, lk, turns=turns, q=q[:, :, cut])
        o, lse = fa.forward_paged_fp8(rq, *parts, table, lk)
        fa.sync_status()
        # the values differ by a step of a raised scale's subnormals, 2^-9 of at most 2^-5: weights hardly, |v| below 5
        assert (o - o1[:, :, cut]).abs().max() <= 2e-2 and (lse - lse1[:, :, cut]).abs().max() <= 2e-2
    assert at == N
    a, b = values(one), values(parts)
    top = torch.maximum(one[2], one[3]).max()
    assert (a - b).abs().max() <= 2.0 ** -9 * top
    exact = v[0].float()
    assert ((a[1] - exact).abs() <= torch.maximum(exact.abs() * 2.0 ** -4, top * 2.0 ** -10)).all()


def test_long_cache_offsets_past_32_bits():
    """A cache whose last pages start more than 2^32 bytes in: appended to and
    read at its end, forked and compacted."""
    Hkv, page, d = 8, 128, 128
    pages = 2 ** 32 // (Hkv * page * d) + 5
    k, v = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros(pages, Hkv, page // 16, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    small = [t[:2].clone() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    small[0], small[1] = small[0].view(E4M3), small[1].view(E4M3)
    near = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    n = 200
    xk, xv = (torch.randn(1, Hkv, n, d).to(BF16).cuda() for _ in range(2))
    lk = torch.tensor([n], dtype=torch.int32, device="cuda")
    fa.kv_append_fp8(xk, xv, k, v, ks, vs, table, lk)
    fa.kv_append_fp8(xk, xv, *small, near, lk)
    for Nq in (1, 6, 60):
        q = torch.randn(1, 4 * Hkv, Nq, d).to(BF16).cuda()
        o, lse = fa.forward_paged_fp8(q, k, v, ks, vs, table, lk)
        o2, lse2 = fa.forward_paged_fp8(q, *small, near, lk)
        fa.sync_status()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(k[pages - 2].view(torch.uint8), small[0][0].view(torch.uint8))
    # the sequence and a sample of it, then the pages in use at the front
    pool = fa.PagePool([k, v, ks, vs], page)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[0].long()] = 1
    refs[:pages - 4] += 1  # (in use elsewhere)
    two, lens, refs = fa.kv_fork(pool, table, lk, refs, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    fa.sync_status()
    assert two.tolist() == [[pages - 1, pages - 2], [pages - 1, pages - 4]]
    refs[:pages - 4] -= 1
    moved, refs, new_ids = fa.kv_compact(pool, two, lens, refs)
    fa.sync_status()
    assert sorted(set(moved.flatten().tolist())) == [0, 1, 2]
    q = torch.randn(1, 4 * Hkv, 3, d).to(BF16).cuda()
    o, _ = fa.forward_paged_fp8(q.expand(2, -1, -1, -1).contiguous(), k, v, ks, vs, moved, lens)
    o2, _ = fa.forward_paged_fp8(q, *small, near, lk)
    fa.sync_status()
    assert torch.equal(o[0], o2[0]) and torch.equal(o[1], o2[0])


def test_strided_tables_and_odd_scales_storage():
    """A block table of stride 0, one that is a slice of a wider tensor, and
    scales that start 4 bytes off a 16-byte boundary."""
    B, Hq, Hkv, d, page = 4, 4, 2, 128, 32
    q, c = make_batch(1, Hq, Hkv, 1, d, page, [500], seed=6)
    q = torch.randn(B, Hq, 1, d).to(BF16)
    lens = [500, 100, 33, 1]
    k, v, ks, vs, table = c.cuda()
    shifted = []
    for s in (ks, vs):
        x = torch.empty(s.numel() + 1, device="cuda")
        x[1:] = s.flatten()
        shifted.append(x[1:].view(s.shape))
    wide = torch.full((B, 40), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for Nq in (1, 12):
        q = torch.randn(B, Hq, Nq, d).to(BF16)
        a = fa.forward_paged_fp8(q.cuda(), k, v, ks, vs, table.expand(B, -1), lk)
        b = fa.forward_paged_fp8(q.cuda(), k, v, *shifted, wide[:, 3:3 + table.shape[1]], lk)
        fa.sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        c.table = table.expand(B, -1).cpu()
        check(a[0], a[1], reference(q, c, lens, None, True), q, c, way_of(Hq, Hkv, Nq))


@pytest.mark.parametrize("Hq,Hkv,N,d", [(20, 20, 4096, 64), (24, 8, 3500, 128)])
def test_many_units_agree_with_the_bf16_cache(Hq, Hkv, N, d):
    """More units than two for every CTA, so that most are drawn from the
    counter: a whole prompt against its own cache agrees with forward_paged over
    the same values, and two runs are equal bit for bit."""
    page = 64
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, h, N, d, generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    pages = -(-N // page)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    c = [torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)] + [
        torch.zeros(pages, Hkv, page // 16, device="cuda") for _ in range(2)]
    lk = torch.tensor([N], dtype=torch.int32, device="cuda")
    fa.kv_append_fp8(k, v, *c, table, lk)
    a = fa.forward_paged_fp8(q, *c, table, lk)
    b = fa.forward_paged_fp8(q, *c, table, lk)
    kb, vb = ((c[i].float() * c[2 + i].repeat_interleave(16, 2)[..., None]).to(BF16) for i in range(2))
    o, lse = fa.forward_paged(q, kb, vb, table, lk)
    fa.sync_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # weights of 8 and 11 bits: |v| below 6, their sum 1
    assert (a[0] - o).abs().max() <= 2 * 2.0 ** -8 * 6 and (a[1] - lse).abs().max() <= 1e-4
