"""Attention over the paged cache (fa_fwd_paged) and behind a shared prefix
(fa_fwd_shared_prefix), against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from oracle import serving
from tests.helpers import scale_for, to64
from tests.test_rope_gpu import make_cache

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=0, q_scale=1.0):
    """q and a cache whose pages hold N(0,1) rows at the sequences' positions
    and NaN everywhere else."""
    g = torch.Generator().manual_seed(seed)
    kp, vp, table = make_cache(B, Hkv, d, page, lens_k, seed=seed)
    for b, n in enumerate(lens_k):
        for i in range((n + page - 1) // page):
            rows = min(page, n - i * page)
            for pages in (kp, vp):
                pages[table[b, i], :, :rows] = torch.randn(Hkv, rows, d, generator=g).to(BF16)
    q = (torch.randn(B, Hq, Nq, d, generator=g) * q_scale).to(BF16)
    return q, kp, vp, table


def exponent_error(q, kp, scale, d):
    """Bound on the error of a scaled score: d products summed in fp32 (each
    addition half a step of the largest partial sum, at most sum |q||k|), the
    scale's and the maximum's two roundings; and the exponential's and its
    sum's 2^-21.  The largest |q| row against the largest |k| row."""
    qn = to64(q).reshape(-1, d)
    kn = np.nan_to_num(to64(kp)).reshape(-1, d)
    top = scale * np.sqrt((qn ** 2).sum(1).max() * (kn ** 2).sum(1).max())
    return (d + 8) * 2.0 ** -24 * top + 2.0 ** -21


def check(o, lse, ref, q, kp, scale, p_bits, what=""):
    """p_bits: the significand bits that the probabilities keep before the
    product with V (16 for a bf16 pair, 8 for bf16, whose correction of the
    largest one in the sum is worth as much again)."""
    o_ref, lse_ref, mass = ref
    d = q.shape[-1]
    e = exponent_error(q, kp, scale, d)
    rel = 2 * e + 2.0 ** -p_bits * (2 if p_bits == 8 else 1)
    got = o.cpu().double().numpy()
    assert np.all(np.isfinite(got)), what
    out = 2.0 ** -8 if o.dtype == BF16 else 2.0 ** -24
    bound = rel * mass + out * (np.abs(o_ref) + rel * mass) + 1e-30
    worst = (np.abs(got - o_ref) - bound).max()
    assert worst <= 0, (what, worst, np.abs(got - o_ref).max())
    lg = lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(lg), np.isneginf(lse_ref)), what
    fin = np.isfinite(lse_ref)
    assert np.all(np.abs(lg[fin] - lse_ref[fin]) <= e + 2.0 ** -21 * (1 + np.abs(lse_ref[fin]))), what


def run(q, kp, vp, table, lens_k, lens_q=None, causal=True, o_dtype=F32, prefix=0, page=16, **kw):
    dev = [t.cuda() for t in (q, kp, vp, table)]
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    lq = torch.tensor(lens_q, dtype=torch.int32, device="cuda") if lens_q is not None else None
    if prefix:
        out = fa.forward_shared_prefix(dev[0], dev[1], dev[2], kw.pop("prefix_table").cuda(), prefix, dev[3], lk, lq,
                                       causal=causal, o_dtype=o_dtype, **kw)
    else:
        out = fa.forward_paged(*dev, lk, lq, causal=causal, o_dtype=o_dtype, **kw)
    fa.sync_status()
    return out


def reference(q, kp, vp, table, lens_k, lens_q, causal):
    scale = scale_for(q.shape[-1])
    lq = lens_q if lens_q is not None else [q.shape[2]] * q.shape[0]
    return serving.paged_forward(to64(q), to64(kp), to64(vp), table.numpy(), scale, causal, lq, lens_k)


STEPS = [
    # B, Hq, Hkv, Nq, d, page, lens_k, lens_q
    (1, 1, 1, 1, 64, 16, [1], None),
    (1, 1, 1, 1, 128, 16, [63], None),
    (1, 4, 2, 1, 128, 64, [64], None),
    (2, 8, 1, 1, 128, 128, [65, 129], None),
    (3, 5, 5, 1, 64, 32, [300, 0, 1], None),                     # an empty sequence
    (2, 14, 2, 1, 128, 16, [777, 1024], None),                   # 7 heads a group
    (4, 16, 2, 1, 128, 48, [100, 2000, 47, 48], None),           # pages that are no power of two
    (2, 6, 3, 1, 64, 256, [700, 255], [1, 0]),                   # a sequence without a query
    (5, 20, 4, 3, 128, 64, [3, 64, 500, 2, 1000], [3, 3, 2, 3, 1]),   # third: more queries than keys
    (1, 32, 4, 2, 128, 64, [5000], None),                        # 16 rows a group
    (70, 2, 1, 1, 64, 16, [(i * 37) % 211 for i in range(70)], None),
    (2, 3, 1, 4, 128, 80, [333, 200], None),
    (1, 8, 8, 1, 128, 64, [9000], None),
    (600, 2, 1, 1, 64, 16, [(i * 53) % 97 for i in range(600)], None),  # more sequences than a launch takes
]


@pytest.mark.parametrize("o_dtype", [F32, BF16])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_steps_match_oracle(case, o_dtype):
    """Single tokens and a few drafted ones (at most 16 rows a key head)."""
    B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B, q_scale=2.0)
    o, lse = run(q, kp, vp, table, lens_k, lens_q, o_dtype=o_dtype)
    check(o, lse, reference(q, kp, vp, table, lens_k, lens_q, True), q, kp, scale_for(d), 16, case)


CHUNKS = [
    (1, 4, 1, 5, 128, 64, [200], None),                          # 20 rows
    (2, 2, 1, 16, 64, 16, [16, 333], None),
    (1, 8, 1, 4, 128, 32, [1000], None),                         # 32 rows
    (2, 7, 1, 19, 128, 64, [400, 19], None),                     # 133 rows: one more tile
    (3, 4, 2, 64, 64, 48, [64, 500, 0], [64, 10, 5]),
    (2, 6, 2, 100, 128, 128, [100, 1234], [100, 37]),
    (1, 2, 2, 300, 128, 64, [700], None),
    (2, 1, 1, 257, 64, 16, [300, 100], [257, 257]),              # second: 157 rows see nothing
    (1, 3, 1, 129, 128, 256, [5000], None),
    (1, 16, 2, 33, 64, 64, [2000], None),
    (1, 1, 1, 140, 128, 16, [41000], None),                      # long ranges: the ring goes round
    (2, 2, 1, 700, 128, 64, [3001, 9001], [700, 600]),           # heads of 700 rows: tiles across two heads
    (3, 3, 3, 200, 64, 32, [6001, 12007, 300], None),
    (1, 4, 1, 32, 128, 64, [9000], None),                        # 128 rows: both row tiles take them
    (2, 5, 1, 21, 64, 32, [1000, 130], [21, 3]),
    (1, 8, 2, 11, 128, 16, [129], None),
    (530, 1, 1, 40, 64, 16, [40 + (i * 31) % 60 for i in range(530)], None),  # more row pairs than a launch takes
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_chunks_match_oracle(case, causal):
    """Chunks of a prompt against what is cached of it."""
    B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    for o_dtype in (F32, BF16):
        o, lse = run(q, kp, vp, table, lens_k, lens_q, causal=causal, o_dtype=o_dtype)
        check(o, lse, reference(q, kp, vp, table, lens_k, lens_q, causal), q, kp, scale_for(d), 8, case)


PREFIXES = [
    # B, Hq, Hkv, Nq, d, page, prefix, lens_k (whole), lens_q
    (1, 1, 1, 1, 64, 16, 16, [17], None),
    (2, 8, 2, 1, 128, 64, 64, [65, 64], None),                   # second: its token is the prefix's last
    (5, 4, 1, 1, 128, 16, 208, [300, 209, 208, 100, 0], None),   # shorter than the prefix, and empty
    (40, 8, 2, 1, 64, 32, 512, [513 + 7 * i for i in range(40)], None),
    (6, 10, 2, 4, 64, 16, 1040, [1044 + 50 * i for i in range(6)], None),
    (3, 6, 2, 70, 128, 64, 640, [710, 1000, 800], [70, 13, 70]),
    (130, 2, 2, 1, 128, 64, 256, [257] * 130, None),             # more rows than one tile
    (20, 16, 1, 1, 128, 48, 960, [961 + i for i in range(20)], [1] * 19 + [0]),
    (3, 2, 1, 150, 64, 128, 128, [278, 200, 150], None),         # new tokens inside the prefix
    (520, 3, 1, 1, 64, 16, 32, [33 + i % 40 for i in range(520)], None),  # groups of rows cross row pairs
    (515, 1, 1, 35, 64, 16, 64, [99 + i % 50 for i in range(515)], None),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", PREFIXES, ids=lambda c: "x".join(str(x) for x in c[:7]))
def test_shared_prefix_matches_oracle(case, causal):
    B, Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    n = prefix // page
    longest = int(np.argmax(lens_k))
    prefix_table = table[longest, :n].clone()
    for b in range(B):  # every sequence starts with the longest one's pages
        table[b, :n] = prefix_table
    ref = reference(q, kp, vp, table, lens_k, lens_q, causal)
    blind = table.clone()
    blind[:, :n] = -1  # entries of the prefix are not read
    for o_dtype in (F32, BF16):
        o, lse = run(q, kp, vp, blind, lens_k, lens_q, causal=causal, o_dtype=o_dtype, prefix=prefix,
                     prefix_table=prefix_table)
        check(o, lse, ref, q, kp, scale_for(d), 8, case)


def test_agrees_with_the_contiguous_calls():
    """The same keys in pages and in one tensor: fa_fwd_decode and
    fa_fwd_varlen agree with fa_fwd_paged to the sum of both bounds."""
    B, H, d, page = 2, 3, 128, 64
    lens = [1000, 333]
    q, kp, vp, table = make_batch(B, H, H, 2, d, page, lens, seed=9)
    width = 1000
    k = torch.tensor(serving.gather_cache(to64(kp), table.numpy(), lens, width)).to(BF16).cuda()
    v = torch.tensor(serving.gather_cache(to64(vp), table.numpy(), lens, width)).to(BF16).cuda()
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = run(q, kp, vp, table, lens)
    for other in (fa.forward_decode, fa.forward_varlen):
        o2, lse2 = other(q.cuda(), k, v, seqlens_k=lk, causal=True)
        fa.sync_status()
        assert (o - o2).abs().max() <= 2e-3 and (lse - lse2).abs().max() <= 1e-4


def test_peaked_scores_and_large_values():
    """One key that dominates, scores of +-200, values of 1e4: no overflow and
    the dominant key's value row comes back."""
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 16
    lens = [500, 77]
    for Nq in (1, 20):
        q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=4, q_scale=12.0)
        vp = (vp.float() * 1e4).to(BF16)
        o, lse = run(q, kp, vp, table, lens)
        check(o, lse, reference(q, kp, vp, table, lens, None, True), q, kp, scale_for(d), 16 if Nq == 1 else 8, Nq)


@pytest.mark.parametrize("Nq", [1, 40])
def test_bad_pages_are_reported_and_read_nothing(Nq):
    """Entries outside the cache are reported; the other sequences' results
    stand, and the bad entries behind a sequence's end are not looked at."""
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    lens = [100, 90, 80]
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=2)
    ref = reference(q, kp, vp, table, lens, None, True)
    table[1, 2] = kp.shape[0]
    dev = [t.cuda() for t in (q, kp, vp, table)]
    o, lse = fa.forward_paged(*dev, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_BAD_PAGE
    assert fa.fa_last_failure()[2:] == [1, kp.shape[0]]
    fa.sync_status()
    keep = [0, 2]
    check(o[keep], lse[keep], [r[keep] for r in ref], q, kp, scale_for(d), 8, Nq)


def test_lengths_are_clamped_and_workspace_is_bounded():
    """Lengths past the table's reach, negative ones, and a workspace of the
    stated size with a guard band behind it."""
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    lens = [96, 96, 96]
    for Nq in (1, 30):
        q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=3)
        table = table[:, :6].contiguous()  # six pages: 96 keys
        ref = reference(q, kp, vp, table, [96, 0, 96], None, True)
        need = fa.fa_fwd_paged_workspace_bytes(B, Hq, Hkv, Nq, d) // 4
        ws = torch.full((need + 64,), 123.0, device="cuda")
        o = torch.full((B * Hq * Nq * d + 64,), 55.0, device="cuda")
        lse = torch.full((B * Hq * Nq + 64,), 55.0, device="cuda")
        out = (o[:-64].view(B, Hq, Nq, d), lse[:-64].view(B, Hq, Nq))
        fa.forward_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                         torch.tensor([10 ** 6, -5, 96], dtype=torch.int32, device="cuda"), workspace=ws[:need],
                         out=out)
        fa.sync_status()
        assert torch.all(ws[need:] == 123.0) and torch.all(o[-64:] == 55.0) and torch.all(lse[-64:] == 55.0)
        check(out[0], out[1], ref, q, kp, scale_for(d), 8, Nq)
    # no lengths: every sequence fills its table
    full = run(q, kp, vp, table, [96] * 3)
    o2, l2 = fa.forward_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda())
    fa.sync_status()
    assert torch.equal(full[0], o2) and torch.equal(full[1], l2)


def test_shared_table_row_and_strided_tables():
    """A block table of stride 0 (every sequence the same keys) and one that
    is a slice of a wider tensor."""
    B, Hq, Hkv, d, page = 4, 4, 2, 128, 32
    q, kp, vp, table = make_batch(1, Hq, Hkv, 1, d, page, [500], seed=6)
    q = torch.randn(B, Hq, 1, d).to(BF16)
    lens = [500, 100, 33, 1]
    wide = torch.full((B, 40), 10 ** 6, dtype=torch.int32)
    wide[:, 3:3 + table.shape[1]] = table
    dev = [t.cuda() for t in (q, kp, vp)]
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = fa.forward_paged(*dev, table.cuda().expand(B, -1), lk)
    b = fa.forward_paged(*dev, wide.cuda()[:, 3:3 + table.shape[1]], lk)
    fa.sync_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref = reference(q, kp, vp, table.expand(B, -1), lens, None, True)
    check(a[0], a[1], ref, q, kp, scale_for(d), 16)


@pytest.mark.parametrize("Nq", [1, 24])
def test_repeats_are_bit_equal_and_streams_are_honoured(Nq):
    """Two calls at once on two streams with their own workspaces, and the
    same call again: the same bits."""
    lens = [3000, 17, 1024]
    q, kp, vp, table = make_batch(3, 8, 2, Nq, 128, 64, lens, seed=8)
    first = run(q, kp, vp, table, lens)
    dev = [t.cuda() for t in (q, kp, vp, table)]
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(fa.forward_paged(*dev, lk))
    torch.cuda.synchronize()
    fa.sync_status()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_decoding_loop_in_a_graph():
    """Append and attention of a step captured once and replayed while the
    sequences grow over page boundaries, behind a shared prefix and without
    one; two graphs share one workspace, one after the other."""
    B, Hq, Hkv, d, page, prefix = 4, 8, 2, 128, 16, 64
    start, grown = [64, 70, 90, 79], [110] * 4
    g = torch.Generator().manual_seed(1)
    q, kp, vp, table = make_batch(B, Hq, Hkv, 1, d, page, grown, seed=12)
    for b in range(B):
        table[b, :prefix // page] = table[0, :prefix // page]
    k0, v0 = to64(kp), to64(vp)
    for b in range(B):  # rows behind the start are stale: the loop has to write them
        for p in range(start[b], 110):
            kp[table[b, p // page], :, p % page] = float("nan")
            vp[table[b, p // page], :, p % page] = float("nan")
    k0, v0 = to64(kp), to64(vp)
    dk, dv, dt = kp.cuda(), vp.cuda(), table.cuda()
    pt = dt[0, :prefix // page].contiguous()
    turns = fa.rope_turns(d, device="cuda")
    lk = torch.tensor(start, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, 1, Hq + 2 * Hkv, d, dtype=BF16, device="cuda")
    xq, xk, xv = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    rq = torch.zeros(B, Hq, 1, d, dtype=BF16, device="cuda")
    need = max(fa.fa_fwd_paged_workspace_bytes(B, Hq, Hkv, 1, d),
               fa.fa_fwd_shared_prefix_workspace_bytes(B, Hq, Hkv, 1, d)) // 4
    ws = torch.empty(need, device="cuda")
    outs = [(torch.empty(B, Hq, 1, d, device="cuda"), torch.empty(B, Hq, 1, device="cuda")) for _ in range(2)]

    def append():
        fa.kv_append(xk, xv, dk, dv, dt, lk, turns=turns, q=xq, q_out=rq)

    def attend(i):
        if i == 0:
            fa.forward_paged(rq, dk, dv, dt, lk, workspace=ws, out=outs[0])
        else:
            fa.forward_shared_prefix(rq, dk, dv, pt, prefix, dt, lk, workspace=ws, out=outs[1])

    lk.add_(1), append(), attend(0), attend(1)  # warm-up: writes step 0's rows with zeros, rewritten below
    torch.cuda.synchronize()
    lk.sub_(1)
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            if i == 0:
                lk.add_(1)
                append()
            attend(i)
        graphs.append(gr)
    lk.copy_(torch.tensor(start, dtype=torch.int32))
    for step in range(20):
        new = torch.randn(B, 1, Hq + 2 * Hkv, d, generator=g).to(BF16)
        x.copy_(new)
        for gr in graphs:
            gr.replay()
        fa.sync_status()
        lens = [n + step + 1 for n in start]
        pos = torch.tensor([[n - 1] for n in lens], dtype=torch.int32, device="cuda")
        tk = fa.rope_forward(xk, turns, pos).cpu()
        k0 = serving.place_tokens(k0, to64(tk), table.numpy(), [1] * B, lens)
        v0 = serving.place_tokens(v0, to64(new[:, :, Hq + Hkv:].transpose(1, 2)), table.numpy(), [1] * B, lens)
        if step % 6 == 0 or step == 19:
            scale = scale_for(d)
            ref = serving.paged_forward(to64(rq.cpu()), k0, v0, table.numpy(), scale, True, [1] * B, lens)
            check(*outs[0], ref, rq.cpu(), torch.tensor(k0), scale, 16, step)
            check(*outs[1], ref, rq.cpu(), torch.tensor(k0), scale, 8, step)


def test_prompt_in_chunks_equals_prompt_at_once():
    """A prompt appended and attended in ragged chunks gives the rows of the
    square causal call on the same rotated tensors."""
    B, H, d, page, N = 1, 2, 64, 16, 300
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, N, 3 * H, d, generator=g).to(BF16).cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([H, H, H], 2))
    turns = fa.rope_turns(d, device="cuda")
    o_ref, lse_ref = fa.forward(fa.rope_forward(q, turns), fa.rope_forward(k, turns), v.contiguous(), causal=True)
    kp, vp, table = make_cache(B, H, d, page, [N])
    kp, vp, table = kp.cuda(), vp.cuda(), table.cuda()
    at = 0
    for n in (100, 1, 7, 128, 64):
        cut = slice(at, at + n)
        at += n
        lk = torch.tensor([at], dtype=torch.int32, device="cuda")
        rq = fa.kv_append(k[:, :, cut], v[:, :, cut], kp, vp, table, lk, turns=turns, q=q[:, :, cut])
        o, lse = fa.forward_paged(rq, kp, vp, table, lk)
        fa.sync_status()
        # both sides within the framework's 1e-2 of the exact rows in general; here |v| < 5 and both round P to
        # 8 bits at most: 2 * 2 * 2^-8 * 5 / 2 on either side's own reference scale
        assert (o - o_ref[:, :, cut]).abs().max() <= 2e-2
        assert (lse - lse_ref[:, :, cut]).abs().max() <= 1e-4
    assert at == N


def test_long_cache_offsets_past_32_bits():
    """A cache whose last pages start more than 2^32 bytes (and 2^31 elements)
    in: appended to and read at its end."""
    Hkv, page, d = 8, 128, 128
    pages = 2 ** 31 // (Hkv * page * d) + 3
    kp = torch.zeros(pages, Hkv, page, d, dtype=BF16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    n = 200
    k, v = (torch.randn(1, Hkv, n, d).to(BF16).cuda() for _ in range(2))
    lk = torch.tensor([n], dtype=torch.int32, device="cuda")
    fa.kv_append(k, v, kp, vp, table, lk)
    for Nq in (1, 6):
        q = torch.randn(1, 4 * Hkv, Nq, d).to(BF16).cuda()
        o, lse = fa.forward_paged(q, kp, vp, table, lk)
        o2, lse2 = fa.forward_varlen(q, k.repeat_interleave(4, 1), v.repeat_interleave(4, 1), causal=True)
        fa.sync_status()
        assert (o - o2).abs().max() <= 2e-2 and (lse - lse2).abs().max() <= 1e-4
    assert torch.equal(kp[pages - 1, :, :page], k[0, :, :page])
    assert torch.equal(kp[pages - 2, :, :n - page], k[0, :, page:])


@pytest.mark.parametrize("Hq,Hkv,N,d", [(20, 20, 4096, 64), (24, 8, 3500, 128)])
def test_many_units_agree_with_the_square_call(Hq, Hkv, N, d):
    """More units than two for every CTA, so that most are drawn from the
    counter: a whole prompt against its own cache agrees with fa_fwd on the
    same tensors, and two runs are equal bit for bit."""
    page = 64
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, h, N, d, generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    kp, vp, table = (t.cuda() for t in make_cache(1, Hkv, d, page, [N]))
    lk = torch.tensor([N], dtype=torch.int32, device="cuda")
    fa.kv_append(k, v, kp, vp, table, lk)
    a = fa.forward_paged(q, kp, vp, table, lk)
    b = fa.forward_paged(q, kp, vp, table, lk)
    G = Hq // Hkv
    o, lse = fa.forward(q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), causal=True)
    fa.sync_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # both round P to bf16 (8 bits) against their own running maximum: |v| below 6, sum of P 1
    assert (a[0] - o).abs().max() <= 2 * 2.0 ** -8 * 6 and (a[1] - lse).abs().max() <= 1e-4


def test_many_units_behind_a_prefix():
    """Drawn units of both parts: the prefix's row pairs and the sequences'."""
    B, Hq, Hkv, Nq, d, page, prefix = 300, 4, 2, 128, 64, 16, 64
    lens = [prefix + Nq + i % 50 for i in range(B)]
    q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=3)
    n = prefix // page
    for b in range(1, B):
        table[b, :n] = table[0, :n]
    o, lse = run(q, kp, vp, table, lens, prefix=prefix, prefix_table=table[0, :n].clone())
    o2, lse2 = run(q, kp, vp, table, lens, prefix=prefix, prefix_table=table[0, :n].clone())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    some = [0, 1, 77, 150, 151, 299]
    ref = reference(q[some], kp, vp, table[some], [lens[b] for b in some], None, True)
    check(o[some], lse[some], ref, q, kp, scale_for(d), 8)


@pytest.mark.parametrize("Nq", [1, 40])
def test_graphs_with_their_own_workspaces_replay_at_once(Nq):
    """Two captured calls without a given workspace, replayed on two streams
    at once beside eager calls."""
    lens = [2500, 100, 900, 64]
    q, kp, vp, table = make_batch(4, 8, 2, Nq, 128, 64, lens, seed=5)
    dev = [t.cuda() for t in (q, kp, vp, table)]
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = fa.forward_paged(*dev, lk)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fa.forward_paged(*dev, lk))
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = fa.forward_paged(*dev, lk)
    torch.cuda.synchronize()
    fa.sync_status()
    for o, lse in outs + [eager]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_host_threads():
    """Calls from two threads on their own streams."""
    import threading
    lens = [1500, 33]
    q, kp, vp, table = make_batch(2, 8, 2, 1, 128, 64, lens, seed=6)
    dev = [t.cuda() for t in (q, kp, vp, table)]
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = fa.forward_paged(*dev, lk)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                o, lse = fa.forward_paged(*dev, lk)
                s.synchronize()
                if not (torch.equal(o, want[0]) and torch.equal(lse, want[1])):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    fa.sync_status()
    assert not bad


def test_captured_call_with_the_librarys_workspace():
    """The C call without a workspace inside a capture: an allocation of the
    graph's, replayed on new contents."""
    lens = [1500, 200]
    q, kp, vp, table = make_batch(2, 8, 2, 1, 128, 64, lens, seed=7)
    dev = [t.cuda() for t in (q, kp, vp, table)]
    lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = torch.zeros(2, 8, 1, 128, device="cuda")
    lse = torch.zeros(2, 8, 1, device="cuda")

    def call():
        assert fa.fa_fwd_paged(dev[0].data_ptr(), dev[1].data_ptr(), dev[2].data_ptr(), kp.shape[0], 64,
                               dev[3].data_ptr(), dev[3].stride(0), dev[3].shape[1], o.data_ptr(), 0, lse.data_ptr(), 0,
                               lk.data_ptr(), 0, 2, 8, 2, 1, 128, 128 ** -0.5, 1,
                               torch.cuda.current_stream().cuda_stream) == 0

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    dev[0].copy_(torch.randn(2, 8, 1, 128).to(BF16))
    lk.sub_(3)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want = fa.forward_paged(*dev, lk)
    fa.sync_status()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Hq,Hkv,d,lens_q,lens_k", [
    (16, 16, 128, [2560], [2560]),                       # one or two whole units a CTA
    (10, 10, 64, [2048, 700], [2048, 3000]),             # the same, one sequence shorter
    (10, 5, 128, [2100, 1], [2100, 2100]),
    (8, 8, 128, [3000], [3000]),                         # fewer units than CTAs, all cut
    (16, 8, 64, [1800, 900, 0], [1800, 2000, 50]),       # all drawn, one sequence without a query
    (40, 40, 64, [1000, 1000], [9000, 8000]),            # units of one length: some cut, the others drawn
    (32, 32, 64, [1300, 1300], [1300, 600]),             # the second: rows that see nothing
    (16, 8, 128, [24 - i % 3 for i in range(48)], [30 + 7 * i for i in range(48)]),  # 48 rows: two row tiles on them
    (64, 8, 128, [16] * 3, [5000, 2100, 17]),            # 128 rows, few units: cut
])
def test_prompts_agree_with_the_padded_call(Hq, Hkv, d, lens_q, lens_k):
    """Prompts whose units are cut, dealt out whole or drawn, against
    fa_fwd_varlen on the same tensors; two runs equal bit for bit."""
    B, Nq, Nk, page = len(lens_q), max(lens_q), max(lens_k), 64
    g = torch.Generator().manual_seed(len(lens_q) + d + Hq)
    q = torch.randn(B, Hq, Nq, d, generator=g).to(BF16).cuda()
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g).to(BF16).cuda() for _ in range(2))
    kp, vp, table = (t.cuda() for t in make_cache(B, Hkv, d, page, [max(n, 1) for n in lens_k]))
    lk, lq = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in (lens_k, lens_q))
    fa.kv_append(k, v, kp, vp, table, lk, lk)
    G = Hq // Hkv
    o, lse = fa.forward_varlen(q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), lq, lk, causal=True)
    for o_dtype in (F32, BF16):
        a = fa.forward_paged(q, kp, vp, table, lk, lq, o_dtype=o_dtype)
        b = fa.forward_paged(q, kp, vp, table, lk, lq, o_dtype=o_dtype)
        fa.sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # both round P to bf16 (8 bits) against their own running maximum: |v| below 6, sum of P 1; O once more
        assert (a[0].float() - o).abs().max() <= 2 * 2.0 ** -8 * 6 + (2.0 ** -8 * 6 if o_dtype == BF16 else 0)
        seen = torch.isfinite(lse)
        assert torch.equal(seen, torch.isfinite(a[1])) and (a[1] - lse)[seen].abs().max() <= 1e-4
        assert not a[0][~seen].any()
