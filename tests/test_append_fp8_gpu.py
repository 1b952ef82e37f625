"""The append into the paged cache in E4M3 (fa_kv_append_fp8), against the
definition in 64 bits."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from oracle import serving
from oracle.rounding import round_e4m3
from tests.helpers import to64
from tests.test_rope_gpu import make_cache

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
NAN = 0x7F


def fitting(largest):
    """The smallest power of two, at least 2^-32, that brings it to at most 448."""
    scale = 2.0 ** -32
    while largest / scale > 448:
        scale *= 2
    return scale


def expected(codes, scales, x, raw, growth, table, lens_q, lens_k):
    """codes [P, H, page, d], scales [P, H, page / 16] with the tokens x [B, H, N,
    d] (raw as they were given: their magnitudes times growth set the scale)."""
    codes, scales = codes.copy(), scales.copy()
    page = codes.shape[2]
    for b in range(x.shape[0]):
        first = lens_k[b] - lens_q[b]
        for cell in range(max(first, 0) // 16, (lens_k[b] + 15) // 16 if lens_q[b] else 0):
            p, at = table[b][cell * 16 // page], cell * 16 % page
            new = [i for i in range(16) if first <= cell * 16 + i < lens_k[b]]
            for h in range(x.shape[1]):
                t = [cell * 16 + i - first for i in new]
                big = np.abs(raw[b, h, t])
                scale = fitting(big[np.isfinite(big)].max(initial=0) * growth)
                if first > cell * 16:
                    old = scales[p, h, at // 16]
                    scale = max(scale, old)
                    n = first - cell * 16
                    codes[p, h, at:at + n] = round_e4m3(codes[p, h, at:at + n] * old / scale)
                rows = x[b, h, t]
                codes[p, h, at + new[0]:at + new[0] + len(new)] = np.where(np.isfinite(rows),
                                                                           round_e4m3(rows / scale), np.nan)
                scales[p, h, at // 16] = scale
    return codes, scales


CASES = [
    # B, Hq, Hkv, N, d, page, lens_k, lens_q, rot, layout, amplitude
    (1, 1, 1, 1, 64, 16, [1], None, 64, "half", 1.0),
    (3, 4, 2, 1, 128, 64, [17, 64, 33], None, 128, "half", 1.0),          # into a cell, its last row, a new one
    (2, 8, 4, 2, 128, 32, [32, 17], None, 64, "interleaved", 1.3),        # across two cells
    (4, 6, 3, 5, 64, 48, [3, 50, 5, 40], [5, 3, 0, 5], 16, "half", 0.7),   # more new tokens than keys; none
    (2, 2, 2, 40, 128, 16, [40, 100], [40, 33], 128, "interleaved", 1.0),
    (2, 5, 5, 33, 64, 128, [300, 35], None, 0, "half", 1.0),              # no rotation
    (1, 0, 7, 130, 128, 64, [1000], None, 32, "half", 1.0),               # no queries
    (70, 2, 1, 1, 64, 16, [1 + (i * 37) % 50 for i in range(70)], None, 64, "half", 1.0),
    (1, 64, 8, 300, 128, 256, [301], None, 128, "half", 1.0),
    (2, 3, 3, 50, 128, 32, [50, 77], None, 32, "half", 0.125),           # a part that is larger than the rotated one
    (1, 2, 2, 50, 64, 32, [60], None, 64, "interleaved", 0.0),            # keys of 0
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_append_matches_the_definition(case):
    """Scales equal; numbers equal to what the exact values round to, but for
    values next to the middle of two (fp32 rotation) which may go to the other;
    everything else as it was."""
    B, Hq, Hkv, N, d, page, lens_k, lens_q, rot, layout, amplitude = case
    g = torch.Generator().manual_seed(B + N + d)
    kp, _, table = make_cache(B, Hkv, d, page, lens_k, seed=N)
    n = kp.shape[0]
    heads = torch.exp2(torch.randn(Hkv, generator=g) * 3)
    k, v = ((torch.randn(B, N, Hkv, d, generator=g) * heads[:, None]).to(BF16) for _ in range(2))
    q = torch.randn(B, N, max(Hq, 1), d, generator=g).to(BF16)
    pages = [torch.randint(0, 256, (n, Hkv, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    for p in pages:
        p[(p & 0x7F) == 0x7F] = 0x35                       # numbers
    scales = [torch.exp2(torch.randint(-9, -3, (n, Hkv, page // 16), generator=g).float()) for _ in range(2)]
    dev = [t.cuda() for t in (*pages, *scales)]
    turns = fa.rope_turns(rot, device="cuda") if rot else None
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    lq = torch.tensor(lens_q, dtype=torch.int32, device="cuda") if lens_q else None
    view = [t.cuda().transpose(1, 2) for t in (k, v, q)]
    q_out = torch.full((B, Hq, N, d), 7.0, dtype=BF16, device="cuda") if Hq else None
    got = fa.kv_append_fp8(view[0], view[1], dev[0].view(E4M3), dev[1].view(E4M3), dev[2], dev[3], table.cuda(), lk, lq,
                           turns=turns, layout=layout, amplitude=amplitude, q=view[2] if Hq else None, q_out=q_out)
    fa.sync_status()
    assert (got is None) == (Hq == 0)
    lens_q = lens_q or [N] * B
    place = np.array([[lens_k[b] - lens_q[b] + t for t in range(N)] for b in range(B)])
    freqs = serving.rope_frequencies(rot) if rot else np.zeros(0)
    x = [to64(t).transpose(0, 2, 1, 3) for t in (k, v, q)]
    turned = [serving.rope(t, place, freqs, layout, amplitude) if rot else t for t in (x[0], x[2])]
    growth = max(np.sqrt(2) * amplitude, 1.0 if rot < d else 0.0) if rot else 1.0
    for i, (new, raw, grow) in enumerate([(turned[0], x[0], growth), (x[1], x[1], 1.0)]):
        before = to64(pages[i].view(E4M3).float())
        codes, sc = expected(before, to64(scales[i]), new, raw, grow, table.numpy(), lens_q, lens_k)
        assert np.array_equal(to64(dev[2 + i]), sc)
        there = to64(dev[i].view(E4M3).float())
        off = there != codes
        if not (rot and i == 0):
            assert not off.any(), off.sum()
        else:
            # a rotated value is off by a few fp32 roundings and the angle's 2^-24
            # turns: less than 2^-19 of the cell's largest; where that crosses the
            # middle of two numbers they are neighbours
            step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(codes), 2.0 ** -6)))) / 8, 2.0 ** -9)
            assert np.all(np.abs(there - codes) <= step * 1.0)
            assert off.mean() <= 1e-4
        # what no token came to is as it was, bit for bit
        untouched = np.ones(before.shape[:3], dtype=bool)
        for b in range(B):
            first = lens_k[b] - lens_q[b]
            for p in range(max(first, 0) // 16 * 16 if lens_q[b] else lens_k[b], lens_k[b]):
                untouched[table[b, p // page], :, p % page] = False
        same = (dev[i].cpu() == pages[i]).numpy()
        assert same[untouched].all()
    if Hq:
        valid = np.arange(N)[None] < np.array(lens_q)[:, None]
        o = to64(q_out)
        want = turned[1]
        mask = np.broadcast_to(valid[:, None, :, None], o.shape)
        assert np.all(o[~mask] == 7.0)
        # half a bf16 step, and the fp32 rotation's error
        assert np.all(np.abs(o - want)[mask] <= 2.0 ** -9 * np.abs(want[mask]) * 2 + 2.0 ** -18 * np.abs(want).max())


def test_infinities_and_nans_are_nan_and_do_not_scale():
    B, H, N, d, page = 1, 2, 20, 64, 16
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(B, H, N, d, generator=g).to(BF16) for _ in range(2))
    clean = [t.clone() for t in (k, v)]
    v[0, 0, 3, 5], v[0, 1, 17, 9], k[0, 0, 2, 1], k[0, 1, 19, 60] = float("inf"), float("nan"), -float("inf"), float("nan")
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    lk = torch.tensor([N], dtype=torch.int32, device="cuda")
    outs = []
    for a, b in ((k, v), clean):
        pages = [torch.zeros(3, H, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(3, H, 1, device="cuda") for _ in range(2)]
        fa.kv_append_fp8(a.cuda(), b.cuda(), pages[0].view(E4M3), pages[1].view(E4M3), *scales, table, lk)
        fa.sync_status()
        outs.append((pages, scales))
    for i, x in enumerate((k, v)):
        bad = ~torch.isfinite(x)[0]
        there = outs[0][0][i].view(E4M3).float().cpu()
        rows = torch.stack([there[[2, 0][t // page], :, t % page] for t in range(N)], 1)
        assert torch.equal(torch.isnan(rows), bad)
        want = torch.stack([outs[1][0][i].view(E4M3).float().cpu()[[2, 0][t // page], :, t % page] for t in range(N)], 1)
        assert torch.equal(rows[~bad], want[~bad])
        assert torch.equal(outs[0][1][i], outs[1][1][i])  # (the bad places hold no cell's largest value)


def test_tokens_without_a_place():
    """Pages outside the cache and positions behind the table are reported and
    store nothing; the queries are rotated all the same."""
    B, H, N, d, page = 2, 2, 24, 64, 16
    g = torch.Generator().manual_seed(5)
    k, v, q = (torch.randn(B, H, N, d, generator=g).to(BF16).cuda() for _ in range(3))
    turns = fa.rope_turns(d, device="cuda")
    for table, lens, detail in (([[0, 9], [1, 2]], [24, 24], [0, 9]), ([[0, 1], [2, 3]], [24, 40], [1, None])):
        pages = [torch.zeros(4, H, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(4, H, 1, device="cuda") for _ in range(2)]
        t = torch.tensor(table, dtype=torch.int32, device="cuda")
        lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = fa.kv_append_fp8(k, v, pages[0].view(E4M3), pages[1].view(E4M3), *scales, t, lk, turns=turns, q=q)
        with pytest.raises(fa.FAError) as e:
            fa.sync_status()
        assert e.value.status == fa.FA_ERR_BAD_PAGE
        where = fa.fa_last_failure()
        assert where[2] == detail[0] and (detail[1] is None or where[3] == detail[1])
        if detail[1] is None:
            assert 32 <= where[3] < 40 and where[1] == 81
        for b in range(B):
            pos = torch.arange(lens[b] - N, lens[b], dtype=torch.int32, device="cuda")
            assert torch.equal(got[b:b + 1], fa.rope_forward(q[b:b + 1], turns, pos))
        fa.sync_status()


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("amplitude", [-1.5, 2.0 ** 40])
def test_given_positions_and_other_amplitudes(shared, amplitude):
    """Angles from positions of their own (for all sequences, or each its own in
    a wider tensor), far apart and repeated; an amplitude below 0 and a large one."""
    B, H, N, d, page = 2, 2, 21, 64, 16
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, H, N, d, generator=g).to(BF16)
    places = torch.tensor([0, 10 ** 6, 5, 5, 131071, -3, 2 ** 31 - 1] * 9, dtype=torch.int32)
    places = places[:N] if shared else torch.stack([places[:N + 5], places[1:N + 6]])[:, 2:2 + N]
    wide = torch.full((B, N + 9), -7, dtype=torch.int32, device="cuda")
    dev = places.cuda() if shared else wide[:, 4:4 + N].copy_(places)
    pages = [torch.zeros(5, H, page, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.zeros(5, H, 1, device="cuda") for _ in range(2)]
    table = torch.tensor([[3, 1], [0, 4]], dtype=torch.int32)
    lk = torch.tensor([N, N], dtype=torch.int32, device="cuda")
    turns = fa.rope_turns(d, device="cuda")
    fa.kv_append_fp8(x.cuda(), x.cuda(), *pages, *scales, table.cuda(), lk, turns=turns, positions=dev,
                     amplitude=amplitude)
    fa.sync_status()
    at = np.broadcast_to(places.numpy(), (B, N))
    want = serving.rope(to64(x), at, serving.rope_frequencies(d), "half", amplitude)
    codes, sc = expected(np.zeros((5, H, page, d)), np.zeros((5, H, 1)), want, to64(x), np.sqrt(2) * abs(amplitude),
                         table.numpy(), [N] * B, [N] * B)
    assert np.array_equal(to64(scales[0]), sc)
    there = to64(pages[0].float())
    # the table's frequencies are doubles: p * 2^-53 turns, 2^-22 at 2^31, where few values' halves are crossed
    step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(codes), 2.0 ** -6)))) / 8, 2.0 ** -9)
    assert np.all(np.abs(there - codes) <= step)
    assert (there != codes).mean() <= 1e-3
