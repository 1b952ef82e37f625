"""Rotary positions (fa_rope) and the append to the paged cache that applies
them (fa_kv_append), against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
import oracle
from oracle import serving
from tests.helpers import scale_for, to64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# Error of a rotated value before its last rounding, relative to
# amplitude * (|a| + |b|), in units of 2^-24 (half a step of fp32): the angle
# in half turns is an integer rounded to fp32 (1/2 step of at most 1, times pi)
# and cut at 2^-32 turns (below 0.1 unit); sincospif 2 steps (4 units); the
# product with the amplitude 1, the product with the value 1, the sum 1:
# 3.2 + 0.1 + 4 + 3 < 11, doubled because a step is up to twice its half.
ROPE_UNITS = 22 * 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def rope_bound(x, ref, rot_dim, layout, amplitude, out_dtype):
    """Element-wise bound on |y - ref|."""
    part = np.zeros_like(ref)
    a = np.abs(x[..., :rot_dim])
    if layout == "half":
        s = a[..., :rot_dim // 2] + a[..., rot_dim // 2:]
        part[..., :rot_dim] = np.concatenate([s, s], -1)
    else:
        part[..., :rot_dim] = np.repeat(a[..., 0::2] + a[..., 1::2], 2, -1)
    e = ROPE_UNITS * abs(amplitude) * part
    return e + half_step(out_dtype) * (np.abs(ref) + e) + 1e-30


SCALINGS = {
    "none": dict(),
    "linear": dict(scaling="linear", factor=4.0),
    "ntk": dict(scaling="ntk", factor=8.0),
    "parts": dict(scaling="parts", factor=8.0, original_len=8192.0, low=1.0, high=32.0),
    "wide": dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
}


@pytest.mark.parametrize("B,H,N,d,rot,layout,scaling,far,x_dtype,y_dtype,inverse", [
    (1, 1, 1, 64, 64, "half", "none", 0, BF16, BF16, False),
    (1, 1, 1, 128, 16, "interleaved", "none", 0, F32, F32, False),
    (2, 3, 17, 128, 128, "half", "linear", 0, BF16, BF16, False),
    (2, 5, 33, 128, 128, "interleaved", "parts", 0, BF16, F32, False),
    (3, 4, 100, 64, 32, "half", "ntk", 1000000, F32, F32, False),
    (1, 7, 257, 128, 48, "interleaved", "wide", 2147483000, F32, F32, False),
    (2, 9, 31, 64, 64, "interleaved", "none", -500, F32, BF16, True),
    (1, 40, 65, 128, 96, "half", "parts", 131072, F32, F32, True),
    (5, 2, 1, 128, 128, "half", "none", 262143, BF16, F32, False),
])
def test_rope_matches_oracle(B, H, N, d, rot, layout, scaling, far, x_dtype, y_dtype, inverse):
    g = torch.Generator().manual_seed(N * 7 + d + rot)
    x = torch.randn(B, H, N, d, generator=g).to(x_dtype)
    pos = (torch.arange(N)[None] + far + torch.arange(B)[:, None] * 3).clamp(max=2 ** 31 - 1).to(torch.int32)
    turns = fa.rope_turns(rot, device="cuda", **SCALINGS[scaling])
    call = fa.rope_backward if inverse else fa.rope_forward
    y = call(x.cuda(), turns, pos.cuda(), layout=layout, amplitude=1.25, out_dtype=y_dtype)
    fa.sync_status()
    freqs = serving.rope_frequencies(rot, **SCALINGS[scaling])
    xx = to64(x)
    ref = serving.rope(xx, pos.numpy(), freqs, layout, 1.25, inverse)
    # an angle of p * f radians in 64 bits is itself off by p * 2^-53 radians, on either side
    err = np.abs(y.cpu().double().numpy() - ref)
    slack = 4 * 2.0 ** -52 * np.abs(pos.numpy().astype(np.float64))[:, None, :, None] * np.abs(xx).max()
    assert np.all(err <= rope_bound(xx, ref, rot, layout, 1.25, y_dtype) + slack)
    assert y.dtype == y_dtype and torch.equal(y[..., rot:].cpu().float(), x[..., rot:].to(y_dtype).float())


def test_rope_default_and_shared_positions():
    x = torch.randn(3, 2, 50, 64).to(BF16).cuda()
    turns = fa.rope_turns(64, device="cuda")
    a = fa.rope_forward(x, turns)
    row = torch.arange(50, dtype=torch.int32, device="cuda")
    assert torch.equal(a, fa.rope_forward(x, turns, row))
    assert torch.equal(a, fa.rope_forward(x, turns, row.expand(3, 50)))
    assert torch.equal(a[:, :, 0], x[:, :, 0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_and_in_place(dtype, layout):
    """The q part of a fused projection read where it lies, outputs in another
    order, in place: the same bits as the contiguous call; nothing beside the
    output is written."""
    B, H, N, d = 2, 6, 37, 128
    fused = torch.randn(B, N, H + 4, d).to(dtype).cuda()
    x = fused[:, :, 1:1 + H].transpose(1, 2)
    turns = fa.rope_turns(64, device="cuda")
    ref = fa.rope_forward(x.contiguous(), turns, layout=layout)
    assert torch.equal(fa.rope_forward(x, turns, layout=layout), ref)
    wide = torch.full((B, N, H + 2, d + 16), 7.0, dtype=dtype, device="cuda")
    out = wide[:, :, 1:1 + H, 8:8 + d].transpose(1, 2)
    assert fa.rope_forward(x, turns, layout=layout, out=out) is out
    assert torch.equal(out, ref)
    out.fill_(7.0)
    assert torch.all(wide == 7.0)
    before = fused.clone()
    fa.rope_forward(x, turns, layout=layout, out=x)
    assert torch.equal(x, ref)
    before[:, :, 1:1 + H] = ref.transpose(1, 2)
    assert torch.equal(fused, before)
    # one row for the whole batch and all heads
    row = torch.randn(1, 1, N, d).to(dtype).cuda()
    assert torch.equal(fa.rope_forward(row.expand(B, H, N, d), turns, layout=layout),
                       fa.rope_forward(row, turns, layout=layout).expand(B, H, N, d))


def test_rope_backward_is_the_gradient():
    """rope_backward against the transpose of the map that the oracle's
    forward is (its columns, one unit vector at a time) and against central
    differences of the forward call in fp32."""
    d, rot, N = 64, 32, 5
    pos = torch.tensor([0, 3, 1000, 77777, 1000000], dtype=torch.int32)
    turns = fa.rope_turns(rot, device="cuda", **SCALINGS["parts"])
    freqs = serving.rope_frequencies(rot, **SCALINGS["parts"])
    dy = torch.randn(1, 1, N, d)
    for layout in ("half", "interleaved"):
        got = fa.rope_backward(dy.cuda(), turns, pos.cuda(), layout=layout, amplitude=1.5).cpu().double().numpy()
        eye = np.broadcast_to(np.eye(d)[:, None, None, :], (d, 1, N, d))
        cols = serving.rope(np.ascontiguousarray(eye), np.broadcast_to(pos.numpy(), (d, N)), freqs, layout, 1.5)
        ref = np.einsum("ihnj,hnj->hni", cols, dy[0].double().numpy())[None]
        assert np.abs(got - ref).max() <= 2 * ROPE_UNITS * 1.5 * 2 * float(dy.abs().max())
        x = torch.randn(1, 1, N, d)
        for i in (0, 1, 17, 40):
            # the map is linear, so the difference quotient is exact but for rounding: 2 values of up to
            # (|x| + eps) * 3 off by ROPE_UNITS each, over 2 eps, summed against dy
            eps = 0.5
            xs = [x.clone(), x.clone()]
            xs[0][..., i] += eps
            xs[1][..., i] -= eps
            f = [fa.rope_forward(t.cuda(), turns, pos.cuda(), layout=layout, amplitude=1.5).cpu().double() for t in xs]
            diff = ((f[0] - f[1]) * dy.double()).sum(-1) / (2 * eps)
            tol = ROPE_UNITS * 1.5 * 2 * (float(x.abs().max()) + eps) * 2 / (2 * eps) * float(dy.abs().sum(-1).max())
            assert np.abs(diff.numpy() - got[..., i]).max() <= tol + 2 * ROPE_UNITS * 3 * float(dy.abs().max())


def test_rope_attention_chain_gradients():
    """Rotation, attention and both backward passes in a row: dX_q and dX_k
    against the oracle's chain."""
    B, H, N, d = 1, 2, 200, 64
    scale = scale_for(d)
    g = torch.Generator().manual_seed(5)
    x = {n: torch.randn(B, N, H, d, generator=g).to(BF16) for n in ("q", "k")}
    v, do = (torch.randn(B, H, N, d, generator=g).to(BF16) for _ in range(2))
    turns = fa.rope_turns(d, device="cuda")
    q, k = (fa.rope_forward(x[n].cuda().transpose(1, 2), turns) for n in ("q", "k"))
    o, lse = fa.forward(q, k, v.cuda(), causal=True, scale=scale)
    dq, dk, dv = fa.backward(q, k, v.cuda(), o, lse, do.cuda(), causal=True, scale=scale)
    gq, gk = (fa.rope_backward(t, turns) for t in (dq, dk))
    fa.sync_status()
    freqs = serving.rope_frequencies(d)
    pos = np.arange(N)[None]
    rq, rk, rv, _ = oracle.backward(to64(q.cpu()), to64(k.cpu()), to64(v), to64(do), scale, True)
    # the attention gradients' stated bound (2e-2 per element) through a rotation: sqrt(2) of it
    for got, ref in ((gq, serving.rope(rq, pos, freqs, inverse=True)), (gk, serving.rope(rk, pos, freqs, inverse=True))):
        assert np.abs(got.cpu().double().numpy() - ref).max() <= 2e-2 * 2 ** 0.5 + 1e-5


def test_rope_graph_and_streams():
    """Captured and replayed on new contents, and queued on a side stream."""
    x = torch.randn(2, 3, 40, 128).to(BF16).cuda()
    turns = fa.rope_turns(128, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    fa.rope_forward(x, turns, pos, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.rope_forward(x, turns, pos, out=y)
    x.copy_(torch.randn(2, 3, 40, 128).to(BF16))
    pos.add_(1234)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = fa.rope_forward(x, turns, pos)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, z)


# ------------------------------------------------------------------- append


def make_cache(B, Hkv, d, page, lens, extra=3, fill=float("nan"), seed=0):
    """Pages full of `fill` and a shuffled table that gives each sequence the
    pages of its length; unused entries are -1."""
    g = torch.Generator().manual_seed(seed)
    used = [(n + page - 1) // page for n in lens]
    total = sum(used) + extra
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((B, max(1, max(used)) + 2), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    kp = torch.full((total, Hkv, page, d), fill).to(BF16)
    return kp, kp.clone(), table


@pytest.mark.parametrize("B,Hq,Hkv,N,d,page,rot,layout,lens_k,lens_q", [
    (1, 1, 1, 1, 64, 16, 64, "half", [1], None),
    (3, 4, 2, 1, 128, 16, 128, "half", [1, 17, 300], None),
    (4, 6, 3, 50, 128, 32, 32, "interleaved", [50, 75, 64, 0], [50, 11, 0, 50]),
    (2, 5, 1, 40, 64, 48, 64, "half", [97, 20], [40, 40]),          # second: 20 tokens before position 0
    (2, 2, 2, 33, 128, 256, 0, "half", [600, 33], [33, 1]),          # no rotation
    (9, 16, 8, 3, 128, 64, 128, "interleaved", [3, 64, 65, 66, 67, 128, 1000, 4, 5], [3, 2, 1, 0, 3, 3, 3, 3, 3]),
])
def test_append_matches_oracle(B, Hq, Hkv, N, d, page, rot, layout, lens_k, lens_q):
    kp, vp, table = make_cache(B, Hkv, d, page, lens_k, fill=3.0)
    g = torch.Generator().manual_seed(N + d)
    fused = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).to(BF16)
    q, k, v = (t.transpose(1, 2) for t in fused.split([Hq, Hkv, Hkv], 2))
    turns = fa.rope_turns(rot, device="cuda", **SCALINGS["wide"]) if rot else None
    dk, dv, dt = kp.cuda(), vp.cuda(), table.cuda()
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    lq = torch.tensor(lens_q, dtype=torch.int32, device="cuda") if lens_q else None
    dev = fused.cuda()
    gq, gk, gv = (t.transpose(1, 2) for t in dev.split([Hq, Hkv, Hkv], 2))
    q_out = torch.full((B, Hq, N, d), 9.0, dtype=BF16, device="cuda")
    res = fa.kv_append(gk, gv, dk, dv, dt, lk, lq, turns=turns, layout=layout, amplitude=1.1, q=gq, q_out=q_out)
    fa.sync_status()
    assert res is q_out
    ql = lens_q or [N] * B
    pos = np.array([[lens_k[b] - ql[b] + t for t in range(N)] for b in range(B)])
    freqs = serving.rope_frequencies(rot, **SCALINGS["wide"]) if rot else np.zeros(0)
    amp = 1.1 if rot else 1.0
    rk = serving.rope(to64(k), pos, freqs, layout, amp)
    bk = rope_bound(to64(k), rk, rot, layout, amp, BF16) if rot else np.zeros_like(rk)
    zero = np.zeros_like(to64(kp))
    want = serving.place_tokens(to64(kp), rk, table.numpy(), ql, lens_k)
    bound = serving.place_tokens(zero, bk, table.numpy(), ql, lens_k)
    assert np.all(np.abs(to64(dk.cpu()) - want) <= bound)
    assert np.array_equal(to64(dv.cpu()), serving.place_tokens(to64(vp), to64(v), table.numpy(), ql, lens_k))
    rq = serving.rope(to64(q), pos, freqs, layout, amp)
    bq = rope_bound(to64(q), rq, rot, layout, amp, BF16) if rot else np.zeros_like(rq)
    live = np.array([[t < ql[b] for t in range(N)] for b in range(B)])[:, None, :, None]
    assert np.all(np.abs(to64(q_out.cpu()) - np.where(live, rq, 9.0)) <= np.where(live, bq, 0.0))
    # the same call without q leaves the same cache
    dk2, dv2 = kp.cuda(), vp.cuda()
    assert fa.kv_append(gk, gv, dk2, dv2, dt, lk, lq, turns=turns, layout=layout, amplitude=1.1) is None
    fa.sync_status()
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
    # a separate rotation gives the same bits as the fused one
    if rot:
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        sep = fa.rope_forward(gq, turns, p, layout=layout, amplitude=1.1)
        lv = torch.tensor(np.broadcast_to(live, sep.shape).copy()).cuda()
        assert torch.equal(torch.where(lv, sep, torch.full_like(sep, 9.0)), q_out)


def test_append_given_positions():
    """positions replace the angles, not the place in the cache."""
    kp, vp, table = make_cache(2, 2, 64, 16, [20, 5], fill=0.0)
    k = torch.randn(2, 2, 4, 64).to(BF16).cuda()
    turns = fa.rope_turns(64, device="cuda")
    pos = torch.tensor([[5, 5, 9, 0], [100, 3, -7, 2]], dtype=torch.int32, device="cuda")
    lk = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    a, b = kp.cuda(), vp.cuda()
    fa.kv_append(k, k, a, b, table.cuda(), lk, turns=turns, positions=pos)
    fa.sync_status()
    turned = fa.rope_forward(k, turns, pos).cpu()
    want = serving.place_tokens(to64(kp), to64(turned), table.numpy(), [4, 4], [20, 5])
    assert np.array_equal(to64(a.cpu()), want)


def test_append_bad_pages_write_nothing_and_are_reported():
    kp, vp, table = make_cache(3, 1, 64, 16, [10, 10, 10], fill=1.0)
    table[0, 0] = -1
    table[2, 0] = kp.shape[0]
    k = torch.randn(3, 1, 2, 64).to(BF16).cuda()
    a, b = kp.cuda(), vp.cuda()
    fa.kv_append(k, k, a, b, table.cuda(), torch.tensor([10, 10, 10], dtype=torch.int32, device="cuda"))
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_BAD_PAGE
    fa.sync_status()  # reported once
    want = serving.place_tokens(to64(kp)[:, :], np.where(np.arange(3)[:, None, None, None] == 1, to64(k.cpu()), 1.0),
                                np.clip(table.numpy(), 0, kp.shape[0] - 1), [0, 2, 0], [10, 10, 10])
    assert np.array_equal(to64(a.cpu()), want) and np.array_equal(to64(b.cpu()), want)


def test_append_captured_steps():
    """A decoding loop's append replayed from a graph while the lengths grow on the device."""
    B, Hkv, d, page = 3, 2, 128, 16
    kp, vp, table = make_cache(B, Hkv, d, page, [40, 40, 40], fill=0.0)
    turns = fa.rope_turns(d, device="cuda")
    a, b, t = kp.cuda(), vp.cuda(), table.cuda()
    lk = torch.tensor([5, 9, 14], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(B, Hkv, 1, d, dtype=BF16, device="cuda") for _ in range(2))
    fa.kv_append(k, v, a, b, t, lk, turns=turns)
    torch.cuda.synchronize()
    a.zero_(), b.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lk.add_(1)
        fa.kv_append(k, v, a, b, t, lk, turns=turns)
    lk.copy_(torch.tensor([5, 9, 14], dtype=torch.int32))
    want_k, want_v = to64(kp), to64(vp)
    for step in range(20):
        nk, nv = torch.randn(2, B, Hkv, 1, d).to(BF16)
        k.copy_(nk), v.copy_(nv)
        graph.replay()
        lens = [5 + step + 1, 9 + step + 1, 14 + step + 1]
        turned = fa.rope_forward(nk.cuda(), turns, torch.tensor([[n - 1] for n in lens], dtype=torch.int32,
                                                                device="cuda")).cpu()
        want_k = serving.place_tokens(want_k, to64(turned), table.numpy(), [1] * B, lens)
        want_v = serving.place_tokens(want_v, to64(nv), table.numpy(), [1] * B, lens)
    torch.cuda.synchronize()
    assert np.array_equal(to64(a.cpu()), want_k) and np.array_equal(to64(b.cpu()), want_v)


def test_many_heads_of_one_token():
    """More heads than a grid's second axis has blocks."""
    H, d = 70000, 64
    x = torch.randn(1, H, 1, d, dtype=BF16, device="cuda")
    turns = fa.rope_turns(d, device="cuda")
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    y = fa.rope_forward(x, turns, pos)
    assert torch.equal(y.view(H, 1, 1, d), fa.rope_forward(x.view(H, 1, 1, d), turns, pos))
    kp, vp = (torch.zeros(1, H, 16, d, dtype=BF16, device="cuda") for _ in range(2))
    fa.kv_append(x, x, kp, vp, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                 torch.tensor([5], dtype=torch.int32, device="cuda"), turns=turns, positions=pos.view(1, 1))
    fa.sync_status()
    assert torch.equal(kp[:, :, 4:5], y) and torch.equal(vp[:, :, 4:5], x)
    assert not kp[:, :, :4].any() and not vp[:, :, 5:].any()


@pytest.mark.parametrize("N,lens_k,lens_q", [
    (1, [97, 96, 300], None),                 # one token past six pages of 16, the last place, far behind the end
    (40, [100, 130, 96], None),               # across the end, 34 tokens past it, up to it
    (3, [2 ** 31 - 1, 2, 98], [3, 3, 1]),     # the largest length; a token before position 0; one past the end
])
def test_append_past_the_table_keeps_the_cache_and_is_reported(N, lens_k, lens_q):
    """Tokens behind the last place that the table reaches: no row of the cache
    changes for them, q is rotated by their own positions, and the call is
    reported; the other tokens are where they belong."""
    B, Hq, Hkv, d, page, pages = 3, 4, 2, 64, 16, 6
    g = torch.Generator().manual_seed(N)
    kp, vp = (torch.randn(B * pages + 1, Hkv, page, d, generator=g).to(BF16) for _ in range(2))
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages)
    q, k, v = (torch.randn(B, h, N, d, generator=g).to(BF16) for h in (Hq, Hkv, Hkv))
    turns = fa.rope_turns(d, device="cuda")
    a, b = kp.cuda(), vp.cuda()
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    lq = torch.tensor(lens_q, dtype=torch.int32, device="cuda") if lens_q else None
    q_out = torch.full((B, Hq, N, d), 9.0, dtype=BF16, device="cuda")
    fa.kv_append(k.cuda(), v.cuda(), a, b, table.cuda(), lk, lq, turns=turns, q=q.cuda(), q_out=q_out)
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_BAD_PAGE
    ql = lens_q or [N] * B
    pos = [[lens_k[i] - ql[i] + t for t in range(N)] for i in range(B)]
    _, site, sequence, position = fa.fa_last_failure()
    assert site == 81 and position in [p for p in pos[sequence][:ql[sequence]] if p >= pages * page]
    fa.sync_status()  # reported once
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    rk, rq = fa.rope_forward(k.cuda(), turns, p).cpu(), fa.rope_forward(q.cuda(), turns, p).cpu()
    for i in range(B):
        for t in range(ql[i]):
            if 0 <= pos[i][t] < pages * page:
                at = table[i, pos[i][t] // page], slice(None), pos[i][t] % page
                kp[at], vp[at] = rk[i, :, t], v[i, :, t]
            assert torch.equal(q_out[i, :, t].cpu(), rq[i, :, t])
        assert bool((q_out[i, :, ql[i]:] == 9.0).all())
    assert torch.equal(a.cpu(), kp) and torch.equal(b.cpu(), vp)


def test_append_loop_runs_over_the_end_of_its_table():
    """A captured decoding loop replayed past the table's end: the last rows
    stay what the last tokens with a place were."""
    kp, vp = (torch.zeros(2, 1, 16, 64, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lk = torch.tensor([0], dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 1, 1, 64, dtype=BF16, device="cuda")
    fa.kv_append(x, x, kp, vp, table, lk)  # a first call: position -1, nothing written
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lk.add_(1)
        x.add_(1)
        fa.kv_append(x, x, kp, vp, table, lk)
    lk.zero_(), x.zero_()
    for _ in range(32):
        graph.replay()
    fa.sync_status()
    want = torch.arange(1, 33).to(BF16).view(2, 16).flip(0)  # page 1 first
    assert torch.equal(kp[:, 0, :, 0].cpu(), want)
    for _ in range(5):
        graph.replay()
    with pytest.raises(fa.FAError):
        fa.sync_status()
    assert torch.equal(kp[:, 0, :, 0].cpu(), want) and torch.equal(vp[:, 0, :, 5].cpu(), want)


def test_angles_are_within_the_stated_bound():
    """Random frequency words and positions of either sign: cosine and sine of
    the phase, whose error is the cut at 2^-32 turns, the rounding to fp32
    (2^-26 turns) and sincospif's own (2 steps of at most 2^-23)."""
    rng = np.random.default_rng(3)
    N, d = 4096, 128
    words = rng.integers(-2 ** 63, 2 ** 63, d // 2, dtype=np.int64)
    words[:4] = [2 ** 63 - 1, -2 ** 63, 2 ** 33 + 1, -1]
    pos = rng.integers(-2 ** 31, 2 ** 31, N)
    pos[:4] = [2 ** 31 - 1, -2 ** 31, 0, -1]
    x = torch.zeros(1, 1, N, d)
    x[..., :d // 2] = 1.0
    y = fa.rope_forward(x.cuda(), torch.tensor(words).cuda(), torch.tensor(pos, dtype=torch.int32).cuda())
    fa.sync_status()
    phase = (words.astype(np.uint64)[None] * pos.astype(np.int64).astype(np.uint64)[:, None])  # modulo 2^64
    angle = phase.astype(np.int64).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    want = np.concatenate([np.cos(angle), np.sin(angle)], -1)
    bound = 2 * np.pi * (2.0 ** -26 + 2.0 ** -32) + 2 * 2.0 ** -23
    assert np.abs(y[0, 0].cpu().double().numpy() - want).max() <= bound
