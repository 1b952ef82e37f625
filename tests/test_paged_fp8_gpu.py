"""Attention over the paged cache in E4M3 (fa_fwd_paged_fp8) and behind a shared
prefix (fa_fwd_shared_prefix_fp8), against the fp64 oracle on the values that
the cache stands for."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from oracle import serving
from tests.helpers import scale_for, to64
from tests.test_paged_gpu import CHUNKS, PREFIXES, STEPS
from tests.test_rope_gpu import make_cache

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Cache:
    """Pages of random E4M3 numbers at the sequences' positions and NaN behind
    them, with a scale of its own (no power of two) for every cell that holds a
    token and NaN for the others."""

    def __init__(self, B, Hkv, d, page, lens_k, seed=0, spread=0.5):
        g = torch.Generator().manual_seed(seed)
        kp, _, self.table = make_cache(B, Hkv, d, page, lens_k, seed=seed)
        n = kp.shape[0]
        self.page, self.pages, self.scales, self.values = page, [], [], []
        live = torch.zeros(n, page, dtype=torch.bool)
        for b, length in enumerate(lens_k):
            for i in range((length + page - 1) // page):
                live[self.table[b, i], :min(page, length - i * page)] = True
        for _ in range(2):
            x = (torch.randn(n, Hkv, page, d, generator=g) * 100).clamp(-448, 448).to(E4M3)
            scale = 0.01 * torch.exp(torch.randn(n, Hkv, page // 16, generator=g) * spread)
            raw = x.view(torch.uint8)
            raw[~live[:, None].expand(n, Hkv, page)] = 0x7F
            scale[~live.view(n, 1, page // 16, 16).any(-1).expand_as(scale)] = float("nan")
            self.pages.append(x)
            self.scales.append(scale)
        self.update()

    def update(self):
        """The values that the cache stands for, in 64 bits."""
        self.values = [to64(x.float()) * np.repeat(to64(s), 16, axis=2)[..., None]
                       for x, s in zip(self.pages, self.scales)]

    def cuda(self):
        return [t.cuda() for t in (*self.pages, *self.scales, self.table)]


def make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=0, q_scale=1.0, spread=0.5):
    g = torch.Generator().manual_seed(seed + 1000)
    q = (torch.randn(B, Hq, Nq, d, generator=g) * q_scale).to(BF16)
    return q, Cache(B, Hkv, d, page, lens_k, seed, spread)


def reference(q, c, lens_k, lens_q, causal):
    lq = lens_q if lens_q is not None else [q.shape[2]] * q.shape[0]
    return serving.paged_forward(to64(q), *c.values, c.table.numpy(), scale_for(q.shape[-1]), causal, lq, lens_k)


def run(q, c, lens_k, lens_q=None, causal=True, o_dtype=F32, prefix=0, prefix_table=None, table=None, **kw):
    k, v, ks, vs, t = c.cuda()
    t = t if table is None else table.cuda()
    lk = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    lq = torch.tensor(lens_q, dtype=torch.int32, device="cuda") if lens_q is not None else None
    if prefix:
        out = fa.forward_shared_prefix_fp8(q.cuda(), k, v, ks, vs, prefix_table.cuda(), prefix, t, lk, lq,
                                           causal=causal, o_dtype=o_dtype, **kw)
    else:
        out = fa.forward_paged_fp8(q.cuda(), k, v, ks, vs, t, lk, lq, causal=causal, o_dtype=o_dtype, **kw)
    fa.sync_status()
    return out


def check(o, lse, ref, q, c, way, what=""):
    """way: "steps" (up to 32 rows a key head) or "tiles".

    A score is off by fp32 sums of d products (each addition half a step of at
    most sum |q||k|), a few roundings of it and of log2 of a scale, and by what
    the form of a query leaves: steps, fp16 with the row's largest value at 2^14
    and more, half a step of 2^-24 at the least, 2^-39 of that value; tiles, two
    E4M3 numbers with it at 2^7 and more, 2^-10 or 2^-17 of it, for each element.
    Exponential, logarithm and sum: 2^-21.

    Weights are fp16: half a step, 2^-11 of themselves, or at least 2^-25, where
    the largest one (steps: of the tile; tiles: the row's reference, which is one
    of its keys') is 2^14 (2^7): for every key 2^-39 (2^-32) of the largest.
    """
    o_ref, lse_ref, mass = ref
    d = q.shape[-1]
    qn, kn = np.abs(to64(q)).reshape(-1, d), np.nan_to_num(np.abs(c.values[0])).reshape(-1, d)
    scale = scale_for(d)
    top = scale * np.sqrt((qn ** 2).sum(1).max() * (kn ** 2).sum(1).max())
    logs = np.abs(np.log2(to64(c.scales[1])[np.isfinite(to64(c.scales[1]))])).max(initial=0)
    left, small = {"steps": (-39, -39), "tiles": (-17, -32)}[way]
    e = ((d + 8) * 2.0 ** -24 * top + 2.0 ** -21 + logs * 2.0 ** -23
         + scale * 2.0 ** left * qn.max() * kn.sum(1).max())
    rel = 2 * e + 2.0 ** -11
    least = c.table.numel() * c.page * 2.0 ** small * np.nan_to_num(np.abs(c.values[1])).max()
    got = o.cpu().double().numpy()
    assert np.all(np.isfinite(got)), what
    out = 2.0 ** -8 if o.dtype == BF16 else 2.0 ** -24
    off = np.abs(got - o_ref)
    bound = rel * mass + least + out * (np.abs(o_ref) + rel * mass + least) + 1e-30
    assert (off - bound).max() <= 0, (what, (off - bound).max(), off.max())
    lg = lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(lg), np.isneginf(lse_ref)), what
    fin = np.isfinite(lse_ref)
    assert np.all(np.abs(lg[fin] - lse_ref[fin]) <= e + 2.0 ** -21 * (1 + np.abs(lse_ref[fin]))), what


def way_of(Hq, Hkv, Nq, prefix=0):
    return "tiles" if prefix or Hq // Hkv * Nq > 32 else "steps"


MORE_STEPS = [
    # B, Hq, Hkv, Nq, d, page, lens_k, lens_q
    (1, 4, 1, 5, 128, 64, [200], None),                          # 20 rows
    (2, 2, 1, 16, 64, 16, [16, 333], None),
    (1, 8, 1, 4, 128, 32, [1000], None),                         # 32 rows
    (3, 3, 1, 7, 64, 48, [700, 0, 129], [7, 7, 2]),
    (2, 24, 2, 2, 128, 128, [1500, 127], [2, 1]),
]


@pytest.mark.parametrize("o_dtype", [F32, BF16])
@pytest.mark.parametrize("case", STEPS + MORE_STEPS, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_steps_match_oracle(case, o_dtype):
    """Single tokens and a few drafted ones (at most 32 rows a key head)."""
    B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B, q_scale=0.7)
    o, lse = run(q, c, lens_k, lens_q, o_dtype=o_dtype)
    check(o, lse, reference(q, c, lens_k, lens_q, True), q, c, way_of(Hq, Hkv, Nq), case)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "x".join(str(x) for x in c[:6]))
def test_chunks_match_oracle(case, causal):
    """Chunks of a prompt against what is cached of it."""
    B, Hq, Hkv, Nq, d, page, lens_k, lens_q = case
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    for o_dtype in (F32, BF16):
        o, lse = run(q, c, lens_k, lens_q, causal=causal, o_dtype=o_dtype)
        check(o, lse, reference(q, c, lens_k, lens_q, causal), q, c, way_of(Hq, Hkv, Nq), case)


def with_prefix(c, prefix, lens_k):
    """Every sequence starts with the longest one's pages: their table, and a
    block table without those entries."""
    n = prefix // c.page
    prefix_table = c.table[int(np.argmax(lens_k)), :n].clone()
    c.table[:, :n] = prefix_table
    blind = c.table.clone()
    blind[:, :n] = -1  # entries of the prefix are not read
    return dict(prefix=prefix, prefix_table=prefix_table, table=blind)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", PREFIXES, ids=lambda c: "x".join(str(x) for x in c[:7]))
def test_shared_prefix_matches_oracle(case, causal):
    B, Hq, Hkv, Nq, d, page, prefix, lens_k, lens_q = case
    q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens_k, seed=Nq + d + B)
    kw = with_prefix(c, prefix, lens_k)
    ref = reference(q, c, lens_k, lens_q, causal)
    for o_dtype in (F32, BF16):
        o, lse = run(q, c, lens_k, lens_q, causal=causal, o_dtype=o_dtype, **kw)
        check(o, lse, ref, q, c, "tiles", case)
