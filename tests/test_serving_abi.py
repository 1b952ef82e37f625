"""Rotary positions and the paged cache on the CPU: what the calls refuse
before they touch a device, the frequency table, the binding's checks, and the
fp64 oracle's own pins."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import serving
from tests.test_abi import fa  # noqa: F401  (fixture: the built library)

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every case below fails validation first
BIG = 1 << 30


def call(fn, base, change):
    a = dict(base)
    a.update(change)
    return fn(*a.values())


ROPE = dict(x=FAKE, x_dtype=1, xs=(4096, 1024, 64), y=FAKE + 65536, y_dtype=1, ys=(4096, 1024, 64), positions=0, psb=0,
            turns=FAKE, rot=64, layout=0, amplitude=1.0, inverse=0, B=2, H=4, N=16, d=64, stream=0)


@pytest.mark.parametrize("change,expect", [
    (dict(x=0), 1), (dict(y=0), 1), (dict(turns=0), 1), (dict(x_dtype=2), 1), (dict(y_dtype=-1), 1),
    (dict(layout=2), 1), (dict(inverse=2), 1), (dict(amplitude=float("nan")), 1), (dict(amplitude=float("inf")), 1),
    (dict(rot=0), 1), (dict(rot=8), 1), (dict(rot=24), 1), (dict(rot=80), 1), (dict(rot=-16), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(N=-1), 1), (dict(B=BIG, H=2), 1), (dict(d=96), 2), (dict(d=32), 2),
    (dict(x=FAKE + 8), 3), (dict(y=FAKE + 2), 3), (dict(turns=FAKE + 4), 3), (dict(positions=FAKE + 2), 3),
    (dict(xs=(4096, 1024, 65)), 3), (dict(ys=(4096, 1028, 64)), 3), (dict(xs=(-4096, 1024, 64)), 1),
    (dict(ys=(0, 1024, 64)), 1), (dict(psb=-1), 1), (dict(ys=(4096, 1024, 48)), 1), (dict(ys=(4096, 32, 256)), 1),
    (dict(y=FAKE, ys=(8192, 1024, 64)), 1),      # in place with other strides
    (dict(y=FAKE, y_dtype=0), 1),                # in place with another type
])
def test_rope_argument_errors(fa, change, expect):
    st = call(fa.fa_rope, ROPE, change)
    assert st == expect, fa.fa_status_string(st)


APPEND = dict(k=FAKE, ks=(4096, 1024, 64), v=FAKE, vs=(4096, 1024, 64), q=FAKE, qs=(8192, 1024, 64),
              q_out=FAKE + 65536, kp=FAKE, vp=FAKE, pages=8, page=16, table=FAKE, stride=4, max_pages=4, lq=FAKE,
              lk=FAKE, positions=0, psb=0, turns=FAKE, rot=64, layout=0, amplitude=1.0, B=2, Hq=8, Hkv=4, N=16, d=64,
              stream=0)


@pytest.mark.parametrize("change,expect", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(table=0), 1), (dict(lk=0), 1),
    (dict(q=0), 1), (dict(q_out=0), 1),                       # one without the other
    (dict(pages=0), 1), (dict(page=8), 1), (dict(page=24), 1), (dict(page=0), 1), (dict(max_pages=0), 1),
    (dict(stride=-1), 1), (dict(max_pages=BIG, page=16), 1), (dict(pages=BIG, Hkv=2), 1),
    (dict(rot=72), 1), (dict(layout=-1), 1), (dict(turns=0, positions=FAKE), 1),
    (dict(B=0), 1), (dict(N=0), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(d=80), 2),
    (dict(k=FAKE + 2), 3), (dict(q_out=FAKE + 8), 3), (dict(kp=FAKE + 4), 3), (dict(lk=FAKE + 1), 3),
    (dict(lq=FAKE + 2), 3), (dict(table=FAKE + 3), 3), (dict(vs=(4096, 1024, 68)), 3), (dict(qs=(8192, 1020, 64)), 3),
    (dict(ks=(-8, 1024, 64)), 1),
    (dict(q_out=FAKE, qs=(8192, 512, 64)), 1),                # in place, not contiguous (N * d is 1024)
])
def test_append_argument_errors(fa, change, expect):
    st = call(fa.fa_kv_append, APPEND, change)
    assert st == expect, fa.fa_status_string(st)


PAGED = dict(q=FAKE, kp=FAKE, vp=FAKE, pages=8, page=16, table=FAKE, stride=4, max_pages=4, o=FAKE, o_dtype=0,
             lse=FAKE, lq=0, lk=FAKE, ws=FAKE, B=2, Hq=8, Hkv=4, Nq=1, d=64, scale=0.125, causal=1, stream=0)
PREFIX = dict(list(PAGED.items())[:5] + [("ptable", FAKE), ("plen", 32)] + list(PAGED.items())[5:])
PAGED_ERRORS = [
    (dict(q=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(table=0), 1),
    (dict(o_dtype=2), 1), (dict(causal=2), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(pages=0), 1), (dict(page=20), 1), (dict(max_pages=0), 1), (dict(stride=-4), 1),
    (dict(Hkv=3), 1), (dict(Hkv=0), 1), (dict(B=0), 1), (dict(Nq=0), 1), (dict(B=BIG, Nq=4), 1), (dict(d=256), 2),
    (dict(max_pages=BIG), 1), (dict(max_pages=(BIG >> 4) + 1), 1), (dict(pages=BIG), 1),
    (dict(q=FAKE + 8), 3), (dict(o=FAKE + 4), 3), (dict(lse=FAKE + 2), 3), (dict(ws=FAKE + 8), 3),
    (dict(lk=FAKE + 1), 3), (dict(lq=FAKE + 1), 3), (dict(kp=FAKE + 2), 3), (dict(table=FAKE + 1), 3),
]


@pytest.mark.parametrize("change,expect", PAGED_ERRORS)
def test_paged_argument_errors(fa, change, expect):
    st = call(fa.fa_fwd_paged, PAGED, change)
    assert st == expect, fa.fa_status_string(st)


@pytest.mark.parametrize("change,expect", PAGED_ERRORS + [
    (dict(ptable=0), 1), (dict(plen=0), 1), (dict(plen=8), 1), (dict(plen=40), 1), (dict(plen=80), 1),
    (dict(plen=-16), 1), (dict(ptable=FAKE + 2), 3),
])
def test_shared_prefix_argument_errors(fa, change, expect):
    st = call(fa.fa_fwd_shared_prefix, PREFIX, change)
    assert st == expect, fa.fa_status_string(st)


def test_workspace_bytes(fa):
    for f in (fa.fa_fwd_paged_workspace_bytes, fa.fa_fwd_shared_prefix_workspace_bytes):
        assert f(1, 8, 2, 1, 128) > 0
        assert f(0, 8, 2, 1, 128) == 0 and f(1, 8, 3, 1, 128) == 0 and f(1, 8, 2, 1, 96) == 0
        assert f(1, 8, 0, 1, 64) == 0 and f(1 << 20, 1 << 12, 1, 1, 64) == 0


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="parts", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
    dict(scaling="parts", factor=16.0, original_len=4096.0, low=0.0, high=32.0),
])
@pytest.mark.parametrize("rot", [16, 48, 128])
def test_turns_are_the_frequencies(fa, rot, kw):
    """turns / 2^64 turns per position = f_i radians, to the roundings of a
    few fp64 operations on either side."""
    turns = fa.rope_turns(rot, **kw)
    assert turns.dtype == torch.int64 and turns.shape == (rot // 2,)
    f = serving.rope_frequencies(rot, **kw)
    got = np.array([int(t) for t in turns]) / 2.0 ** 64 * 2 * math.pi
    assert np.all(np.abs(got - f) <= 32 * 2.0 ** -53 * f + 2.0 ** -62)


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 1.0, 1.0, 32.0), (24, 1e4, 0, 1.0, 1.0, 1.0, 32.0), (64, 1.0, 0, 1.0, 1.0, 1.0, 32.0),
    (64, float("nan"), 0, 1.0, 1.0, 1.0, 32.0), (64, 1e4, 4, 1.0, 1.0, 1.0, 32.0), (64, 1e4, 1, 0.5, 1.0, 1.0, 32.0),
    (64, 1e4, 3, 2.0, 0.0, 1.0, 32.0), (64, 1e4, 3, 2.0, 100.0, 4.0, 4.0), (64, 1e300, 2, 1e300, 1.0, 1.0, 32.0),
])
def test_turns_argument_errors(fa, args):
    out = (ctypes.c_longlong * 64)()
    assert fa.binding.lib().fa_rope_turns(out, *args) == 1
    assert fa.binding.lib().fa_rope_turns(None, 64, 1e4, 0, 1.0, 1.0, 1.0, 32.0) == 1


def test_phase_arithmetic_wraps_to_the_exact_angle(fa):
    """position * turns modulo 2^64 is the angle modulo one turn, at positions
    of either sign up to the largest int."""
    turns = [int(t) for t in fa.rope_turns(128)]
    f = serving.rope_frequencies(128)
    for p in (1, -1, 4097, 10 ** 6, -10 ** 6, 2 ** 31 - 1, -2 ** 31):
        for t, w in zip(turns[::7], f[::7]):
            phase = (p * t) % 2 ** 64
            top = phase >> 32
            top -= 2 ** 32 if top >= 2 ** 31 else 0
            angle = top / 2.0 ** 32 * 2 * math.pi
            err = abs(complex(math.cos(angle), math.sin(angle)) - complex(math.cos(p * w), math.sin(p * w)))
            assert err <= 2 * math.pi * 2.0 ** -32 + 64 * 2.0 ** -53 * abs(p)


def test_status_string_of_bad_pages(fa):
    assert fa.fa_status_string(fa.FA_ERR_BAD_PAGE).startswith("FA_ERR_BAD_PAGE")


def test_binding_refuses_cpu_tensors(fa):
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    turns = fa.rope_turns(64)
    pages = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.ones(1, dtype=torch.int32)
    for f in (lambda: fa.rope_forward(x, turns), lambda: fa.rope_backward(x, turns),
              lambda: fa.kv_append(x, x, pages, pages, table, lens),
              lambda: fa.forward_paged(x, pages, pages, table, lens),
              lambda: fa.forward_shared_prefix(x, pages, pages, table[0], 16, table, lens)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        fa.rope_turns(64, scaling="yarn")
    with pytest.raises(fa.FAError):
        fa.rope_turns(63)


# ------------------------------------------------------------ the oracle's pins


def test_oracle_rope_is_complex_multiplication():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 16))
    pos = rng.integers(-50, 50, (2, 5))
    f = serving.rope_frequencies(8)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001])
    unit = 1.5 * np.exp(1j * pos[:, None, :, None] * f)
    y = serving.rope(x, pos, f, "half", 1.5)
    z = (x[..., :4] + 1j * x[..., 4:8]) * unit
    assert np.allclose(y[..., :4], z.real) and np.allclose(y[..., 4:8], z.imag) and np.array_equal(y[..., 8:], x[..., 8:])
    y = serving.rope(x, pos, f, "interleaved", 1.5)
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * unit
    assert np.allclose(y[..., 0:8:2], z.real) and np.allclose(y[..., 1:8:2], z.imag)
    back = serving.rope(serving.rope(x, pos, f), pos, f, inverse=True)
    assert np.allclose(back, x)
    # scores of rotated rows depend on the distance alone
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    s = [float((serving.rope(q, [[a + 7]], f) * serving.rope(k, [[a]], f)).sum()) for a in (0, 5, 900)]
    assert np.allclose(s, s[0])


def test_oracle_cache_round_trip():
    """Tokens placed through a shuffled table come back in order, and paged
    attention is the contiguous attention on them."""
    rng = np.random.default_rng(1)
    new = rng.standard_normal((2, 2, 20, 8))
    table = np.array([[3, 0, -1], [4, 1, 2]])
    pages = np.full((5, 2, 8, 8), np.nan)
    out = serving.place_tokens(pages, new, table, [13, 20], [13, 20])
    back = serving.gather_cache(out, table, [13, 20], 20)
    assert np.array_equal(back[0, :, :13], new[0, :, :13]) and np.array_equal(back[1], new[1])
    q = rng.standard_normal((2, 4, 3, 8))
    o, lse, mass = serving.paged_forward(q, out, out, table, 0.3, True, [3, 2], [13, 20])
    kv = np.repeat(back, 2, axis=1)
    o2, lse2 = oracle.forward_varlen(q, kv, kv, 0.3, True, [3, 2], [13, 20])
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2) and np.all(mass >= np.abs(o) - 1e-12)


# ---------------------------------------------------------------- output rows


@pytest.mark.parametrize("ys,bad", [
    # B, H, N, d = 2, 4, 16, 64; what passes is refused behind it, for a misaligned x
    ((4096, 1024, 64), False), ((4096, 64, 256), False), ((64, 2048, 128), False), ((1 << 40, 1 << 30, 64), False),
    ((64, 1024, 64), True),           # two sequences a row apart, where the tokens lie
    ((4096, 512, 64), True),          # heads that begin inside the one before
    ((1024, 1024, 64), True),         # every sequence on the other's heads
    ((4096, 960, 64), True),          # the last token on the next head's first
    ((192, 128, 1024), False),        # sequences in the gaps between the heads
    ((160, 128, 1024), True),         # the same, half a row too near
    ((192, 384, 2048), False),        # sequences three rows apart inside the heads' gaps
    ((8192, 136, 512), False),        # gaps between the heads
    ((2048, 136, 512), True),         # the second sequence on the first one's fourth token
    ((1216, 4096, 128), False),       # not nested, and yet apart: 1216 is between two tokens' rows
    ((1152, 4096, 128), True),        # nine tokens further
])
def test_rope_output_rows_must_not_overlap(fa, ys, bad):
    """The check against the offsets of all rows, and what fa_rope makes of it."""
    offs = sorted(b * ys[0] + h * ys[1] + n * ys[2] for b in range(2) for h in range(4) for n in range(16))
    assert bad == any(b - a < 64 for a, b in zip(offs, offs[1:]))
    st = call(fa.fa_rope, ROPE, dict(ys=ys, x=FAKE + 8))
    assert st == (1 if bad else 3), fa.fa_status_string(st)


def test_rope_output_rows_of_random_strides(fa):
    rng = np.random.default_rng(5)
    seen = [0, 0]
    for _ in range(3000):
        B, H, N = (int(n) for n in rng.integers(1, 7, 3))
        ys = tuple(int(x) * 8 for x in rng.integers(0, 60, 3))
        used = [s if n > 1 else 0 for s, n in zip(ys, (B, H, N))]
        offs = sorted(b * used[0] + h * used[1] + n * used[2] for b in range(B) for h in range(H) for n in range(N))
        bad = any(b - a < 64 for a, b in zip(offs, offs[1:]))
        seen[bad] += 1
        st = call(fa.fa_rope, ROPE, dict(ys=ys, x=FAKE + 8, B=B, H=H, N=N))
        assert st == (1 if bad else 3), (B, H, N, ys)
    assert min(seen) > 300


def test_rope_output_rows_of_many_rows_are_checked_quickly(fa):
    """Strides that do not nest, with as many rows as a call may have."""
    many = dict(x=FAKE + 8, B=1023, H=1023, N=1023)
    assert call(fa.fa_rope, ROPE, dict(many, ys=(1 << 41, (1 << 24) + 64, 1 << 24))) == 3
    assert call(fa.fa_rope, ROPE, dict(many, ys=(1 << 41, (1 << 24) + 56, 1 << 24))) == 1


# --------------------------------------------------------------------- status


def test_sync_status_reads_the_device_it_is_given(fa, monkeypatch):
    """The status word is the current device's: sync_status makes the given
    device current around the call (as the calls that may set it do)."""
    binding = fa.binding
    current = [0]

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before = current[0]
            if self.device is not None:
                current[0] = self.device

        def __exit__(self, *_):
            current[0] = self.before

    class Stream:
        def __init__(self, device):
            self.cuda_stream = 100 + (current[0] if device is None else device)

    seen = []

    def status(stream):
        seen.append((current[0], stream))
        return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(binding, "fa_sync_status", status)
    fa.sync_status()
    fa.sync_status(1)
    assert seen == [(0, 100), (1, 101)] and current == [0]
