"""fp64 CPU oracle for rotary positions and the paged key/value cache.

TEST INFRASTRUCTURE ONLY, like oracle/attention.py.  Written from the
definitions: a pair (a, b) at position p turns by the angle p * f_i; position
p of sequence b lives in row p % page_size of page table[b][p // page_size];
attention over the cache is the padded-batch attention of oracle/attention.py
on the keys and values gathered position by position, query head h reading key
head h // (Hq / Hkv).
"""

from __future__ import annotations

import numpy as np

from .attention import forward_varlen

__all__ = ["rope_frequencies", "rope", "place_tokens", "gather_cache", "paged_forward"]


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=1.0, low=1.0, high=32.0):
    """Radians per position of each pair (see include/fa.h, fa_rope_scaling)."""
    out = []
    for i in range(rot_dim // 2):
        b = base * factor ** (rot_dim / (rot_dim - 2)) if scaling == "ntk" else base
        f = 1.0 / b ** (2 * i / rot_dim)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            turns = original_len * f / (2 * np.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out)


def rope(x, positions, freqs, layout="half", amplitude=1.0, inverse=False):
    """x [B, H, N, d] rotated; positions [B, N]."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    angle = np.asarray(positions, dtype=np.float64)[:, None, :] * (-1.0 if inverse else 1.0)
    for i, f in enumerate(freqs):
        ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = amplitude * (a * np.cos(angle * f) - b * np.sin(angle * f))
        y[..., ib] = amplitude * (b * np.cos(angle * f) + a * np.sin(angle * f))
    return y


def place_tokens(pages, new, table, seqlens_q, seqlens_k):
    """pages [P, Hkv, page, d] with the tokens new [B, Hkv, N, d] at their positions."""
    out = np.array(pages, dtype=np.float64)
    page = pages.shape[2]
    for b in range(new.shape[0]):
        for t in range(int(seqlens_q[b])):
            p = int(seqlens_k[b]) - int(seqlens_q[b]) + t
            if p >= 0:
                out[table[b][p // page], :, p % page] = new[b, :, t]
    return out


def gather_cache(pages, table, seqlens_k, width):
    """[B, Hkv, width, d]: the sequences' rows in order, zeros behind them."""
    _, hkv, page, d = pages.shape
    out = np.zeros((len(table), hkv, width, d))
    for b, n in enumerate(seqlens_k):
        for p in range(int(n)):
            out[b, :, p] = pages[table[b][p // page], :, p % page]
    return out


def paged_forward(q, k_pages, v_pages, table, scale, causal, seqlens_q, seqlens_k):
    """O, LSE and sum_j P_ij |v_j| of q [B, Hq, Nq, d] over the paged cache."""
    width = max(1, max(int(n) for n in seqlens_k))
    group = q.shape[1] // k_pages.shape[1]
    k = np.repeat(gather_cache(k_pages, table, seqlens_k, width), group, axis=1)
    v = np.repeat(gather_cache(v_pages, table, seqlens_k, width), group, axis=1)
    o, lse = forward_varlen(q, k, v, scale, causal, seqlens_q, seqlens_k)
    mass, _ = forward_varlen(q, k, np.abs(v), scale, causal, seqlens_q, seqlens_k)
    return o, lse, mass
