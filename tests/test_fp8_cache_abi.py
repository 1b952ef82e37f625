"""The cache in E4M3 and the calls on its pages, on the CPU: what they refuse
before they touch a device, and the binding's checks."""

import ctypes

import pytest
import torch

from tests.test_abi import fa  # noqa: F401  (fixture: the built library)
from tests.test_serving_abi import APPEND, BIG, FAKE, PAGED, PAGED_ERRORS, PREFIX, call


def with_scales(base):
    a = {}
    for name, value in base.items():
        a[name] = value
        if name == "vp":
            a["ks"], a["vs"] = FAKE, FAKE
    return a


APPEND8 = {}
for _name, _value in APPEND.items():
    APPEND8[_name] = _value
    if _name == "vp":
        APPEND8["kscale"], APPEND8["vscale"] = FAKE, FAKE


@pytest.mark.parametrize("change,expect", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(kscale=0), 1), (dict(vscale=0), 1),
    (dict(table=0), 1), (dict(lk=0), 1), (dict(q=0), 1), (dict(q_out=0), 1),
    (dict(pages=0), 1), (dict(page=8), 1), (dict(page=24), 1), (dict(max_pages=0), 1), (dict(stride=-1), 1),
    (dict(max_pages=BIG, page=16), 1), (dict(pages=BIG, Hkv=2), 1), (dict(rot=72), 1), (dict(layout=-1), 1),
    (dict(turns=0, positions=FAKE), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(Hkv=0), 1), (dict(d=80), 2),
    (dict(amplitude=float("inf")), 1), (dict(kscale=FAKE + 2), 3), (dict(vscale=FAKE + 1), 3),
    (dict(k=FAKE + 2), 3), (dict(q_out=FAKE + 8), 3), (dict(kp=FAKE + 4), 3), (dict(lk=FAKE + 1), 3),
    (dict(vs=(4096, 1024, 68)), 3), (dict(ks=(-8, 1024, 64)), 1), (dict(q_out=FAKE, qs=(8192, 512, 64)), 1),
])
def test_append_argument_errors(fa, change, expect):
    st = call(fa.fa_kv_append_fp8, APPEND8, change)
    assert st == expect, fa.fa_status_string(st)


SCALE_ERRORS = [(dict(ks=0), 1), (dict(vs=0), 1), (dict(ks=FAKE + 2), 3), (dict(vs=FAKE + 3), 3)]


@pytest.mark.parametrize("change,expect", PAGED_ERRORS + SCALE_ERRORS)
def test_paged_argument_errors(fa, change, expect):
    st = call(fa.fa_fwd_paged_fp8, with_scales(PAGED), change)
    assert st == expect, fa.fa_status_string(st)


@pytest.mark.parametrize("change,expect", PAGED_ERRORS + SCALE_ERRORS + [
    (dict(ptable=0), 1), (dict(plen=0), 1), (dict(plen=8), 1), (dict(plen=40), 1), (dict(plen=80), 1),
    (dict(plen=-16), 1), (dict(ptable=FAKE + 2), 3),
])
def test_shared_prefix_argument_errors(fa, change, expect):
    st = call(fa.fa_fwd_shared_prefix_fp8, with_scales(PREFIX), change)
    assert st == expect, fa.fa_status_string(st)


def tensors(fa, *items):
    a = (fa.fa_page_tensor * max(1, len(items)))()
    for x, (base, heads, rows, row_bytes) in zip(a, items):
        x.base, x.heads, x.rows, x.row_bytes = base, heads, rows, row_bytes
    return a


FORK = dict(tensors=None, count=0, pages=8, page=16, table=FAKE, stride=4, max_pages=4, lk=FAKE, B=2, refs=FAKE,
            sources=FAKE, rows=3, out_table=FAKE + 4096, out_stride=4, out_lk=FAKE + 8192, out_refs=FAKE + 12288,
            ws=FAKE + 20480, stream=0)
COMPACT = dict(tensors=None, count=0, pages=8, page=16, table=FAKE, stride=4, max_pages=4, lk=FAKE, B=2, refs=FAKE,
               out_table=FAKE + 4096, out_stride=4, out_refs=FAKE + 12288, new_ids=FAKE + 16384, ws=FAKE + 20480,
               stream=0)
TABLE_ERRORS = [
    (dict(table=0), 1), (dict(lk=0), 1), (dict(refs=0), 1), (dict(out_table=0), 1), (dict(out_refs=0), 1),
    (dict(pages=0), 1), (dict(page=0), 1), (dict(page=24), 1), (dict(max_pages=0), 1), (dict(max_pages=BIG), 1),
    (dict(B=0), 1), (dict(stride=-1), 1), (dict(out_stride=3), 1), (dict(count=-1), 1), (dict(count=1), 1),
    (dict(table=FAKE + 2), 3), (dict(lk=FAKE + 1), 3), (dict(refs=FAKE + 2), 3), (dict(out_table=FAKE + 4098), 3),
    (dict(out_refs=FAKE + 12289), 3), (dict(ws=FAKE + 8), 3),
    (dict(out_table=FAKE), 1), (dict(out_table=FAKE + 28), 1), (dict(out_refs=FAKE), 1), (dict(out_refs=FAKE + 28), 1),
    (dict(pages=(1 << 30) + 1), 1), (dict(out_refs=FAKE + 4096), 1), (dict(ws=FAKE + 16), 1), (dict(ws=FAKE + 4096), 1),
    (dict(lk=FAKE + 4096), 1), (dict(lk=FAKE + 12292), 1),
]


@pytest.mark.parametrize("change,expect", TABLE_ERRORS + [
    (dict(sources=0), 1), (dict(out_lk=0), 1), (dict(rows=0), 1), (dict(sources=FAKE + 2), 3),
    (dict(out_lk=FAKE + 1), 3), (dict(out_lk=FAKE + 4), 1), (dict(sources=FAKE + 4096), 1), (dict(out_lk=FAKE + 12288), 1),
])
def test_fork_argument_errors(fa, change, expect):
    st = call(fa.fa_kv_fork, FORK, change)
    assert st == expect, fa.fa_status_string(st)


@pytest.mark.parametrize("change,expect", TABLE_ERRORS + [
    (dict(new_ids=0), 1), (dict(new_ids=FAKE + 16385), 3), (dict(new_ids=FAKE), 1), (dict(new_ids=FAKE + 12288), 1),
])
def test_compact_argument_errors(fa, change, expect):
    st = call(fa.fa_kv_compact, COMPACT, change)
    assert st == expect, fa.fa_status_string(st)


@pytest.mark.parametrize("item,expect", [
    ((0, 1, 16, 128), 1), ((FAKE, 0, 16, 128), 1), ((FAKE, 1, 0, 128), 1), ((FAKE, 1, 5, 128), 1), ((FAKE, 1, 32, 128), 1),
    ((FAKE, 1, 16, 0), 1), ((FAKE, 1, 16, 2), 1), ((FAKE, 1, 16, 6), 1), ((FAKE + 2, 1, 16, 128), 3),
    ((FAKE, 1 << 20, 16, 128), 1),
])
def test_page_tensor_errors(fa, item, expect):
    good = (FAKE, 2, 1, 4)
    for fn, base in ((fa.fa_kv_fork, FORK), (fa.fa_kv_compact, COMPACT)):
        st = call(fn, base, dict(tensors=tensors(fa, good, item), count=2))
        assert st == expect, fa.fa_status_string(st)


def test_workspace_bytes(fa):
    assert fa.fa_kv_fork_workspace_bytes(0, 1) == 0 and fa.fa_kv_fork_workspace_bytes(1, 0) == 0
    assert 0 < fa.fa_kv_fork_workspace_bytes(4, 8) < fa.fa_kv_fork_workspace_bytes(4, 800)
    assert fa.fa_kv_compact_workspace_bytes(0) == 0
    assert 0 < fa.fa_kv_compact_workspace_bytes(1) < fa.fa_kv_compact_workspace_bytes(1000)


def test_status_strings(fa):
    assert fa.FA_ERR_NO_PAGES == 8 and "FA_ERR_NO_PAGES" in fa.fa_status_string(8)


def test_binding_refuses_cpu_tensors_and_wrong_types(fa):
    z = torch.zeros
    q = z(1, 2, 1, 64, dtype=torch.bfloat16)
    pages = z(2, 2, 16, 64, dtype=torch.float8_e4m3fn)
    scales, table, lens = z(2, 2, 1), z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.forward_paged_fp8(q, pages, pages, scales, scales, table, lens)
    with pytest.raises(ValueError):
        fa.forward_shared_prefix_fp8(q, pages, pages, scales, scales, table[0], 16, table, lens)
    with pytest.raises(ValueError):
        fa.kv_append_fp8(q, q, pages, pages, scales, scales, table, lens)
    with pytest.raises(ValueError):
        fa.PagePool([pages], 16)
    with pytest.raises(ValueError):
        fa.PagePool([], 16)


def test_page_tensor_layout_is_the_headers(fa):
    assert ctypes.sizeof(fa.fa_page_tensor) == 24
    assert [getattr(fa.fa_page_tensor, n).offset for n in ("base", "heads", "rows", "row_bytes")] == [0, 8, 12, 16]
