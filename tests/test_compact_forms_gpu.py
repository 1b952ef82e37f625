"""fa_kv_compact as a program calls it: outputs with a row stride, a guarded
workspace, two streams at once, captured calls whose counts change, other
devices' and other sizes' tensors refused."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa
from exact_tiled_attention_18_gb300.binding import FA_ERR_INVALID_ARG
from tests.test_pages_gpu import KV8, compact, cuda, make_tensors, moved, raw

pytestmark = pytest.mark.gpu

PAGE, PAGES, WIDTH = 16, 90, 12
LENS = [150, 16, 0, 77]


def make_case(seed, share):
    """A table and the counts of its pages, others in use besides."""
    r = np.random.RandomState(seed)
    refs = np.where(r.rand(PAGES) < share, r.randint(1, 4, PAGES), 0).astype(np.int32)
    table = np.full((len(LENS), WIDTH), -5, dtype=np.int32)
    ids = r.permutation(PAGES)
    at = 0
    for b, n in enumerate(LENS):
        used = -(-n // PAGE)
        table[b, :used] = ids[at:at + used]
        at += used
        np.add.at(refs, table[b, :used], 1)
    return table, refs


def test_outputs_workspaces_and_streams():
    g = torch.Generator().manual_seed(4)
    tensors = make_tensors(g, PAGES, PAGE, KV8)
    cases = [make_case(s, share) for s, share in ((1, 0.3), (2, 0.0), (3, 0.9))]
    need = fa.fa_kv_compact_workspace_bytes(PAGES) // 4
    sets = []
    for _ in cases:
        dev = [t.clone().cuda() for t in tensors]
        wide = torch.full((len(LENS), WIDTH + 5), 77, dtype=torch.int32, device="cuda")
        guarded = [torch.full((PAGES + 8,), 55, dtype=torch.int32, device="cuda") for _ in range(2)]
        ws = torch.full((need + 8,), 99, dtype=torch.int32, device="cuda")
        out = (wide[:, 2:2 + WIDTH], guarded[0][:PAGES], guarded[1][:PAGES])
        sets.append((dev, fa.PagePool(dev, PAGE), wide, ws, guarded, out, torch.cuda.Stream()))
    inputs = [cuda(table, LENS, refs) for table, refs in cases]
    torch.cuda.synchronize()
    for s, x in zip(sets, inputs):
        with torch.cuda.stream(s[6]):
            got = fa.kv_compact(s[1], *x, workspace=s[3][:need], out=s[5])
            assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, s[5]))
    torch.cuda.synchronize()
    fa.sync_status()

    def verify(s, case):
        table, refs = case
        out, out_refs, new_ids, copies = compact(table, LENS, refs, PAGE)
        for t, w in zip(s[5], (out, out_refs, new_ids)):
            assert np.array_equal(t.cpu().numpy(), w)
        for t, w in zip(s[0], moved(tensors, copies, PAGE)):
            assert np.array_equal(raw(t), w)
        assert torch.all(s[2][:, :2] == 77) and torch.all(s[2][:, 2 + WIDTH:] == 77)
        assert torch.all(s[3][need:] == 99) and all(torch.all(x[PAGES:] == 55) for x in s[4])

    for s, case, x in zip(sets, cases, inputs):
        verify(s, case)
        for t, w in zip(x, (case[0], LENS, case[1])):
            assert np.array_equal(t.cpu().numpy(), w)
    # two captured calls, each with a workspace of its graph's, replayed at once
    # while their tables and counts change
    graphs = []
    for s, x in zip(sets[:2], inputs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.kv_compact(s[1], *x, out=s[5])
        graphs.append(graph)
    for turn in range(3):
        now = [cases[(turn + i) % 3] for i in range(2)]
        for s, x, (table, refs) in zip(sets, inputs, now):
            for t, fresh in zip(s[0], tensors):
                t.copy_(fresh)
            x[0].copy_(torch.tensor(table))
            x[2].copy_(torch.tensor(refs))
        torch.cuda.synchronize()
        for s, graph in zip(sets, graphs):
            with torch.cuda.stream(s[6]):
                graph.replay()
        torch.cuda.synchronize()
        fa.sync_status()
        for s, case in zip(sets, now):
            verify(s, case)


def test_wrong_outputs_and_workspaces_are_refused():
    g = torch.Generator().manual_seed(4)
    tensors = [t.cuda() for t in make_tensors(g, PAGES, PAGE, KV8)]
    before = [raw(t) for t in tensors]
    pool = fa.PagePool(tensors, PAGE)
    table, refs = make_case(1, 0.3)
    x = cuda(table, LENS, refs)
    out = [torch.empty_like(t) for t in (x[0], x[2], x[2])]
    need = fa.fa_kv_compact_workspace_bytes(PAGES) // 4
    for bad in ([out[0][:, 1:], out[1], out[2]], [out[0], out[1][1:], out[2]], [out[0], out[1].long(), out[2]],
                [out[0], out[1].cpu(), out[2]], out[:2]):
        with pytest.raises(ValueError):
            fa.kv_compact(pool, *x, out=bad)
    for bad in (torch.empty(need - 1, dtype=torch.int32, device="cuda"), torch.empty(need, device="cuda"),
                torch.empty(need, dtype=torch.int32)):
        with pytest.raises(ValueError):
            fa.kv_compact(pool, *x, workspace=bad)
    both = torch.empty(len(LENS), 2 * WIDTH, dtype=torch.int32, device="cuda")
    both[:, :WIDTH] = x[0]
    for old, bad in ((x[0], [x[0], out[1], out[2]]), (x[0], [out[0], x[2], out[2]]), (x[0], [out[0], out[1], out[1]]),
                     (both[:, :WIDTH], [both[:, WIDTH:], out[1], out[2]])):
        with pytest.raises(fa.FAError) as e:
            fa.kv_compact(pool, old, x[1], x[2], out=bad)
        assert e.value.status == FA_ERR_INVALID_ARG
    fa.sync_status()
    for t, w in zip(tensors, before):
        assert np.array_equal(raw(t), w)
