"""Forks and compaction of the cache's pages (fa_kv_fork, fa_kv_compact)
against the definition, page by page, and in a run with the appends and the
attention that use the pages."""

import numpy as np
import pytest
import torch

import exact_tiled_attention_18_gb300 as fa

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def fork(table, lens, refs, sources, page):
    """(table, lens, refs, copies (src, dst, tokens)) by the definition; refs is
    not changed."""
    refs, copies = refs.copy(), []
    width, limit = table.shape[1], table.shape[1] * page
    lens = [min(max(n, 0), limit) for n in lens]
    used = [-(-n // page) for n in lens]
    good = lambda p: 0 <= p < len(refs)  # noqa: E731
    for b in range(len(lens)):
        for p in table[b, :used[b]]:
            if good(p):
                refs[p] -= 1
    out = np.full((len(sources), width), -1, dtype=np.int32)
    out_lens, taken, need = [], set(), []
    for i, s in enumerate(sources):
        s = s if 0 <= s < len(lens) else -1
        out_lens.append(lens[s] if s >= 0 else 0)
        if s < 0:
            continue
        out[i, :used[s]] = table[s, :used[s]]
        for k in range(used[s]):
            p = table[s, k]
            if not good(p):
                continue
            if k == lens[s] // page and s in taken:  # being filled, and another row has it
                need.append((i, k, p, lens[s] % page))
            else:
                refs[p] += 1
        taken.add(s)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for (i, k, p, tokens), to in zip(need, free + [-1] * len(need)):
        out[i, k] = to
        if to >= 0:
            refs[to] = 1
            copies.append((p, to, tokens))
    return out, np.array(out_lens, dtype=np.int32), refs, copies


def compact(table, lens, refs, page):
    live = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    movers = [p for p in live if p >= n]
    new_ids = np.full(len(refs), -1, dtype=np.int32)
    out_refs = np.zeros(len(refs), dtype=np.int32)
    for p in live:
        new_ids[p] = p
    for p, to in zip(movers, holes):
        new_ids[p] = to
    for p in live:
        out_refs[new_ids[p]] = refs[p]
    out = table.copy()
    for b in range(len(lens)):
        for k in range(-(-min(max(lens[b], 0), table.shape[1] * page) // page)):
            out[b, k] = new_ids[table[b, k]]
    return out, out_refs, new_ids, [(p, to, page) for p, to in zip(movers, holes)]


def make_batch(g, lens, page, extra, width_more=1, shared=0):
    """A table of shuffled pages, the sequences' first `shared` pages in common."""
    used = [-(-n // page) for n in lens]
    total = sum(used) + extra
    order = torch.randperm(total, generator=g).numpy().astype(np.int32)
    table = np.full((len(lens), max(used) + width_more), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    for b in range(1, len(lens)):
        n = min(shared, lens[0] // page, lens[b] // page)
        table[b, :n] = table[0, :n]
    refs = np.zeros(total, dtype=np.int32)
    for b, n in enumerate(used):
        np.add.at(refs, table[b, :n], 1)
    return table, refs


def make_tensors(g, pages, page, shapes):
    """One random tensor for each (heads, kind)."""
    out = []
    for heads, kind in shapes:
        if kind == "scale":
            out.append(torch.randn(pages, heads, page // 16, generator=g))
        elif kind == "odd":  # rows of four bytes, and of twelve
            out.append(torch.randint(0, 1 << 30, (pages, heads, page, 3), generator=g, dtype=torch.int32))
        else:
            d = {"b64": 64, "b128": 128, "h64": 128}[kind]
            x = torch.randint(0, 256, (pages, heads, page, d), generator=g, dtype=torch.uint8)
            out.append(x.view(torch.bfloat16) if kind == "h64" else x.view(E4M3))
    return out


def raw(t):
    return t.cpu().contiguous().view(torch.uint8).view(*t.shape[:3], -1).numpy()


def moved(tensors, copies, page):
    want = []
    for t in tensors:
        x = raw(t).copy()
        before = x.copy()
        unit = page // x.shape[2]
        for src, dst, tokens in copies:
            rows = -(-tokens // unit)
            x[dst, :, :rows] = before[src, :, :rows]
        want.append(x)
    return want


def cuda(*xs):
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in xs]


KV8 = [(2, "b64"), (2, "b64"), (2, "scale"), (2, "scale")]
FORKS = [
    # what, lens, sources, page, extra, shared, tensors
    ("one sequence to itself", [5], [0], 16, 0, 0, KV8),
    ("a prompt's samples", [70], [0] * 9, 32, 20, 0, [(3, "h64"), (3, "h64")]),
    ("samples of full pages", [64, 128], [0, 1, 0, 1, 1], 32, 0, 0, [(1, "b128")]),
    ("beams change places", [33, 40, 47, 48, 20, 21, 22, 1], [2, 2, 0, 3, 5, 7, 7, 7], 16, 30, 2, KV8),
    ("some end", [100, 17, 0, 64], [3, -1, 0], 16, 0, 0, [(2, "h64")]),
    ("all end", [100, 17, 5], [-1, 99], 16, 0, 1, KV8),
    ("empty sequences", [0, 0, 3], [0, 1, 0, 2, 2], 16, 3, 0, KV8),
    ("pages that are no power of two", [100, 30], [0, 0, 1, 1, 0], 48, 5, 0, [(5, "odd"), (5, "scale")]),
    ("freed pages are taken again", [40, 41, 42, 43], [0, 0, 0, 0], 16, 0, 0, KV8),
    ("many rows", [1 + (i * 37) % 200 for i in range(300)], [(i * 7) % 300 for i in range(3000)], 16, 3000, 3,
     [(1, "scale")]),
    ("many pages", [20000, 30001, 7], [1, 0, 0, 1, 1, 2], 16, 60000, 5, [(1, "scale"), (1, "odd")]),
    ("many tensors", [50, 33], [0, 0, 1, 1], 16, 4, 0, [(1 + i % 3, ["b64", "scale", "h64"][i % 3]) for i in range(250)]),
    ("long rows", [300, 200], [0, 1, 0, 0], 256, 6, 0, [(8, "b128"), (8, "h64"), (8, "scale")]),
]


@pytest.mark.parametrize("case", FORKS, ids=lambda c: c[0].replace(" ", "-"))
def test_fork_matches_the_definition(case):
    _, lens, sources, page, extra, shared, shapes = case
    g = torch.Generator().manual_seed(len(lens) + page)
    table, refs = make_batch(g, lens, page, extra, shared=shared)
    tensors = [t.cuda() for t in make_tensors(g, len(refs), page, shapes)]
    out, out_lens, out_refs, copies = fork(table, lens, refs, sources, page)
    want = moved(tensors, copies, page)
    pool = fa.PagePool(tensors, page)
    dev = cuda(table, lens, refs, sources)
    for _ in range(2):  # the old tables are as they were, and the copies repeat themselves
        got = fa.kv_fork(pool, *dev)
        fa.sync_status()
        assert np.array_equal(got[0].cpu().numpy(), out)
        assert np.array_equal(got[1].cpu().numpy(), out_lens)
        assert np.array_equal(got[2].cpu().numpy(), out_refs)
        for t, w in zip(tensors, want):
            assert np.array_equal(raw(t), w)
        for t, x in zip(dev, (table, lens, refs, sources)):
            assert np.array_equal(t.cpu().numpy(), x)


def test_fork_without_enough_pages():
    """The first rows get what is free, the others -1, and the call reports it."""
    g = torch.Generator().manual_seed(1)
    lens, sources, page = [20, 37], [0, 0, 1, 1, 1, 0], 16
    table, refs = make_batch(g, lens, page, 2)
    tensors = [t.cuda() for t in make_tensors(g, len(refs), page, KV8)]
    out, out_lens, out_refs, copies = fork(table, lens, refs, sources, page)
    assert len(copies) == 2
    want = moved(tensors, copies, page)
    got = fa.kv_fork(fa.PagePool(tensors, page), *cuda(table, lens, refs, sources))
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_NO_PAGES
    assert fa.fa_last_failure()[1:] == [87, 4, 2]  # row 4 is the first without a page, two are
    for t, w in zip(got, (out, out_lens, out_refs)):
        assert np.array_equal(t.cpu().numpy(), w)
    for t, w in zip(tensors, want):
        assert np.array_equal(raw(t), w)
    fa.sync_status()


def test_fork_with_bad_entries_and_lengths():
    """Entries outside the cache count nothing and are passed on; lengths past
    the table and negative ones are cut; entries behind the end are not read."""
    g = torch.Generator().manual_seed(2)
    lens, page = [40, 33, 30], 16
    table, refs = make_batch(g, lens, page, 5, width_more=0)
    table[0, 2] = len(refs) + 7                                  # the page that is being filled
    table[1, 0] = -4
    refs = np.zeros_like(refs)
    for b, n in enumerate(lens):
        for p in table[b, :-(-n // page)]:
            if 0 <= p < len(refs):
                refs[p] += 1
    lens = [40, 10 ** 9, -3]                                     # 48, 0
    refs[table[2, :2]] = 0
    sources = [0, 0, 1, 2, 1]
    tensors = [t.cuda() for t in make_tensors(g, len(refs), page, KV8)]
    out, out_lens, out_refs, copies = fork(table, lens, refs, sources, page)
    want = moved(tensors, copies, page)
    got = fa.kv_fork(fa.PagePool(tensors, page), *cuda(table, lens, refs, sources))
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_BAD_PAGE and fa.fa_last_failure()[1] == 85
    for t, w in zip(got, (out, out_lens, out_refs)):
        assert np.array_equal(t.cpu().numpy(), w)
    for t, w in zip(tensors, want):
        assert np.array_equal(raw(t), w)


COMPACTS = [
    # what, pages, in use, lens, page, tensors
    ("nothing in use", 9, 0.0, [0], 16, KV8),
    ("all in use", 7, 1.0, [33], 16, KV8),
    ("one page", 1, 1.0, [3], 16, [(1, "scale")]),
    ("a few", 40, 0.4, [100, 30, 0, 64], 16, KV8),
    ("most", 300, 0.9, [500, 100], 32, [(2, "h64"), (2, "odd")]),
    ("few of many", 70001, 0.01, [3000], 48, [(1, "scale")]),
    ("half of many", 50000, 0.5, [3000, 9999], 16, [(1, "odd")]),
    ("long rows", 30, 0.5, [1000], 128, [(8, "b128"), (8, "h64"), (8, "scale")]),
]


@pytest.mark.parametrize("case", COMPACTS, ids=lambda c: c[0].replace(" ", "-"))
def test_compact_matches_the_definition(case):
    _, pages, share, lens, page, shapes = case
    g = torch.Generator().manual_seed(pages)
    live = torch.rand(pages, generator=g).numpy() < share
    ids = np.flatnonzero(live).astype(np.int32)
    np.random.RandomState(3).shuffle(ids)
    refs = np.where(live, torch.randint(1, 5, (pages,), generator=g).numpy(), 0).astype(np.int32)
    refs[~live] -= (torch.rand(pages, generator=g).numpy() < 0.1)[~live]  # counts below 0 are free pages too
    used = [-(-n // page) for n in lens]
    lens = [min(n, len(ids) * page) for n in lens]
    table = np.full((len(lens), max(1, max(used)) + 1), -7, dtype=np.int32)
    for b, n in enumerate(lens):
        n = -(-n // page)
        table[b, :n] = np.roll(ids, 13 * b)[:n]
    tensors = [t.cuda() for t in make_tensors(g, pages, page, shapes)]
    out, out_refs, new_ids, copies = compact(table, lens, refs, page)
    want = moved(tensors, copies, page)
    got = fa.kv_compact(fa.PagePool(tensors, page), *cuda(table, lens, refs))
    fa.sync_status()
    for t, w in zip(got, (out, out_refs, new_ids)):
        assert np.array_equal(t.cpu().numpy(), w)
    for t, w in zip(tensors, want):
        assert np.array_equal(raw(t), w)


def test_layers_of_one_tensor_at_odd_places():
    """Layers that are slices of one allocation each: scales whose layers begin 4,
    8 and 12 bytes off a 16-byte boundary, keys 4 bytes off."""
    page, lens, sources = 16, [40, 7, 33], [0, 0, 1, 2, 1, 2]
    g = torch.Generator().manual_seed(11)
    table, refs = make_batch(g, lens, page, 4)
    n = len(refs) | 1                                            # an odd number of pages
    refs = np.concatenate([refs, np.zeros(n - len(refs), dtype=np.int32)])
    scales = torch.randn(4, n, 1, 1, generator=g).cuda()
    keys = torch.randint(0, 1 << 30, (n * page * 16 + 1,), generator=g, dtype=torch.int32).cuda()[1:].view(n, 1, page, 16)
    tensors = [*scales.unbind(0), keys]
    assert {t.data_ptr() % 16 for t in tensors} == {0, 4, 8, 12}
    out, out_lens, out_refs, copies = fork(table, lens, refs, sources, page)
    want = moved(tensors, copies, page)
    pool = fa.PagePool(tensors, page)
    got = fa.kv_fork(pool, *cuda(table, lens, refs, sources))
    fa.sync_status()
    for t, w in zip([*got, *tensors], [out, out_lens, out_refs, *want]):
        assert np.array_equal(raw(t) if t.dim() > 2 else t.cpu().numpy(), w)
    gone = out_refs.copy()
    kept = out.copy()
    for b in (0, 1):                                             # two rows end
        for p in kept[b, :-(-out_lens[b] // page)]:
            gone[p] -= 1
        out_lens[b] = 0
    out, out_refs, new_ids, copies = compact(kept, out_lens, gone, page)
    want = moved(tensors, copies, page)
    got = fa.kv_compact(pool, *cuda(kept, out_lens, gone))
    fa.sync_status()
    for t, w in zip([*got, *tensors], [out, out_refs, new_ids, *want]):
        assert np.array_equal(raw(t) if t.dim() > 2 else t.cpu().numpy(), w)


def test_compact_reports_entries_of_free_pages():
    g = torch.Generator().manual_seed(4)
    tensors = [t.cuda() for t in make_tensors(g, 6, 16, KV8)]
    table, lens, refs = np.array([[5, 2, 9]], dtype=np.int32), [40], np.array([0, 1, 0, 0, 0, 1], dtype=np.int32)
    got = fa.kv_compact(fa.PagePool(tensors, 16), *cuda(table, lens, refs))
    with pytest.raises(fa.FAError) as e:
        fa.sync_status()
    assert e.value.status == fa.FA_ERR_BAD_PAGE and fa.fa_last_failure()[1:3] == [86, 0]
    assert got[0].cpu().tolist() == [[0, 2, 9]]
    assert got[1].cpu().tolist() == [1, 1, 0, 0, 0, 0]


def test_outputs_workspaces_and_streams():
    """Given outputs with a row stride, given workspaces with a guard behind
    them, two streams at once, and a captured call whose inputs change."""
    g = torch.Generator().manual_seed(6)
    lens, page = [100, 37, 64, 5], 16
    table, refs = make_batch(g, lens, page, 12)
    orders = [[0, 0, 1, 1, 2], [3, 3, 3, 0, 1], [2, 1, 0, 3, 3]]
    tensors = make_tensors(g, len(refs), page, KV8)
    width = table.shape[1]
    need = fa.fa_kv_fork_workspace_bytes(4, 5) // 4
    sets = []
    for _ in orders:
        dev = [t.clone().cuda() for t in tensors]
        wide = torch.full((5, width + 3), 77, dtype=torch.int32, device="cuda")
        ws = torch.full((need + 8,), 99, dtype=torch.int32, device="cuda")
        out = (wide[:, 1:1 + width], *(torch.empty(n, dtype=torch.int32, device="cuda") for n in (5, len(refs))))
        sets.append((dev, fa.PagePool(dev, page), wide, ws, out, torch.cuda.Stream()))
    inputs = [cuda(table, lens, refs, o) for o in orders]
    torch.cuda.synchronize()
    for s, x in zip(sets, inputs):
        with torch.cuda.stream(s[5]):
            fa.kv_fork(s[1], *x, workspace=s[3][:need], out=s[4])
    torch.cuda.synchronize()
    fa.sync_status()

    def verify(s, order):
        out, out_lens, out_refs, copies = fork(table, lens, refs, order, page)
        for t, w in zip(s[4], (out, out_lens, out_refs)):
            assert np.array_equal(t.cpu().numpy(), w)
        for t, w in zip(s[0], moved(tensors, copies, page)):
            assert np.array_equal(raw(t), w)
        assert torch.all(s[2][:, 0] == 77) and torch.all(s[2][:, 1 + width:] == 77)
        assert torch.all(s[3][need:] == 99)

    for s, o in zip(sets, orders):
        verify(s, o)
    # one captured call, its sources changed between replays
    s = sets[0]
    x = inputs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv_fork(s[1], *x, out=s[4])
    for o in orders:
        for t, fresh in zip(s[0], tensors):
            t.copy_(fresh)
        x[3].copy_(torch.tensor(o, dtype=torch.int32))
        graph.replay()
        fa.sync_status()
        verify(s, o)


@pytest.mark.parametrize("fp8", [True, False])
def test_a_run_of_prompts_samples_beams_and_compaction(fp8):
    """Prompts are appended, become several sequences, each goes on with its own
    tokens, some change places and end, the pages are moved together: at every
    step the attention gives, bit for bit, what it gives over a cache without
    any sharing that was filled with the same tokens."""
    B, Hq, Hkv, d, page, layers = 2, 4, 2, 64, 16, 2
    g = torch.Generator().manual_seed(8)
    turns = fa.rope_turns(d, device="cuda")

    class Store:
        def __init__(self, pages):
            if fp8:
                self.t = [[torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3)
                           for _ in range(2)] + [torch.zeros(pages, Hkv, page // 16, device="cuda") for _ in range(2)]
                          for _ in range(layers)]
            else:
                self.t = [[torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                          for _ in range(layers)]
            self.pool = fa.PagePool([t for layer in self.t for t in layer], page)

        def append(self, layer, k, v, table, lens, n=None):
            call = fa.kv_append_fp8 if fp8 else fa.kv_append
            call(k, v, *self.t[layer], table, lens, n, turns=turns)

        def attend(self, layer, q, table, lens):
            call = fa.forward_paged_fp8 if fp8 else fa.forward_paged
            return call(q, *self.t[layer], table, lens)

    pages, width = 64, 8
    a, b = Store(pages), Store(256)
    refs = np.zeros(pages, dtype=np.int32)
    lens = [37, 48]
    table = np.full((B, width), -1, dtype=np.int32)
    at = 5
    for i, n in enumerate(lens):
        for k in range(-(-n // page)):
            table[i, k] = at
            refs[at] = 1
            at += 3
    plain = np.arange(16 * width, dtype=np.int32).reshape(16, width)   # the other cache: a row's own pages
    tokens = [[torch.randn(2, layers, Hkv, n, d, generator=g).to(torch.bfloat16)] for n in lens]  # by sequence

    def grow(table, refs, lens):
        """Room for one more token a sequence: the program's own part."""
        for i, n in enumerate(lens):
            if n % page == 0:
                p = int(np.flatnonzero(refs == 0)[-1])
                table[i, n // page], refs[p] = p, 1
            lens[i] += 1

    def compare(table, lens, rows):
        q = torch.randn(rows, Hq, 1, d, generator=g).to(torch.bfloat16).cuda()
        for layer in range(layers):
            for r, seq in enumerate(tokens):
                parts = []
                done = 0
                for t in seq:  # in the same pieces
                    done += t.shape[3]
                    kv = t[:, layer].cuda()
                    b.append(layer, kv[0][None], kv[1][None], *cuda(plain[r:r + 1], [done]))
            x = a.attend(layer, q, *cuda(table, lens))
            y = b.attend(layer, q, *cuda(plain[:rows], lens))
            fa.sync_status()
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])

    for layer in range(layers):
        for i, n in enumerate(lens):
            kv = tokens[i][0][:, layer].cuda()
            a.append(layer, kv[0][None], kv[1][None], *cuda(table[i:i + 1], [n]))
    compare(table, lens, B)
    for sources in ([0, 0, 1, 1, 1, 0], [5, 5, 2, 4, 1, 0, 0], [3, 1, 6]):
        new = fa.kv_fork(a.pool, *cuda(table, lens, refs, sources))
        fa.sync_status()
        table, lens, refs = new[0].cpu().numpy(), new[1].cpu().tolist(), new[2].cpu().numpy()
        tokens = [list(tokens[s]) for s in sources]
        compare(table, lens, len(sources))
        for _ in range(12):
            grow(table, refs, lens)
            fresh = torch.randn(len(sources), 2, layers, Hkv, 1, d, generator=g).to(torch.bfloat16)
            for layer in range(layers):
                kv = fresh[:, :, layer].cuda()
                a.append(layer, kv[:, 0], kv[:, 1], *cuda(table, lens))
            for r in range(len(sources)):
                tokens[r].append(fresh[r])
        compare(table, lens, len(sources))
        new = fa.kv_compact(a.pool, *cuda(table, lens, refs))
        fa.sync_status()
        table, refs = new[0].cpu().numpy(), new[1].cpu().numpy()
        assert (refs > 0).sum() == np.flatnonzero(refs > 0).max() + 1
        compare(table, lens, len(sources))
