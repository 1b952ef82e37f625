"""The paged key/value cache in 8 bits, the attention that reads it, and the sharing of its pages: cases, plain forms and
exact values.

A cache in E4M3 holds twice the keys of a bf16 one in the same memory and halves what a decoding step reads.  Every 16
tokens of a key head have one scale of their own, for keys and for values: a stored value is scale * E4M3.  A serving
step rotates q and k, rounds k and v into the cache and attends over it; a batch behind one prompt reads the prompt's
pages once for all.  Where one sequence becomes several (samples of a prompt, beams) they share its full pages, each
with a count of the sequences that use it, and get a copy of the page that is still being filled; what nobody uses is
free, and the pages in use can be moved together.

Layouts: q [B, Hq, Nq, d]; pages [pages, Hkv, page, d], scales [pages, Hkv, page / 16]; block_table[b, p // page] is the
page of position p of sequence b.  With L keys in the cache (the new tokens among them) query i sits at position
L - Nq + i and sees the keys up to it.
"""

import math

import torch

own = False

TWO_PI = 2.0 * math.pi
TOKENS = 16            # tokens of a scale
LARGEST = 448.0        # of E4M3
LOWEST = -32           # a scale is at least 2^-32


# ------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step of 8 sequences: q rotated, one k and v row a sequence into the cache
        dict(name="append8_step", op="append", B=8, Hq=32, Hkv=8, N=1, d=128, page=64, Lmin=500, Lmax=8192, rot=128,
             layout="half", scaling="none", with_q=True),
        # prompts of four sequences of different lengths into an empty cache
        dict(name="append8_prompts", op="append", B=4, Hq=16, Hkv=16, N=8192, d=128, page=128, Lmin=2048, Lmax=8192,
             rot=128, layout="half", scaling="parts", with_q=True),
        # one sequence answering: latency
        dict(name="paged8_step_one", op="paged", B=1, Hq=32, Hkv=8, Nq=1, d=128, page=16, Lmin=1000, Lmax=1000),
        # a serving batch of very different lengths
        dict(name="paged8_step_ragged", op="paged", B=32, Hq=32, Hkv=4, Nq=1, d=128, page=64, Lmin=100, Lmax=16384),
        # the decoding benchmark's cache, 8 sequences x 32 heads x 32768 keys
        dict(name="paged8_step_long", op="paged", B=8, Hq=32, Hkv=32, Nq=1, d=128, page=128, Lmin=32768, Lmax=32768),
        # a chunk of two prompts against what is cached of them
        dict(name="paged8_chunk", op="paged", B=2, Hq=32, Hkv=8, Nq=1000, d=128, page=64, Lmin=9001, Lmax=16384),
        # drafted tokens of a batch behind one prompt, an odd number of heads a group, small heads
        dict(name="prefix8_drafts", op="prefix", B=24, Hq=20, Hkv=4, Nq=4, d=64, page=16, P=8208, Lmin=4, Lmax=777),
        # many samples of one long document
        dict(name="prefix8_batch", op="prefix", B=256, Hq=64, Hkv=8, Nq=1, d=128, page=64, P=32768, Lmin=1, Lmax=1024),
        # beams of four requests change places between two tokens, a cache in 8 bits
        dict(name="fork_beams", op="fork", B=16, rows=16, layers=16, Hkv=4, d=128, page=16, Lmin=100, Lmax=700,
             fp8=True, beams=4, spare=200),
        # sixty-four samples of each of two prompts, bf16, pages of 128 tokens
        dict(name="fork_samples", op="fork", B=2, rows=128, layers=8, Hkv=8, d=128, page=128, Lmin=1001, Lmax=4000,
             fp8=False, beams=0, spare=130),
        # a small cache after a few sequences have ended
        dict(name="compact_small", op="compact", B=5, layers=4, Hkv=2, d=64, page=32, Lmin=10, Lmax=900, fp8=False,
             pages=200),
        # half of a large cache is free, in pieces
        dict(name="compact_large", op="compact", B=40, layers=8, Hkv=8, d=128, page=64, Lmin=300, Lmax=2000, fp8=True,
             pages=1200),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "prefix", "fork", "compact"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op in ("fork", "compact"):
        Hkv, layers = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 16)
        values = layers * Hkv * page * d  # of a page id
        most = max(8, min(4000, 2 ** 28 // values))  # pages
        if op == "compact":
            pages = _log(rng, 8, most)
            B = rng.randint(1, 40)
            Lmax = max(1, min(2000, pages * page // (2 * B)))
            return dict(op=op, B=B, layers=layers, Hkv=Hkv, d=d, page=page, Lmin=max(1, Lmax // rng.randint(1, 20)),
                        Lmax=Lmax, fp8=rng.random() < 0.5, pages=pages + B)
        beams = rng.choice([0, 2, 4, 5])
        B = beams * rng.randint(1, 8) if beams else rng.randint(1, 16)
        rows = B if beams else _log(rng, B, 128)
        Lmax = max(1, min(4000, (most - rows) * page // (B + 1)))
        return dict(op=op, B=B, rows=rows, layers=layers, Hkv=Hkv, d=d, page=page, Lmin=max(1, Lmax // 8), Lmax=Lmax,
                    fp8=rng.random() < 0.5, beams=beams, spare=rows + rng.randint(0, 100))
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        N = _log(rng, 1, 4096)
        return dict(op=op, B=rng.randint(1, 8), Hq=G * Hkv, Hkv=Hkv, N=N, d=d, page=page, Lmin=N,
                    Lmax=N + _log(rng, 1, 4096), rot=rng.choice([16, 32, 64, d]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                    with_q=rng.random() < 0.7)
    if op == "paged":
        Nq = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 1000)])
        B = _log(rng, 1, 64)
        L = _log(rng, 64, 32768)
        while B * Hkv * L * d > 2 ** 28 or B * Hkv * G * Nq * L > 2 ** 29:
            L = (L + 1) // 2
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, Nq=Nq, d=d, page=page, Lmin=Nq + rng.randint(0, 64),
                    Lmax=max(L, Nq + 64))
    Nq = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 200)])
    B = _log(rng, 2, 256)
    while B * Hkv * G * Nq > 16384:
        if B > 1:
            B = (B + 1) // 2
        else:  # one sequence's rows alone
            Nq = (Nq + 1) // 2
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, Nq=Nq, d=d, page=page, P=page * _log(rng, 4, 32768 // page), Lmin=Nq,
                Lmax=Nq + _log(rng, 1, 1024))


def _spread(case):
    """The sequences' lengths in the cache (behind the prefix, where there is one): spread evenly over their logarithm,
    in an order that is not sorted.  They follow from the case alone."""
    B, lo, hi = case["B"], case["Lmin"], case["Lmax"]
    steps = [i / max(1, B - 1) if B > 1 else 1.0 for i in range(B)]
    lens = [int(round(lo * (hi / lo) ** s)) for s in steps]
    return [lens[(i * 7 + 3) % B] for i in range(B)] if B % 7 else lens


def _new_tokens(case):
    """How many tokens each sequence appends: all N of a step or chunk; a whole prompt where the cache was empty."""
    return [min(case["N"], n) for n in _spread(case)]


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits (base 10000)."""
    rot, kind = case["rot"], case["scaling"]
    base, factor, length = 10000.0, 8.0, 8192.0
    if kind == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if kind == "linear":
        f = f / factor
    if kind == "parts":  # pairs that turn often within the trained length keep their frequency, slow ones are stretched
        ramp = ((f * length / TWO_PI - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * ramp + f / factor * (1.0 - ramp)
    return f


def _amplitude(case):
    return 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "parts" else 1.0


def _fitting(largest):
    """The smallest power of two, at least 2^LOWEST, that brings `largest` to at most 448 = 7/8 2^9."""
    m, e = torch.frexp(largest)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=LOWEST)
    return ((e + 127) << 23).view(torch.float32)


def _stored(x):
    """A cache that holds x [pages, Hkv, page, d]: E4M3 values and the scales of each 16 tokens of a head."""
    blocks = x.unflatten(2, (-1, TOKENS))
    scale = _fitting(blocks.abs().amax((-2, -1)).float())
    return (blocks.float() / scale[..., None, None]).to(torch.float8_e4m3fn).flatten(2, 3), scale


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case=case)
    if case["op"] in ("fork", "compact"):
        return _prepare_pages(case, s, g, dev)
    f = _frequencies(case) if "rot" in case else None
    if f is not None:
        s["freq"] = f.to(dev)
        s["turns"] = (f / TWO_PI * 2.0 ** 64).round().to(torch.int64).to(dev)  # 2^-64 turns per position
        s["amplitude"] = _amplitude(case)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    P = case.get("P", 0)
    lens = [n + P for n in _spread(case)]
    shared = P // page
    used = [(n + page - 1) // page - shared for n in lens]
    order = torch.randperm(shared + sum(used), generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(shared + n for n in used)), -1, dtype=torch.int32, device=dev)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(used):
        table[b, shared:shared + n] = order[at:at + n]
        at += n
    s["block_table"] = table
    s["seqlens_k"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # heads differ in size, as a model's do
    size = torch.exp2(torch.linspace(-1.0, 1.0, Hkv, device=dev)).to(torch.bfloat16)[:, None, None]
    s["k_pages"], s["k_scales"] = _stored(normal(at, Hkv, page, d) * size)
    s["v_pages"], s["v_scales"] = _stored(normal(at, Hkv, page, d) * size.flip(0))
    if case["op"] == "append":
        N, Hq = case["N"], case["Hq"]
        fused = normal(B, N, Hq + 2 * Hkv, d)
        fused[:, :, Hq:Hq + Hkv] *= size[:, 0] * 2.0
        s["q"] = fused[:, :, :Hq].transpose(1, 2)
        s["k"] = fused[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["v"] = fused[:, :, Hq + Hkv:].transpose(1, 2)
        s["seqlens_q"] = torch.tensor(_new_tokens(case), dtype=torch.int32, device=dev)
        s["q_out"] = torch.zeros(B, Hq, N, d, dtype=torch.bfloat16, device=dev) if case["with_q"] else None
        return s
    s["q"] = normal(B, case["Hq"], case["Nq"], d) * 1.5
    s["prefix_table"] = table[0, :shared].contiguous()
    s["scale"] = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    return s


def _prepare_pages(case, s, g, dev):
    """A cache of several layers whose pages lie in any order; the page ids are the same in every layer."""
    B, page, fork = case["B"], case["page"], case["op"] == "fork"
    lens = _spread(case)
    used = [(n + page - 1) // page for n in lens]
    pages = sum(used) + case["spare"] if fork else max(case["pages"], sum(used))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device=dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    if fork and case["beams"]:  # the beams of a request have its prompt's first pages in common
        beams = case["beams"]
        for b in range(B):
            n = min(used[b], used[b - b % beams]) // 2
            table[b, :n] = table[b - b % beams, :n]
    s["block_table"] = table
    s["seqlens_k"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), (table >= 0).flatten().to(torch.int32))
    s["refs"] = refs
    shape = (case["layers"], pages, case["Hkv"], page, case["d"])
    names = []
    for name in ("k_pages", "v_pages"):
        x = torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)
        if case["fp8"]:
            x, scale = _stored(x.flatten(0, 1))
            s[name], s[name + "_scales"] = x.view(shape), scale.view(*shape[:3], page // TOKENS)
            names += [name, name + "_scales"]
        else:
            s[name] = x
            names += [name]
    s["names"] = names
    if fork:
        rows, beams = case["rows"], case["beams"]
        i = torch.arange(rows, device=dev)
        if beams:  # any beam of the same request, some twice, some not at all
            sources = i - i % beams + torch.randint(0, beams, (rows,), generator=g, device=dev)
        else:
            sources = i * B // rows
        s["sources"] = sources.to(torch.int32)
    return s


# --------------------------------------------------------------------------------------------------- the plain forms

def _turn(x, positions, s):
    """x [B, H, N, d] rotated by the angles positions [B, N] x frequencies; 32 bits, the angles in 64."""
    case = s["case"]
    rot = 2 * s["freq"].numel()
    angle = positions.to(torch.float64)[:, None, :, None] * s["freq"]
    c = (angle.cos() * s["amplitude"]).float()
    n = (angle.sin() * s["amplitude"]).float()
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([head, rest], -1)


def _write(s, pages, scales, x, largest):
    """x [B, H, N, d] in 32 bits, the new tokens, into their 16 tokens' cells: the scale that the largest of |largest|
    asks for, or the one that the 16 tokens have if they hold older tokens and it is larger."""
    case, table, page = s["case"], s["block_table"], s["case"]["page"]
    B, H, N, d = x.shape
    lk = s["seqlens_k"].long()
    first = lk - s["seqlens_q"].long()
    cells = torch.arange((N + TOKENS - 2) // TOKENS + 1, device=x.device)
    cell = torch.minimum(first[:, None] // TOKENS + cells, (lk[:, None] - 1) // TOKENS)  # the last one again behind it
    pos = cell[..., None] * TOKENS + torch.arange(TOKENS, device=x.device)           # [B, cells, 16]
    new, old = (pos >= first[:, None, None]) & (pos < lk[:, None, None]), pos < first[:, None, None]
    t = (pos - first[:, None, None]).clamp(0, N - 1).flatten(1)[:, None, :, None].expand(B, H, -1, d)
    value = x.gather(2, t).unflatten(2, (-1, TOKENS))                                # [B, H, cells, 16, d]
    big = largest.abs().amax(-1).float().gather(2, t[..., 0]).unflatten(2, (-1, TOKENS))
    big = torch.where(new[:, None], big, torch.zeros_like(big)).amax(-1)             # [B, H, cells]
    b = torch.arange(B, device=x.device)[:, None]
    at, inside = table.long()[b, cell * TOKENS // page], cell * TOKENS % page // TOKENS
    heads = torch.arange(H, device=x.device)[:, None]
    before = scales[at[:, None], heads, inside[:, None]]
    scale = _fitting(big)
    scale = torch.where(old.any(-1)[:, None], torch.maximum(scale, before), scale)
    codes = pages.view(torch.uint8).unflatten(2, (-1, TOKENS))                       # [pages, H, page / 16, 16, d]
    had = codes[at[:, None], heads, inside[:, None]]
    again = had.view(torch.float8_e4m3fn).float() * (before / scale)[..., None, None]
    now = torch.where(new[:, None, ..., None], value / scale[..., None, None], again).to(torch.float8_e4m3fn)
    keep = ~(new | old)[:, None, ..., None]
    codes[at[:, None], heads, inside[:, None]] = torch.where(keep, had, now.view(torch.uint8))
    scales[at[:, None], heads, inside[:, None]] = scale


def _append(s):
    case = s["case"]
    lq, lk = s["seqlens_q"].long()[:, None], s["seqlens_k"].long()[:, None]
    t = torch.arange(case["N"], device=s["k"].device)[None]
    place = lk - lq + t
    if s["q_out"] is not None:
        turned = _turn(s["q"], place, s).to(torch.bfloat16)
        s["q_out"].copy_(torch.where((t < lq)[:, None, :, None], turned, s["q_out"]))
    # a rotated pair's values are at most sqrt(2) times the pair's larger one
    _write(s, s["k_pages"], s["k_scales"], _turn(s["k"], place, s), s["k"].float() * (math.sqrt(2.0) * s["amplitude"]))
    _write(s, s["v_pages"], s["v_scales"], s["v"].float(), s["v"])


def _keys(pages, scales, table):
    """[B, Hkv, positions, d] in 32 bits: the pages that the tables name, one behind the other."""
    at = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float().unflatten(3, (-1, TOKENS))
    return (x * scales[at][..., None, None]).flatten(3, 4).transpose(1, 2).flatten(2, 3)


def _partial(q, k, v, seen, scale):
    """Row maximum, sum and unnormalised output over the keys that `seen` allows; 32 bits."""
    z = q @ k.transpose(-1, -2) * scale
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return m, p.sum(-1, keepdim=True), p @ v


def _join(parts, shape):
    m = torch.stack([p[0] for p in parts]).amax(0)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    total = sum(torch.exp(p[0] - base) * p[1] for p in parts)
    out = sum(torch.exp(p[0] - base) * p[2] for p in parts)
    o = torch.where(total > 0, out / total, torch.zeros_like(out)).reshape(shape)
    lse = torch.where(total > 0, m + total.log(), torch.full_like(m, -math.inf)).reshape(shape[:-1])
    return o.to(torch.bfloat16), lse


def _attend(s):
    case, q = s["case"], s["q"]
    B, Hq, Nq, d = q.shape
    Hkv, P, page = case["Hkv"], case.get("P", 0), case["page"]
    G = Hq // Hkv
    rows = q.float().reshape(B, Hkv, G * Nq, d)
    last = (s["seqlens_k"].long()[:, None] - Nq + torch.arange(Nq, device=q.device)).repeat(1, G)[:, None, :, None]
    table = s["block_table"][:, P // page:]
    k, v = _keys(s["k_pages"], s["k_scales"], table), _keys(s["v_pages"], s["v_scales"], table)
    at = P + torch.arange(k.shape[2], device=q.device)
    parts = [_partial(rows, k, v, at <= last, s["scale"])]
    if P:  # every sequence's rows against one copy of the prefix
        k = _keys(s["k_pages"], s["k_scales"], s["prefix_table"][None])[0]
        v = _keys(s["v_pages"], s["v_scales"], s["prefix_table"][None])[0]
        all_rows = rows.transpose(0, 1).reshape(Hkv, B * G * Nq, d)
        ends = last.expand(B, Hkv, G * Nq, 1).transpose(0, 1).reshape(Hkv, B * G * Nq, 1)
        first = _partial(all_rows, k, v, torch.arange(P, device=q.device) <= ends, s["scale"])
        parts.append([x.reshape(Hkv, B, G * Nq, -1).transpose(0, 1) for x in first])
    return _join(parts, (B, Hq, Nq, d))


def _counts(pages, table, used):
    """How often each page is named by the first used[b] entries of the rows of the table."""
    named = torch.arange(table.shape[1], device=table.device) < used[:, None]
    return torch.zeros(pages, dtype=torch.int32, device=table.device).index_add_(
        0, torch.where(named, table, torch.zeros_like(table)).flatten().long(), named.flatten().to(torch.int32))


def _bytes(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _fork(s):
    """Row i continues sequence sources[i]: its full pages are shared; the page that is being filled goes to the first
    row that continues the sequence, and the others have a copy, in the free pages of the lowest ids."""
    page, table, refs = s["case"]["page"], s["block_table"], s["refs"]
    lens, source = s["seqlens_k"].long(), s["sources"].long()
    rows, n = torch.arange(source.numel(), device=refs.device), lens[source]
    used = (n + page - 1) // page
    out = torch.where(torch.arange(table.shape[1], device=refs.device) < used[:, None], table[source],
                      torch.full_like(table[source], -1))
    first = torch.full_like(lens, source.numel()).scatter_reduce_(0, source, rows, "amin")
    copies = (n % page != 0) & (first[source] != rows)  # rows that need a page of their own
    tail = (used - 1).clamp(min=0)
    shared = _counts(refs.numel(), out, used - copies.long())
    left = refs - _counts(refs.numel(), table, (lens + page - 1) // page) + shared
    order = torch.argsort((left != 0).to(torch.int32), stable=True)   # free pages first, by id
    mine = order[(copies.long().cumsum(0) - 1).clamp(min=0)]
    src = torch.where(copies, out[rows, tail].long(), torch.zeros_like(mine))
    dst = torch.where(copies, mine, torch.zeros_like(mine))
    out[rows, tail] = torch.where(copies, mine.to(torch.int32), out[rows, tail])
    left = left.index_add(0, dst, copies.to(torch.int32))
    # the rows without a copy repeat one that is made (page 0 onto itself where there is none)
    one = copies.to(torch.int32).argmax()
    filled = torch.where(copies, n % page, (n % page)[one])
    src, dst = torch.where(copies, src, src[one]), torch.where(copies, dst, dst[one])
    for name in s["names"]:
        x = _bytes(s[name])
        unit = page // x.shape[3]  # tokens of a cell: 1, or 16 of a scale
        have = torch.arange(x.shape[3], device=refs.device) * unit < filled[:, None]
        have = have[None, :, None, :].reshape((1, -1, 1, x.shape[3]) + (1,) * (x.dim() - 4))
        x[:, dst] = torch.where(have, x[:, src], x[:, dst])
    return dict(table=out, seqlens=n.to(torch.int32), refs=left, **{name: s[name] for name in s["names"]})


def _compact(s):
    """The pages in use at or behind the number of pages in use move into the free ones before it, both by id."""
    refs, table, page = s["refs"], s["block_table"], s["case"]["page"]
    live, ids = refs > 0, torch.arange(refs.numel(), device=refs.device)
    count = live.sum()
    away, hole = live & (ids >= count), ~live & (ids < count)
    holes = torch.argsort((~hole).to(torch.int32), stable=True)
    movers = torch.argsort((~away).to(torch.int32), stable=True)
    new_ids = torch.where(away, holes[(away.long().cumsum(0) - 1).clamp(min=0)], ids)
    comes = torch.where(hole, movers[(hole.long().cumsum(0) - 1).clamp(min=0)], ids)  # where a page's content is now
    used = (s["seqlens_k"].long() + page - 1) // page
    named = torch.arange(table.shape[1], device=refs.device) < used[:, None]
    out = torch.where(named, new_ids[table.clamp(min=0).long()].to(torch.int32), table)
    for name in s["names"]:
        x = _bytes(s[name])
        x.copy_(x[:, comes])
    left = torch.where(ids < count, refs[comes], torch.zeros_like(refs))
    return dict(table=out, refs=left, new_ids=torch.where(live, new_ids, torch.full_like(new_ids, -1)).to(torch.int32),
                **{name: s[name] for name in s["names"]})


def run(state):
    s, case = state, state["case"]
    if own:
        import exact_tiled_attention_18_gb300 as fa
        if case["op"] in ("fork", "compact") and "pool" not in s:  # the program's handle of its cache, made once
            s["pool"] = fa.PagePool([s[name][i] for i in range(case["layers"]) for name in s["names"]], case["page"])
        if case["op"] == "fork":
            table, lens, refs = fa.kv_fork(s["pool"], s["block_table"], s["seqlens_k"], s["refs"], s["sources"])
            return dict(table=table, seqlens=lens, refs=refs, **{name: s[name] for name in s["names"]})
        if case["op"] == "compact":
            table, refs, new_ids = fa.kv_compact(s["pool"], s["block_table"], s["seqlens_k"], s["refs"])
            return dict(table=table, refs=refs, new_ids=new_ids, **{name: s[name] for name in s["names"]})
        cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if case["op"] == "append":
            fa.kv_append_fp8(s["k"], s["v"], *cache, s["block_table"], s["seqlens_k"], s["seqlens_q"],
                             turns=s["turns"], layout=case["layout"], amplitude=s["amplitude"],
                             q=s["q"] if case["with_q"] else None, q_out=s["q_out"])
            return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                        q=s["q_out"])
        if case["op"] == "paged":
            o, lse = fa.forward_paged_fp8(s["q"], *cache, s["block_table"], s["seqlens_k"], causal=True,
                                          scale=s["scale"], o_dtype=torch.bfloat16)
            return dict(o=o, lse=lse)
        o, lse = fa.forward_shared_prefix_fp8(s["q"], *cache, s["prefix_table"], case["P"], s["block_table"],
                                              s["seqlens_k"], causal=True, scale=s["scale"], o_dtype=torch.bfloat16)
        return dict(o=o, lse=lse)
    if case["op"] == "fork":
        return _fork(s)
    if case["op"] == "compact":
        return _compact(s)
    if case["op"] == "append":
        _append(s)
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                    q=s["q_out"])
    o, lse = _attend(s)
    return dict(o=o, lse=lse)


# --------------------------------------------------------------------------------------------- what they cannot avoid

def work(case):
    d, B = case["d"], case["B"]
    lens = _spread(case)
    if case["op"] in ("fork", "compact"):
        page, layers, Hkv = case["page"], case["layers"], case["Hkv"]
        token = 2 * layers * Hkv * (d + 4 / TOKENS if case["fp8"] else 2 * d)  # bytes of a token, keys and values
        used = [(n + page - 1) // page for n in lens]
        width = max(used) + 1
        if case["op"] == "fork":
            rows, pages = case["rows"], sum(used) + case["spare"]
            # of beams that are drawn with replacement a share of (1 - 1/k)^k is not drawn, as many rows need a copy
            k = case["beams"]
            new = rows * (1 - 1 / k) ** k if k else rows - B
            tail = sum(n % page for n in lens) / B
            return {"bytes": 2 * token * tail * new + 4 * (2 * pages + (B + rows) * width + B + 3 * rows), "flops": 0}
        pages = max(case["pages"], sum(used))
        moved = sum(used) * (1 - sum(used) / pages)  # of pages in any order
        return {"bytes": 2 * token * page * moved + 4 * (3 * pages + 2 * B * width + B), "flops": 0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "append":
        tokens = sum(_new_tokens(case))
        turned = Hkv + (Hq if case["with_q"] else 0)
        stored = 2 * tokens * Hkv * (d + 4 / TOKENS)
        return {"bytes": 2 * tokens * (turned + Hkv) * d + (2 * tokens * Hq * d if case["with_q"] else 0) + stored,
                "flops": tokens * (3 * turned * case["rot"] + 4 * Hkv * d)}
    P, Nq = case.get("P", 0), case["Nq"]
    pairs = sum((P + n) * Nq - Nq * (Nq - 1) // 2 for n in lens)
    rows = B * Hq * Nq
    return {"bytes": 2 * Hkv * (d + 4 / TOKENS) * (P + sum(lens)) + rows * (2 * d + 2 * d + 4),
            "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------------------------------------ the exact values

def _exact_turn(x, positions, case):
    """The rotation of [heads, tokens, d] as a product of complex numbers in 64 bits."""
    f = _frequencies(case).to(x.device)
    rot = 2 * f.numel()
    theta = positions.double().unsqueeze(-1) * f
    unit = torch.polar(torch.full_like(theta, _amplitude(case)), theta)
    y = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * unit
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """The nearest value of E4M3 (ties to even), in 64 bits: steps of 2^-3 of a value's power of two, 2^-9 at least."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-LARGEST, LARGEST)


def _exact_append(s, case):
    page = case["page"]
    out = dict(q=s["q_out"].double() if case["with_q"] else None)
    for name in ("k", "v"):
        out[name + "_pages"] = s[name + "_pages"].to(torch.float32).double()
        out[name + "_scales"] = s[name + "_scales"].double()
    for b, (n, total) in enumerate(zip(s["seqlens_q"].tolist(), s["seqlens_k"].tolist())):
        pos = torch.arange(total - n, total, device=s["k"].device)
        if case["with_q"]:
            out["q"][b, :, :n] = _exact_turn(s["q"][b, :, :n], pos, case)
        turned = dict(k=_exact_turn(s["k"][b, :, :n], pos, case), v=s["v"][b, :, :n].double())
        bound = dict(k=math.sqrt(2.0) * _amplitude(case), v=1.0)
        begin, end = (total - n) // TOKENS * TOKENS, (total + TOKENS - 1) // TOKENS * TOKENS
        older = total - n - begin  # tokens of the first cell that were there
        at = torch.arange(begin, end, TOKENS, device=pos.device)
        where = s["block_table"][b].long()[torch.div(at, page, rounding_mode="floor")]
        inside = torch.div(at.remainder(page), TOKENS, rounding_mode="floor")
        for name in ("k", "v"):
            cells = out[name + "_pages"].unflatten(2, (-1, TOKENS))
            H, d = cells.shape[1], cells.shape[4]
            fresh = torch.zeros(H, end - begin, d, dtype=torch.float64, device=pos.device)
            big = torch.zeros(H, end - begin, dtype=torch.float64, device=pos.device)
            fresh[:, older:older + n] = turned[name]
            big[:, older:older + n] = s[name][b, :, :n].double().abs().amax(-1) * bound[name]
            m, e = torch.frexp((big.unflatten(1, (-1, TOKENS)).amax(-1) / LARGEST).clamp(min=2.0 ** LOWEST))
            scale = _power(e - (m == 0.5).to(e.dtype))
            had = cells[where, :, inside].transpose(0, 1)
            before = out[name + "_scales"][where, :, inside].transpose(0, 1)
            if older:
                scale[:, 0] = torch.maximum(scale[:, 0], before[:, 0])
            now = _exact_e4m3(fresh.unflatten(1, (-1, TOKENS)) / scale[..., None, None])
            now[:, 0, :older] = _exact_e4m3(had[:, 0, :older] * (before[:, 0] / scale[:, 0])[:, None, None])
            rest = end - total  # rows behind the last token stay as they are
            if rest:
                now[:, -1, TOKENS - rest:] = had[:, -1, TOKENS - rest:]
            cells[where, :, inside] = now.transpose(0, 1)
            out[name + "_scales"][where, :, inside] = scale.transpose(0, 1)
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):  # whole numbers and copies: the plain form's are exact
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s, case)
    page = case["page"]
    B, Hq, Nq, d = s["q"].shape
    Hkv = case["Hkv"]
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(B, Hq, Nq, dtype=torch.float64, device=s["q"].device)

    def held(name, named, h, total):
        x = s[name + "_pages"].view(torch.uint8)[named, h].view(torch.float8_e4m3fn).to(torch.float32).double()
        scale = s[name + "_scales"][named, h].double().repeat_interleave(TOKENS, 1)
        return (x * scale[..., None]).reshape(-1, d)[:total]

    for b, total in enumerate(s["seqlens_k"].tolist()):
        named = s["block_table"][b, :(total + page - 1) // page].long()
        sees = torch.arange(total, device=o.device)[None, :] <= torch.arange(total - Nq, total, device=o.device)[:, None]
        for h in range(Hkv):
            group = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            key, value = held("k", named, h, total), held("v", named, h, total)
            logits = torch.einsum("gnd,ld->gnl", s["q"][b, group].double(), key) * s["scale"]
            logits = logits.masked_fill(~sees, -math.inf)
            lse[b, group] = torch.logsumexp(logits, -1)
            o[b, group] = torch.einsum("gnl,ld->gnd", torch.exp(logits - lse[b, group].unsqueeze(-1)), value)
    return dict(o=o, lse=lse)
