"""Rotary positions, the paged key/value cache and the attention that reads it: cases, plain forms and exact values.

A serving step takes fresh projections, rotates q and k by their positions, appends k and v to a cache held in pages,
and attends over it; a batch that starts with one common prompt attends over the prompt's pages once for all.  Training
rotates q and k before the forward pass and rotates the gradients back after the backward pass.

Layouts: q [B, Hq, Nq, d]; pages [pages, Hkv, page, d]; block_table[b, p // page] is the page of position p of sequence
b.  With L keys in the cache (the new tokens among them) query i sits at position L - Nq + i and sees the keys up to it.
"""

import math

import torch

own = False

TWO_PI = 2.0 * math.pi


# ------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # q of a training step (4 x 16 heads x 8192 tokens), rotated out of the fused projection's layout
        dict(name="rope_training_q", op="rope", B=4, H=16, N=8192, d=128, rot=128, layout="half", scaling="none",
             dtype="bf16", out="bf16", inverse=False, far=0, packed=False),
        # fp32 gradient of a long-context sequence of packed documents, rotated back, by-parts scaling
        dict(name="rope_gradient_long", op="rope", B=1, H=32, N=16384, d=128, rot=128, layout="interleaved",
             scaling="parts", dtype="fp32", out="bf16", inverse=True, far=0, packed=True),
        # one token of each of 8 sequences far into a long context, a quarter of each head rotated
        dict(name="rope_step_partial", op="rope", B=8, H=32, N=1, d=64, rot=16, layout="half", scaling="ntk",
             dtype="bf16", out="bf16", inverse=False, far=1000000, packed=False),
        # a decoding step of 8 sequences: q rotated, one k and v row a sequence into the cache
        dict(name="append_step", op="append", B=8, Hq=32, Hkv=8, N=1, d=128, page=64, Lmin=500, Lmax=8192, rot=128,
             layout="half", scaling="none", with_q=True),
        # prompts of four sequences of different lengths into an empty cache
        dict(name="append_prompts", op="append", B=4, Hq=16, Hkv=16, N=8192, d=128, page=128, Lmin=2048, Lmax=8192,
             rot=128, layout="half", scaling="parts", with_q=True),
        # one sequence answering: latency
        dict(name="paged_step_one", op="paged", B=1, Hq=32, Hkv=8, Nq=1, d=128, page=16, Lmin=1000, Lmax=1000),
        # a serving batch of very different lengths
        dict(name="paged_step_ragged", op="paged", B=32, Hq=32, Hkv=4, Nq=1, d=128, page=64, Lmin=100, Lmax=16384),
        # the decoding benchmark's cache, 8 sequences x 32 heads x 32768 keys
        dict(name="paged_step_long", op="paged", B=8, Hq=32, Hkv=32, Nq=1, d=128, page=128, Lmin=32768, Lmax=32768),
        # a chunk of two prompts against what is cached of them
        dict(name="paged_chunk", op="paged", B=2, Hq=32, Hkv=8, Nq=1000, d=128, page=64, Lmin=9001, Lmax=16384),
        # a few conversations behind one system prompt
        dict(name="prefix_step", op="prefix", B=16, Hq=32, Hkv=8, Nq=1, d=128, page=64, P=4096, Lmin=1, Lmax=300),
        # many samples of one long document
        dict(name="prefix_batch", op="prefix", B=256, Hq=64, Hkv=8, Nq=1, d=128, page=64, P=32768, Lmin=1, Lmax=1024),
        # drafted tokens of a batch behind one prompt, an odd number of heads a group, small heads
        dict(name="prefix_drafts", op="prefix", B=24, Hq=20, Hkv=4, Nq=4, d=64, page=16, P=8208, Lmin=4, Lmax=777),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "paged", "paged", "prefix"])
    d = rng.choice([64, 128])
    heads = dict(rot=rng.choice([16, 32, 64, d]), layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "ntk", "parts"]))
    if op == "rope":
        B, H, N = rng.randint(1, 8), rng.randint(1, 32), _log(rng, 1, 16384)
        while B * H * N * d > 4 * 16 * 8192 * 128:
            N = (N + 1) // 2
        inverse = rng.random() < 0.5
        return dict(op=op, B=B, H=H, N=N, d=d, **heads, dtype=rng.choice(["bf16", "fp32"]),
                    out=rng.choice(["bf16", "fp32"]), inverse=inverse, far=rng.choice([0, _log(rng, 1, 1000000)]),
                    packed=rng.random() < 0.3)
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        N = _log(rng, 1, 4096)
        B = rng.randint(1, 8)
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, N=N, d=d, page=page, Lmin=N, Lmax=N + _log(rng, 1, 4096),
                    **heads, with_q=rng.random() < 0.7)
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
    P = page * _log(rng, 4, 32768 // page)
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, Nq=Nq, d=d, page=page, P=P, Lmin=Nq,
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


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    s = dict(case=case)
    if "rot" in case:
        f = _frequencies(case)
        s["freq"] = f.to(dev)
        s["turns"] = (f / TWO_PI * 2.0 ** 64).round().to(torch.int64).to(dev)  # 2^-64 turns per position
        s["amplitude"] = _amplitude(case)
    if case["op"] == "rope":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["inverse"]:  # a gradient, in the attention's own layout
            s["x"] = normal(B, H, N, d, dtype=t) * 0.01
        else:  # the q part of a fused projection [B, N, (H + 2) * d]
            s["x"] = normal(B, N, H + 2, d, dtype=t)[:, :, :H].transpose(1, 2)
        if case["packed"]:  # documents packed into each row: positions start again at random places
            starts = torch.rand(B, N, generator=g, device=dev) < 8.0 / N
            starts[:, 0] = True
            i = torch.arange(N, device=dev).expand(B, N)
            first = torch.where(starts, i, torch.zeros_like(i)).cummax(1).values
            s["positions"] = (i - first + case["far"]).to(torch.int32)
        else:
            off = torch.randint(0, 1000, (B, 1), generator=g, device=dev) if case["far"] else torch.zeros(
                B, 1, device=dev, dtype=torch.int64)
            s["positions"] = (torch.arange(N, device=dev) + case["far"] + off).to(torch.int32)
        return s

    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    P = case.get("P", 0)
    lens = [n + P for n in _spread(case)]
    shared = P // page
    used = [(n + page - 1) // page - shared for n in lens]
    order = torch.randperm(shared + sum(used), generator=g, device=dev).to(torch.int32)
    width = max(shared + n for n in used)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(used):
        table[b, shared:shared + n] = order[at:at + n]
        at += n
    s["block_table"] = table
    s["seqlens_k"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_pages"] = normal(at, Hkv, page, d)
    s["v_pages"] = normal(at, Hkv, page, d)
    if case["op"] == "append":
        N, Hq = case["N"], case["Hq"]
        fused = normal(B, N, Hq + 2 * Hkv, d)
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


# --------------------------------------------------------------------------------------------------- the plain forms

def _turn(x, positions, s, sign):
    """x [B, H, N, d] rotated by the angles positions [B, N] x frequencies; 32 bits, the angles in 64."""
    case = s["case"]
    rot = 2 * s["freq"].numel()
    angle = positions.to(torch.float64)[:, None, :, None] * s["freq"]
    c = (angle.cos() * s["amplitude"]).float()
    n = (angle.sin() * (s["amplitude"] * sign)).float()
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([head, rest], -1)


def _keys(pages, table):
    """[B, Hkv, positions, d] in 32 bits: the pages that the tables name, one behind the other."""
    x = pages[table.clamp(min=0).long()].float()
    return x.transpose(1, 2).flatten(2, 3)


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
    k, v = _keys(s["k_pages"], table), _keys(s["v_pages"], table)
    at = P + torch.arange(k.shape[2], device=q.device)
    parts = [_partial(rows, k, v, at <= last, s["scale"])]
    if P:  # every sequence's rows against one copy of the prefix
        k, v = _keys(s["k_pages"], s["prefix_table"][None])[0], _keys(s["v_pages"], s["prefix_table"][None])[0]
        all_rows = rows.transpose(0, 1).reshape(Hkv, B * G * Nq, d)
        ends = last.expand(B, Hkv, G * Nq, 1).transpose(0, 1).reshape(Hkv, B * G * Nq, 1)
        first = _partial(all_rows, k, v, torch.arange(P, device=q.device) <= ends, s["scale"])
        parts.append([x.reshape(Hkv, B, G * Nq, -1).transpose(0, 1) for x in first])
    return _join(parts, (B, Hq, Nq, d))


def _append(s):
    case, table, page = s["case"], s["block_table"], s["case"]["page"]
    lq, lk = s["seqlens_q"].long()[:, None], s["seqlens_k"].long()[:, None]
    t = torch.arange(case["N"], device=table.device)[None]
    place = lk - lq + t
    if s["q_out"] is not None:
        turned = _turn(s["q"], place, s, 1.0).to(torch.bfloat16)
        s["q_out"].copy_(torch.where((t < lq)[:, None, :, None], turned, s["q_out"]))
    # a row behind a sequence's last new token repeats that token: the same value at the same place once more
    t = torch.minimum(t, lq - 1)
    place = lk - lq + t
    b = torch.arange(case["B"], device=table.device)[:, None]
    at, row = table.long()[b, place // page], place % page
    k = _turn(s["k"], lk - lq + torch.arange(case["N"], device=table.device)[None], s, 1.0).to(torch.bfloat16)
    s["k_pages"][at, :, row] = k.transpose(1, 2)[b, t]
    s["v_pages"][at, :, row] = s["v"].transpose(1, 2)[b, t]


def run(state):
    s, case = state, state["case"]
    if own:
        import exact_tiled_attention_18_gb300 as fa
        if case["op"] == "rope":
            call = fa.rope_backward if case["inverse"] else fa.rope_forward
            return call(s["x"], s["turns"], s["positions"], layout=case["layout"], amplitude=s["amplitude"],
                        out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        if case["op"] == "append":
            fa.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seqlens_k"],
                         s["seqlens_q"], turns=s["turns"], layout=case["layout"], amplitude=s["amplitude"],
                         q=s["q"] if case["with_q"] else None, q_out=s["q_out"])
            return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], q=s["q_out"])
        if case["op"] == "paged":
            o, lse = fa.forward_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seqlens_k"],
                                      causal=True, scale=s["scale"], o_dtype=torch.bfloat16)
            return dict(o=o, lse=lse)
        o, lse = fa.forward_shared_prefix(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], case["P"],
                                          s["block_table"], s["seqlens_k"], causal=True, scale=s["scale"],
                                          o_dtype=torch.bfloat16)
        return dict(o=o, lse=lse)
    if case["op"] == "rope":
        y = _turn(s["x"], s["positions"], s, -1.0 if case["inverse"] else 1.0)
        return y.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if case["op"] == "append":
        _append(s)
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], q=s["q_out"])
    o, lse = _attend(s)
    return dict(o=o, lse=lse)


# --------------------------------------------------------------------------------------------- what they cannot avoid

def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["H"] * case["N"]
        size = {"bf16": 2, "fp32": 4}
        return {"bytes": n * d * (size[case["dtype"]] + size[case["out"]]) + case["B"] * case["N"] * 4,
                "flops": 3 * n * case["rot"]}
    Hq, Hkv, B = case["Hq"], case["Hkv"], case["B"]
    if case["op"] == "append":
        tokens = sum(_new_tokens(case))
        turned = Hkv + (Hq if case["with_q"] else 0)
        return {"bytes": 4 * tokens * (turned + Hkv) * d, "flops": 3 * tokens * turned * case["rot"]}
    lens, P, Nq = _spread(case), case.get("P", 0), case["Nq"]
    pairs = sum((P + n) * Nq - Nq * (Nq - 1) // 2 for n in lens)
    rows = B * Hq * Nq
    return {"bytes": 4 * Hkv * d * (P + sum(lens)) + rows * (2 * d + 2 * d + 4), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------------------------------------ the exact values

def _exact_turn(x, positions, case, sign):
    """The rotation as a product of complex numbers in 64 bits."""
    f = _frequencies(case).to(x.device)
    rot = 2 * f.numel()
    theta = positions.double().unsqueeze(-1) * f * sign
    unit = torch.polar(torch.full_like(theta, _amplitude(case)), theta).unsqueeze(1)
    y = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * unit
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"].contiguous(), s["positions"], case, -1.0 if case["inverse"] else 1.0)
    page = case["page"]
    if case["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        qo = s["q_out"].double() if case["with_q"] else None
        for b, (n, total) in enumerate(zip(s["seqlens_q"].tolist(), s["seqlens_k"].tolist())):
            pos = torch.arange(total - n, total, device=kp.device)
            where = s["block_table"][b].long()[torch.div(pos, page, rounding_mode="floor")]
            slot = pos.remainder(page)
            k = _exact_turn(s["k"][b:b + 1, :, :n], pos[None], case, 1.0)[0]
            kp[where, :, slot] = k.permute(1, 0, 2)
            vp[where, :, slot] = s["v"][b, :, :n].double().permute(1, 0, 2)
            if qo is not None:
                qo[b, :, :n] = _exact_turn(s["q"][b:b + 1, :, :n], pos[None], case, 1.0)[0]
        return dict(k_pages=kp, v_pages=vp, q=qo)
    B, Hq, Nq, d = s["q"].shape
    Hkv = case["Hkv"]
    o = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(B, Hq, Nq, dtype=torch.float64, device=s["q"].device)
    for b, total in enumerate(s["seqlens_k"].tolist()):
        named = s["block_table"][b, :(total + page - 1) // page].long()
        sees = torch.arange(total, device=o.device)[None, :] <= torch.arange(total - Nq, total, device=o.device)[:, None]
        for h in range(Hkv):
            group = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            key = s["k_pages"][named, h].reshape(-1, d)[:total].double()
            value = s["v_pages"][named, h].reshape(-1, d)[:total].double()
            logits = torch.einsum("gnd,ld->gnl", s["q"][b, group].double(), key) * s["scale"]
            logits = logits.masked_fill(~sees, -math.inf)
            lse[b, group] = torch.logsumexp(logits, -1)
            o[b, group] = torch.einsum("gnl,ld->gnd", torch.exp(logits - lse[b, group].unsqueeze(-1)), value)
    return dict(o=o, lse=lse)
