"""Measured cases of the operators that give sequences their pages, place image and video tokens in them, and let
sequences share a prompt.

A decoder that mixes recurrent (KDA) layers with full-attention layers keeps keys and values in pages.  Before a step
the pages of every sequence are made to fit its new length, and each new token row is told its place ("pages"); the new
queries and keys are turned by their position in time, height and width and the keys and values written to those places
("axes"); and sequences that begin alike, the beams of one request or the users of one system prompt, attend to the
common part of the cache together and to their own part alone ("prefix").  A case is one call of one of these.

``run`` computes the plain form with elementary torch operations where ``own`` is false and calls the library where it
is true; ``exact`` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

HEADS = {"32/8": (32, 8), "16/16": (16, 16), "24/8": (24, 8), "12/1": (12, 1), "32/2": (32, 2)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------


def _pages(name, kind, batch, length, tokens, page):
    c = {"op": "pages", "kind": kind, "batch": batch, "length": length, "tokens": tokens, "page": page}
    return dict(c, name=name) if name else c


def _axes(name, kind, batch, tokens, heads, dim, rot, interleaved, cyclic, page, dtype):
    c = {"op": "axes", "kind": kind, "batch": batch, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
         "interleaved": interleaved, "cyclic": cyclic, "page": page, "dtype": dtype}
    return dict(c, name=name) if name else c


def _prefix(name, groups, beams, prefix, tail, heads, dim, page, window, dtype):
    c = {"op": "prefix", "groups": groups, "beams": beams, "prefix": prefix, "tail": tail, "heads": heads, "dim": dim,
         "page": page, "window": window, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a few interactive requests
        _pages("pages-step-small", "step", 8, 3000, 1, 16),
        # a full decode batch: most requests grow by a token, some have ended, some drop rejected speculative tokens
        _pages("pages-step-full", "mixed", 512, 20000, 4, 16),
        # many long prompts admitted at once
        _pages("pages-prompts", "prompt", 48, 16384, 16384, 64),
        # decode rows of a conversation about pictures
        _axes("axes-step", "text", 16, 1, "32/8", 128, 128, False, False, 16, "bf16"),
        # one picture of 37 x 51 patches and its question
        _axes("axes-image", "image", 1, 1900, "32/8", 128, 128, False, False, 64, "bf16"),
        # a batch of clips: axes in turn over the pairs, half of each head
        _axes("axes-video", "video", 12, 2900, "24/8", 128, 64, True, True, 64, "bf16"),
        # float32 cache, one key head per query head, odd page size
        _axes("axes-image-f32", "image", 5, 777, "16/16", 64, 64, False, True, 24, "f32"),
        # one request of four beams, short prompt: latency
        _prefix("prefix-one", 1, 4, 1000, 40, "32/8", 128, 16, 0, "bf16"),
        # sixteen requests of four beams after long prompts
        _prefix("prefix-beams", 16, 4, 8192, 300, "32/8", 128, 64, 0, "bf16"),
        # the largest: a batch under one long system prompt
        _prefix("prefix-system", 1, 256, 32768, 600, "32/8", 128, 64, 0, "bf16"),
        # prompts of different few-shot tasks, narrow heads, one key head
        _prefix("prefix-tasks", 7, 20, 6000, 500, "12/1", 64, 24, 0, "bf16"),
        # float32 cache, beams
        _prefix("prefix-beams-f32", 6, 6, 5000, 100, "16/16", 64, 16, 0, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "axes", "prefix", "prefix"])
    if op == "pages":
        kind = rng.choice(["step", "mixed", "prompt"])
        length = _log(rng, 10, 60000)
        batch = max(1, min(_log(rng, 1, 2000), 700000 // length if kind == "prompt" else 16000000 // length))
        return _pages(None, kind, batch, length, length if kind == "prompt" else _log(rng, 1, 9),
                      rng.choice([1, 7, 16, 64, 128]))
    if op == "axes":
        dim, dtype = rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
        kind = rng.choice(["text", "image", "video"])
        tokens = 1 if kind == "text" else _log(rng, 20, 5000)
        batch = max(1, min(_log(rng, 1, 256), 8000 * 128 // (tokens * dim)))
        return _axes(None, kind, batch, tokens, rng.choice(["32/8", "16/16", "24/8", "12/1"]), dim,
                     rng.choice([dim, dim // 2, dim // 4]), rng.random() < 0.5, rng.random() < 0.5,
                     rng.choice([1, 7, 16, 64, 128]), dtype)
    heads, dim, dtype = rng.choice(["32/8", "16/16", "24/8", "12/1", "32/2"]), rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    hq, hkv = HEADS[heads]
    row = 2 * hkv * dim * DTYPES[dtype].itemsize
    prefix, tail, beams = _log(rng, 1, 40000), _log(rng, 1, 1500), _log(rng, 1, 128)
    groups = max(1, min(_log(rng, 1, 40), (1 << 29) // (row * (prefix + beams * tail)),
                        (1 << 35) // (beams * hq * dim * (prefix + tail))))
    beams = max(1, min(beams, (1 << 29) // (row * tail), (1 << 35) // (groups * hq * dim * (prefix + tail))))
    return _prefix(None, groups, beams, prefix, tail, heads, dim, rng.choice([1, 16, 24, 64, 256]),
                   rng.choice([0, 0, 0, prefix + tail // 2 + 1]), dtype)


# ---- inputs ----------------------------------------------------------------------------------


def _fixed(case):
    """What sizes the work (lengths, group sizes) depends on the case alone."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, n, hi):
    r = _fixed(case)
    return [hi] + [r.randint((hi + 3) // 4, hi) for _ in range(n - 1)]


def _growth(case):
    """(lengths now, lengths wanted) of every sequence."""
    r, n, hi = _fixed(case), case["batch"], case["length"]
    old, new = [], []
    for length in _lengths(case, n, hi):
        what = r.random()
        if case["kind"] == "prompt":
            a, b = 0, length
        elif case["kind"] == "step" or what < 0.8:
            a, b = length, length + r.randint(1, case["tokens"])
        elif what < 0.9:  # drafted tokens that were not accepted
            a, b = length, max(0, length - r.randint(1, case["tokens"]))
        elif what < 0.95:  # has ended
            a, b = length, 0
        else:  # takes the place of one that has
            a, b = 0, max(1, length // 8)
        old.append(a)
        new.append(b)
    return old, new


def _grid(case):
    """(time, height, width) of every token row of every sequence: text counts on all axes alike, pictures and clips
    keep the first position of theirs in time and spread over height and width."""
    r, rows = _fixed(case), []
    for n in _lengths(case, case["batch"], case["tokens"]):
        at = r.randint(0, 30000)
        if case["kind"] == "text":
            rows.append([(at + i,) * 3 for i in range(n)])
            continue
        frames = 1 if case["kind"] == "image" else max(1, min(16, n // 40))
        wide = max(1, int(math.sqrt(1.4 * n / frames)))
        tall = max(1, n // (frames * wide))
        seen = [(at + f, at + y, at + x) for f in range(frames) for y in range(tall) for x in range(wide)][:n]
        last = at + max(frames, tall, wide)
        rows.append(seen + [(last + i,) * 3 for i in range(n - len(seen))])
    return rows


def _sections(rot):
    """Pairs turned by time, height and width: a quarter and three eighths twice."""
    half = rot // 2
    other = 3 * half // 8
    return [half - 2 * other, other, other]


def _pair_axes(rot, cyclic):
    left, axes = _sections(rot), []
    if not cyclic:
        return [a for a, n in enumerate(left) for _ in range(n)]
    while len(axes) < rot // 2:
        for a in range(3):
            if left[a] > 0:
                left[a] -= 1
                axes.append(a)
    return axes


def _groups(case):
    """Sequences of every group, length of its prefix and of every sequence."""
    r, g = _fixed(case), case["groups"]
    sizes = [case["beams"]] + [r.randint((case["beams"] + 1) // 2, case["beams"]) for _ in range(g - 1)]
    prefixes = [case["prefix"]] + [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(g - 1)]
    if r.random() < 0.5:  # a prefix cache that shares whole pages
        prefixes = [max(case["page"], p // case["page"] * case["page"]) for p in prefixes]
    lens = [p + r.randint(1, case["tail"]) for p, n in zip(prefixes, sizes) for _ in range(n)]
    return sizes, prefixes, lens


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.as_tensor(values, dtype=torch.int32).contiguous().cuda()

    s = {"case": case}
    page = case["page"]
    if case["op"] == "pages":
        old, new = _growth(case)
        held = [-(-x // page) for x in old]
        width = max(-(-max(a, b) // page) for a, b in zip(old, new)) + 3
        # a sixteenth of the pages is free beyond what the step needs
        need = sum(max(0, -(-b // page) - h) for b, h in zip(new, held))
        count = sum(held) + need + need // 16 + 5
        order = (torch.randperm(count, generator=host) + 1).to(torch.int32)
        table = torch.zeros(case["batch"], width, dtype=torch.int32)
        col = torch.arange(width)[None, :]
        live = col < torch.tensor(held)[:, None]
        table[live] = order[:sum(held)]
        head = int(torch.randint(0, count, (1,), generator=host))
        free = count - sum(held)
        ring = torch.zeros(count, dtype=torch.int32)
        ring[(head + torch.arange(free)) % count] = order[sum(held):]
        s["table"], s["free"], s["state"] = table.cuda(), ring.cuda(), ints([head, free])
        s["old"], s["new"] = ints(old), ints(new)
        s["rows"] = sum(max(0, b - a) for a, b in zip(old, new)) + 7  # a padded batch
    elif case["op"] == "axes":
        (hq, hkv), d, dt, rot = HEADS[case["heads"]], case["dim"], DTYPES[case["dtype"]], case["rot"]
        grid = _grid(case)
        rows = sum(len(g) for g in grid)
        s["positions"] = ints([p for g in grid for p in g])
        pages = -(-rows // page) + case["batch"] + 1
        proj = normal(rows, (hq + 2 * hkv) * d, dtype=dt)  # one packed projection row per token
        s["q"] = proj[:, :hq * d].view(rows, hq, d)
        s["k"] = proj[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
        s["v"] = proj[:, (hq + hkv) * d:].view(rows, hkv, d)
        # rows lie one after another on shuffled pages
        order = torch.randperm(pages - 1, generator=host) + 1
        row = torch.arange(rows)
        s["slots"] = ints(order[row // page] * page + row % page)
        freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
        s["freq"] = freq.cuda()
        # the library takes a frequency as a step of turns per position, in 64 bits of fixed point
        s["steps"] = torch.round(freq * (2.0 ** 64 / (2 * math.pi))).to(torch.int64).view(torch.int32).view(-1, 2).cuda()
        s["axes"] = ints(_pair_axes(rot, case["cyclic"]))
        s["k_pages"] = normal(pages, page, hkv, d, dtype=dt)
        s["v_pages"] = normal(pages, page, hkv, d, dtype=dt)
    else:
        (hq, hkv), d, dt = HEADS[case["heads"]], case["dim"], DTYPES[case["dtype"]]
        sizes, prefixes, lens = _groups(case)
        n = len(lens)
        width = -(-max(lens) // page)
        table = torch.zeros(n, width, dtype=torch.int32)
        whole = [p // page for p in prefixes]  # pages that the group shares
        ends = [-(-x // page) for x in lens]
        at, total = 0, sum(whole) + sum(ends[i] - whole[g] for g, i in _members(sizes))
        order = (torch.randperm(total, generator=host) + 1).to(torch.int32)
        for g, first in enumerate(_starts(sizes)[:-1]):
            table[first:first + sizes[g], :whole[g]] = order[at:at + whole[g]]
            at += whole[g]
        for g, i in _members(sizes):
            table[i, whole[g]:ends[i]] = order[at:at + ends[i] - whole[g]]
            at += ends[i] - whole[g]
        s["k_pages"] = normal(total + 1, page, hkv, d, dtype=dt)
        s["v_pages"] = normal(total + 1, page, hkv, d, dtype=dt)
        # a prefix that ends inside a page: every sequence has a copy of that page's first part
        src, dst, keep = [], [], []
        for g, i in _members(sizes):
            if prefixes[g] % page and i != _starts(sizes)[g]:
                src.append(int(table[_starts(sizes)[g], whole[g]]))
                dst.append(int(table[i, whole[g]]))
                keep.append(prefixes[g] % page)
        if src:
            src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
            some = (torch.arange(page, device="cuda")[None, :] < torch.tensor(keep, device="cuda")[:, None])[..., None, None]
            for pool in (s["k_pages"], s["v_pages"]):
                pool[dst] = torch.where(some, pool[src], pool[dst])
        s["q"] = normal(n, hq, d, dtype=dt)
        s["table"], s["lens"] = table.cuda(), ints(lens)
        s["starts"], s["prefixes"] = ints(_starts(sizes)), ints(prefixes)
        s["host"] = (sizes, prefixes, lens)  # a scheduler knows its requests
    return s


def _starts(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


def _members(sizes):
    return [(g, i) for g, (a, b) in enumerate(zip(_starts(sizes), _starts(sizes)[1:])) for i in range(a, b)]


# ---- the plain forms ---------------------------------------------------------------------------


def _plain_pages(s):
    page, table, ring = s["case"]["page"], s["table"], s["free"]
    old, new = s["old"].long(), s["new"].long()
    n, width = table.shape
    size = ring.shape[0]
    head, count = s["state"][0].long(), s["state"][1].long()
    held, want = -(-old // page), -(-new // page)
    take = (want - held).clamp(min=0)
    through = take.cumsum(0)
    granted = (take == 0) | (through <= count)
    lens = torch.where(granted, new, old)
    take = torch.where(granted, take, 0)
    base = take.cumsum(0) - take
    col = torch.arange(width, device="cuda")[None, :]
    fresh = granted[:, None] & (col >= held[:, None]) & (col < want[:, None])
    given = ring[(head + base[:, None] + col - held[:, None]) % size]
    gone = (col >= want[:, None]) & (col < held[:, None]) & (table > 0) & (table <= size)
    place = gone.flatten().cumsum(0) - 1
    released = gone.sum()
    spill = torch.cat([ring, ring[:1]])  # one place more, for what is not released
    spill[torch.where(gone.flatten(), (head + count + place) % size, size)] = table.flatten()
    ring.copy_(spill[:-1])
    table.copy_(torch.where(fresh, given, table))
    rows = (lens - old).clamp(min=0)
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = torch.where(real, old[seq] + row - cu[seq], 0)
    slots = torch.where(real, table[seq, pos // page].long() * page + pos % page, -1)
    state = torch.stack([(head + take.sum()) % size, count - take.sum() + released])
    return {"lens": lens.to(torch.int32), "state": state.to(torch.int32), "cu": cu.to(torch.int32),
            "slots": slots.to(torch.int32), "table": table, "free": ring}


def _plain_axes(s):
    case, rot, page = s["case"], s["case"]["rot"], s["case"]["page"]
    where = s["positions"][:, s["axes"].long()].double()
    angle = where * s["freq"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turned(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., :rot:2], x[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([r, x[..., rot:]], -1)

    slots = s["slots"].long()
    s["k_pages"][slots // page, slots % page] = turned(s["k"]).to(s["k_pages"].dtype)
    s["v_pages"][slots // page, slots % page] = s["v"].to(s["v_pages"].dtype)
    return {"q": turned(s["q"]).to(s["q"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_prefix(s):
    case, page = s["case"], s["case"]["page"]
    n, hq, d = s["q"].shape
    hkv = s["k_pages"].shape[2]
    per, scale = hq // hkv, d ** -0.5
    sizes, prefixes, lens = s["host"]
    out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, hq, dtype=torch.float32, device="cuda")
    for g, a in enumerate(_starts(sizes)[:-1]):
        b, p = a + sizes[g], prefixes[g]
        rows, first, last = b - a, p // page, -(-max(lens[a:b]) // page)
        q = s["q"][a:b].float().view(rows, hkv, per, d)
        shared = s["table"][a, :-(-p // page)].long()
        k = s["k_pages"][shared].view(-1, hkv, d)[:p].permute(1, 2, 0).float()
        v = s["v_pages"][shared].view(-1, hkv, d)[:p].transpose(0, 1).float()
        # the common part, all rows of the group against it
        x = torch.matmul(q.transpose(0, 1).reshape(hkv, rows * per, d), k) * scale
        at = torch.arange(p, device="cuda")
        if case["window"]:
            hidden = at[None, :] < (s["lens"][a:b, None] - case["window"])
            x = x.view(hkv, rows, per, p).masked_fill(hidden[None, :, None, :], -math.inf).view(hkv, rows * per, p)
        # each row's own part
        own_pages = s["table"][a:b, first:last].long()
        ko = s["k_pages"][own_pages].view(rows, -1, hkv, d).permute(0, 2, 3, 1).float()
        vo = s["v_pages"][own_pages].view(rows, -1, hkv, d).transpose(1, 2).float()
        y = torch.matmul(q, ko) * scale
        at = torch.arange(first * page, last * page, device="cuda")[None, :]
        live = (at >= p) & (at < s["lens"][a:b, None])
        if case["window"]:
            live &= at >= s["lens"][a:b, None] - case["window"]
        y = y.masked_fill(~live[:, None, None, :], -math.inf)
        x = x.view(hkv, rows, per, p).transpose(0, 1)
        top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        x, y = torch.exp(x - top), torch.exp(y - top)
        total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.matmul(x.transpose(0, 1).reshape(hkv, rows * per, p), v).view(hkv, rows, per, d).transpose(0, 1)
        o = (o + torch.matmul(y, vo)) / total
        out[a:b] = o.reshape(rows, hq, d).to(torch.bfloat16)
        lse[a:b] = (top + total.log()).view(rows, hq)
    return {"out": out, "lse": lse}


# ---- one pass ------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"pages": _own_pages, "axes": _own_axes, "prefix": _own_prefix}[op](state)
    return {"pages": _plain_pages, "axes": _plain_axes, "prefix": _plain_prefix}[op](state)


def _own_pages(s):
    import linear_attention_decode_02_gb300 as kda
    lens, state, cu, slots = kda.kda_page_assign(s["old"], s["new"], s["table"], s["free"], s["state"],
                                                 s["case"]["page"], s["rows"])
    return {"lens": lens, "state": state, "cu": cu, "slots": slots, "table": s["table"], "free": s["free"]}


def _own_axes(s):
    import linear_attention_decode_02_gb300 as kda
    q = kda.kda_rope_axes_append(s["q"], s["k"], s["v"], s["steps"], s["axes"], s["positions"], s["slots"],
                                 s["k_pages"], s["v_pages"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_prefix(s):
    import linear_attention_decode_02_gb300 as kda
    out, lse = kda.kda_prefix_attention_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["starts"],
                                               s["prefixes"], window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    page = case["page"]
    if case["op"] == "pages":
        old, new = _growth(case)
        moved = sum(abs(-(-b // page) - -(-a // page)) for a, b in zip(old, new))
        rows = sum(max(0, b - a) for a, b in zip(old, new)) + 7
        return {"bytes": 4 * (4 * case["batch"] + 2 * moved + rows), "flops": 0}
    if case["op"] == "axes":
        (hq, hkv), d = HEADS[case["heads"]], case["dim"]
        rows = sum(_lengths(case, case["batch"], case["tokens"]))
        return {"bytes": rows * (2 * (hq + 2 * hkv) * d * DTYPES[case["dtype"]].itemsize + 16),
                "flops": 3 * rows * (hq + hkv) * case["rot"]}
    (hq, hkv), d, size = HEADS[case["heads"]], case["dim"], DTYPES[case["dtype"]].itemsize
    sizes, prefixes, lens = _groups(case)
    seen = [min(x, case["window"] or x) for x in lens]
    shared = sum(min(p, max(seen[i] - lens[i] + p for i in range(a, a + n)))
                 for p, n, a in zip(prefixes, sizes, _starts(sizes)))
    tails = sum(min(seen[i], lens[i] - prefixes[g]) for g, i in _members(sizes))
    return {"bytes": 2 * (shared + tails) * hkv * d * size + len(lens) * hq * (d * (size + 2) + 4),
            "flops": 4 * sum(seen) * hq * d}


# ---- the definition in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(s)
    if case["op"] == "axes":
        return _exact_axes(s)
    return _exact_prefix(s)


def _exact_pages(s):
    page, rows = s["case"]["page"], s["rows"]
    table, ring = s["table"].cpu(), s["free"].tolist()
    head, count = s["state"].tolist()
    lens, cu, places, taken, back, asked = [], [0], [], 0, [], 0
    for i, (a, b) in enumerate(zip(s["old"].tolist(), s["new"].tolist())):
        held, want = (a + page - 1) // page, (b + page - 1) // page
        asked += max(0, want - held)
        if want > held and asked > count:
            b = a
        elif want > held:
            table[i, held:want] = torch.tensor([ring[(head + taken + j) % len(ring)] for j in range(want - held)],
                                               dtype=torch.int32)
            taken += want - held
        else:
            back += [p for p in table[i, want:held].tolist() if 1 <= p <= len(ring)]
        lens.append(b)
        cu.append(cu[-1] + max(0, b - a))
        at = torch.arange(a, max(a, b))
        places.append(table[i].long()[at // page] * page + at % page)
    for j, p in enumerate(back):
        ring[(head + count + j) % len(ring)] = p
    places.append(torch.full((rows - cu[-1],), -1))
    values = {"lens": lens, "state": [(head + taken) % len(ring), count - taken + len(back)], "cu": cu,
              "slots": torch.cat(places), "table": table, "free": ring}
    return {k: torch.as_tensor(v).to(torch.int32).cuda() for k, v in values.items()}


def _exact_axes(s):
    rot, page = s["case"]["rot"], s["case"]["page"]
    angle = torch.stack([s["positions"][:, a].double() * f for a, f in zip(s["axes"].tolist(), s["freq"].unbind())], 1)
    turn = torch.complex(torch.cos(angle), torch.sin(angle))[:, None, :]

    def rotated(x):
        y = x.double().clone()
        if s["case"]["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    k_pages, v_pages, slots = s["k_pages"].double(), s["v_pages"].double(), s["slots"].long()
    k_pages.view(-1, *k_pages.shape[2:]).index_copy_(0, slots, rotated(s["k"]))
    v_pages.view(-1, *v_pages.shape[2:]).index_copy_(0, slots, s["v"].double())
    return {"q": rotated(s["q"]), "k_pages": k_pages, "v_pages": v_pages}


def _exact_prefix(s):
    """Every sequence alone, over the whole of its pages."""
    case, page = s["case"], s["case"]["page"]
    n, hq, d = s["q"].shape
    hkv = s["k_pages"].shape[2]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["host"][2]):
        first = max(0, length - case["window"]) if case["window"] else 0
        at = torch.arange(first, length, device="cuda")
        index = s["table"][i].long()[at // page] * page + at % page
        k = s["k_pages"].view(-1, hkv, d)[index].double().permute(1, 2, 0)
        v = s["v_pages"].view(-1, hkv, d)[index].double().transpose(0, 1)
        logits = torch.matmul(s["q"][i].double().view(hkv, hq // hkv, d), k) / math.sqrt(d)
        total = torch.logsumexp(logits, -1, keepdim=True)
        lse[i] = total.flatten()
        out[i] = torch.matmul(torch.exp(logits - total), v).reshape(hq, d)
    return {"out": out, "lse": lse}
