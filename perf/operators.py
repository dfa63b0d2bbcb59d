"""Measured cases of the operators around the recurrent layers in one beam-search step.

A decoder that mixes recurrent (KDA) layers with full-attention layers runs, per new token:
rotary positions with the write of keys and values into the paged cache ("rope"), attention of
the new token over that cache ("attention"), the selection of the next beams over the
vocabulary ("beam"), and the copy of recurrent states and cache pages from each beam's parent
("move").  A case is one call of one of these.

``run`` computes the plain form with elementary torch operations where ``own`` is false and
calls the library where it is true; ``exact`` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

HEADS = {"32/8": (32, 8), "16/16": (16, 16), "24/8": (24, 8), "12/1": (12, 1), "8/8": (8, 8), "32/2": (32, 2)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------


def _rope(name, batch, tokens, heads, dim, rot, interleaved, page, far, factor, dtype):
    c = {"op": "rope", "batch": batch, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
         "interleaved": interleaved, "page": page, "far": far, "factor": factor, "dtype": dtype}
    return dict(c, name=name) if name else c


def _attention(name, batch, length, heads, dim, page, window, dtype):
    c = {"op": "attention", "batch": batch, "length": length, "heads": heads, "dim": dim, "page": page,
         "window": window, "dtype": dtype}
    return dict(c, name=name) if name else c


def _beam(name, batch, beams, vocab, out, dtype):
    c = {"op": "beam", "batch": batch, "beams": beams, "vocab": vocab, "out": out, "dtype": dtype}
    return dict(c, name=name) if name else c


def _move(name, rows, beams, what, heads, layers, dtype):
    c = {"op": "move", "rows": rows, "beams": beams, "what": what, "heads": heads, "layers": layers, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a few interactive requests
        _rope("rope-step-small", 4, 1, "32/8", 128, 128, False, 16, 2000, 1.0, "bf16"),
        # a full decode batch late in long documents: interleaved, half of each head rotated, scaled
        _rope("rope-step-far", 384, 1, "24/8", 128, 64, True, 64, 1000000, 8.0, "bf16"),
        # ragged prompts appended in one call
        _rope("rope-prompts", 24, 1500, "32/8", 128, 128, False, 64, 4000, 4.0, "bf16"),
        # one request, short history: latency
        _attention("attend-one", 1, 1000, "32/8", 128, 16, 0, "bf16"),
        # a serving batch of ragged histories
        _attention("attend-batch", 64, 8192, "32/8", 128, 64, 0, "bf16"),
        # two very long documents
        _attention("attend-long", 2, 131072, "32/8", 128, 64, 0, "bf16"),
        # float32 cache, one key head per query head, sliding window, odd page size
        _attention("attend-window-f32", 48, 6000, "16/16", 64, 24, 2048, "f32"),
        # beams of one request
        _beam("beam-one", 1, 4, 32000, 4, "bf16"),
        # a batch with an odd vocabulary, twice as many candidates as beams
        _beam("beam-odd-f32", 12, 6, 50257, 12, "f32"),
        # the largest: many requests, a large vocabulary
        _beam("beam-large", 32, 8, 131072, 8, "bf16"),
        # one request forked into four beams: 12-head bf16 states and conv caches of one layer
        _move("fork-one", 4, 1, "state", 12, 1, "bf16"),
        # reorder of 16 requests x 4 beams: 32-head float32 states and conv caches of four layers
        _move("reorder-states", 16, 4, "state", 32, 4, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "beam", "move"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        tokens = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        batch = max(1, min(_log(rng, 1, 512), 16384 // tokens, 512 * 128 // dim))
        return _rope(None, batch, tokens, rng.choice(["32/8", "16/16", "24/8", "12/1"]), dim,
                     rng.choice([dim, dim // 2, dim // 4]), rng.random() < 0.5, rng.choice([1, 7, 16, 64, 128]),
                     _log(rng, 100, 200000), rng.choice([1.0, 4.0, 32.0]), rng.choice(["bf16", "bf16", "f32"]))
    if op == "attention":
        heads, dim, dtype = rng.choice(["32/8", "16/16", "24/8", "12/1", "32/2"]), rng.choice([64, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
        row = 2 * HEADS[heads][1] * dim * (2 if dtype == "bf16" else 4)
        length = _log(rng, 1, 100000)
        batch = max(1, min(_log(rng, 1, 128), (1 << 30) // (row * length)))
        return _attention(None, batch, length, heads, dim, rng.choice([1, 16, 24, 64, 256]),
                          rng.choice([0, 0, max(1, length // 3)]), dtype)
    if op == "beam":
        vocab = _log(rng, 500, 150000)
        beams = rng.choice([1, 2, 3, 4, 6, 8, 16])
        batch = max(1, min(_log(rng, 1, 64), (1 << 24) // (vocab * beams)))
        return _beam(None, batch, beams, vocab, min(32, beams * rng.choice([1, 2])), rng.choice(["bf16", "f32"]))
    beams = rng.choice([1, 1, 2, 3, 4, 8])
    what, dtype = rng.choice(["state", "pages"]), rng.choice(["bf16", "f32"])
    heads, layers = rng.choice([1, 4, 8, 12]), rng.choice([1, 2, 5])
    return _move(None, max(1, _log(rng, 1, 256) // (beams * layers)), beams, what, heads, layers, dtype)


# ---- inputs ----------------------------------------------------------------------------------


def _fixed(case):
    """What sizes the work (lengths, which slots move) depends on the case alone."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, n, hi):
    r = _fixed(case)
    return [hi] + [r.randint((hi + 3) // 4, hi) for _ in range(n - 1)]


def _table(first, last, page, width, gen):
    """Page table [n, width] whose pages first[i]//page .. last[i]//page are live and in random order, the rest null."""
    live = [(a // page, b // page + 1) if b >= a else (0, 0) for a, b in zip(first, last)]
    count = sum(b - a for a, b in live)
    order = (torch.randperm(count, generator=gen) + 1).to(torch.int32)
    table = torch.zeros(len(first), width, dtype=torch.int32)
    at = 0
    for i, (a, b) in enumerate(live):
        table[i, a:b] = order[at:at + b - a]
        at += b - a
    return table.cuda(), count + 1


def _frequencies(rot, base, factor, original, low, high):
    """Angular frequencies, by parts slowed down for long contexts: those that turn at least `high` times over the
    original length are kept, those that turn at most `low` times are divided by `factor`."""
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    return f * (keep + (1 - keep) / factor)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        (hq, hkv), d, n, dt = HEADS[case["heads"]], case["dim"], case["batch"], DTYPES[case["dtype"]]
        new = _lengths(case, n, case["tokens"])
        r = _fixed(case)
        start = [r.randint(0, case["far"]) for _ in range(n)]
        total = [a + b for a, b in zip(start, new)]
        rows, page = sum(new), case["page"]
        table, pages = _table(start, [x - 1 for x in total], page, -(-max(total) // page), host)
        proj = normal(rows, (hq + 2 * hkv) * d, dtype=dt)  # one packed projection row per token
        s["q"] = proj[:, :hq * d].view(rows, hq, d)
        s["k"] = proj[:, hq * d:(hq + hkv) * d].view(rows, hkv, d)
        s["v"] = proj[:, (hq + hkv) * d:].view(rows, hkv, d)
        s["freq"] = _frequencies(case["rot"], 10000.0, case["factor"], 4096, 1.0, 32.0).cuda()
        # the library takes a frequency as a step of turns per position, in 64 bits of fixed point
        s["steps"] = torch.round(s["freq"] * (2.0 ** 64 / (2 * math.pi))).to(torch.int64).view(torch.int32).view(-1, 2)
        s["amplitude"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        s["cu"] = None
        if case["tokens"] > 1:
            s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        s["table"] = table
        s["k_pages"] = normal(pages, page, hkv, d, dtype=dt)
        s["v_pages"] = normal(pages, page, hkv, d, dtype=dt)
    elif case["op"] == "attention":
        (hq, hkv), d, n, dt, page = HEADS[case["heads"]], case["dim"], case["batch"], DTYPES[case["dtype"]], case["page"]
        lens = _lengths(case, n, case["length"])
        table, pages = _table([0] * n, [x - 1 for x in lens], page, -(-max(lens) // page), host)
        s["q"] = normal(n, hq, d, dtype=dt)
        s["k_pages"] = normal(pages, page, hkv, d, dtype=dt)
        s["v_pages"] = normal(pages, page, hkv, d, dtype=dt)
        s["table"] = table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    elif case["op"] == "beam":
        n, b, v = case["batch"], case["beams"], case["vocab"]
        s["logits"] = (2.5 * normal(n, b, v)).to(DTYPES[case["dtype"]])
        s["scores"] = -12.0 + 1.5 * normal(n, b)
        s["finished"] = (torch.rand(n, b, generator=gen, device="cuda") < 0.1).to(torch.int32)
        s["eos"] = 2
    else:
        rows, b, h, dt = case["rows"], case["beams"], case["heads"], DTYPES[case["dtype"]]
        slots = 2 * rows * b + 2
        if case["what"] == "state":  # recurrent states and width-4 conv caches of q, k and v
            shapes = [((slots, h, 128, 128), dt), ((slots, 9 * h * 128), torch.bfloat16)]
        else:  # pages of 64 tokens of keys and of values
            shapes = [((slots, 64, h, 128), dt), ((slots, 64, h, 128), dt)]
        s["pools"] = [normal(*shape, dtype=t) for _ in range(case["layers"]) for shape, t in shapes]
        order = (torch.randperm(slots - 1, generator=host) + 1).to(torch.int32)
        mine, other = order[:rows * b].view(rows, b), order[rows * b:2 * rows * b].view(rows, b)
        parents = _parents(case)
        if b > 1:  # each request's beams take their parents' slots over, in place
            s["src"], s["dst"], s["parents"] = mine, mine, torch.tensor(parents, dtype=torch.int32)
        else:  # fork or compaction: from one slot to a free one; a parent of -1 clears the slot for a new request
            s["src"] = torch.where(torch.tensor(parents) < 0, 0, mine if rows > 4 else mine[:1].expand(rows, 1)).to(torch.int32)
            s["dst"], s["parents"] = other, None
        for k in ("src", "dst", "parents"):
            s[k] = None if s[k] is None else s[k].contiguous().cuda()
    return s


def _parents(case):
    """Parent beam of every beam; now and then -1, a beam that has none.  The first beam always has another for its parent."""
    r = _fixed(case)
    parents = [[r.randrange(case["beams"]) if r.random() > 0.05 else -1 for _ in range(case["beams"])]
               for _ in range(case["rows"])]
    parents[0][0] = case["beams"] - 1
    return parents


# ---- the plain forms ---------------------------------------------------------------------------


def _plain_rope(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    rows, rot, page = q.shape[0], case["rot"], case["page"]
    n = s["lens"].shape[0]
    cu = s["cu"] if s["cu"] is not None else torch.arange(n + 1, device="cuda", dtype=torch.int32)
    row = torch.arange(rows, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    pos = (s["lens"][seq] - cu[seq + 1] + row).long()
    angle = pos.double()[:, None] * s["freq"][None, :]
    cos = (s["amplitude"] * angle.cos()).float()[:, None, :]
    sin = (s["amplitude"] * angle.sin()).float()[:, None, :]

    def turned(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., :rot:2], x[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([r, x[..., rot:]], -1)

    live = s["table"][seq, pos // page].long()
    s["k_pages"][live, pos % page] = turned(k).to(s["k_pages"].dtype)
    s["v_pages"][live, pos % page] = v.to(s["v_pages"].dtype)
    return {"q": turned(q).to(q.dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attention(s):
    case, q = s["case"], s["q"].float()
    n, hq, d = q.shape
    hkv, page = s["k_pages"].shape[2], case["page"]
    table = s["table"].long()
    length = table.shape[1] * page
    k = s["k_pages"][table].view(n, length, hkv, d).transpose(1, 2).float()
    v = s["v_pages"][table].view(n, length, hkv, d).transpose(1, 2).float()
    scores = torch.matmul(q.view(n, hkv, hq // hkv, d), k.transpose(2, 3)) * d ** -0.5
    at = torch.arange(length, device="cuda")[None, :]
    live = (at < s["lens"][:, None]) & (table > 0).repeat_interleave(page, 1)
    if case["window"]:
        live &= at >= s["lens"][:, None] - case["window"]
    scores = scores.masked_fill(~live[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total
    return {"out": out.view(n, hq, d).to(torch.bfloat16), "lse": (top + total.log()).view(n, hq)}


def _plain_beam(s):
    case, x = s["case"], s["logits"].double()  # which of two close candidates wins needs 64 bits
    n, b, v = x.shape
    top = x.amax(-1, keepdim=True)
    c = x - top - (x - top).exp().sum(-1, keepdim=True).log() + s["scores"].double()[..., None]
    done = s["finished"][..., None] != 0
    only = torch.arange(v, device="cuda") == s["eos"]
    c = torch.where(done, torch.where(only, s["scores"].double()[..., None], -math.inf), c).view(n, b * v)
    value, at = torch.sort(c, dim=-1, descending=True, stable=True)  # ties: the lowest beam and token first
    value, at = value[:, :case["out"]], at[:, :case["out"]]
    none = value == -math.inf
    return {"scores": value.float(), "parents": torch.where(none, -1, at // v).to(torch.int32),
            "tokens": torch.where(none, -1, at % v).to(torch.int32)}


def _plain_move(s):
    src, dst = s["src"].long(), s["dst"].long()
    if s["parents"] is not None:
        held = s["parents"] < 0
        src = torch.gather(src, 1, s["parents"].long().clamp(min=0))
        src, dst = torch.where(held, dst, src), dst  # a beam without a parent keeps its slot
    src, dst = src.flatten(), dst.flatten()

    def moved(pool):
        values = pool[src]
        values *= (src > 0).to(pool.dtype).view(-1, *[1] * (pool.dim() - 1))
        pool[dst] = values
        return pool

    return list(map(moved, s["pools"]))


# ---- one pass ------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attention": _own_attention, "beam": _own_beam, "move": _own_move}[op](state)
    return {"rope": _plain_rope, "attention": _plain_attention, "beam": _plain_beam, "move": _plain_move}[op](state)


def _own_rope(s):
    import linear_attention_decode_02_gb300 as kda
    q = kda.kda_rope_append(s["q"], s["k"], s["v"], s["steps"], s["lens"], s["table"], s["k_pages"], s["v_pages"],
                            cu_seqlens=s["cu"], interleaved=s["case"]["interleaved"], amplitude=s["amplitude"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_attention(s):
    import linear_attention_decode_02_gb300 as kda
    out, lse = kda.kda_paged_attention_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                              window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_beam(s):
    import linear_attention_decode_02_gb300 as kda
    scores, parents, tokens = kda.kda_beam_select(s["logits"], s["scores"], s["case"]["out"], finished=s["finished"],
                                                  eos_token=s["eos"])
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _own_move(s):
    import linear_attention_decode_02_gb300 as kda
    kda.kda_pool_move(s["pools"], s["src"], s["dst"], parents=s["parents"])
    return s["pools"]


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    if case["op"] == "rope":
        (hq, hkv), d = HEADS[case["heads"]], case["dim"]
        rows = sum(_lengths(case, case["batch"], case["tokens"]))
        return {"bytes": 2 * rows * (hq + 2 * hkv) * d * DTYPES[case["dtype"]].itemsize,
                "flops": 3 * rows * (hq + hkv) * case["rot"]}
    if case["op"] == "attention":
        (hq, hkv), d, size = HEADS[case["heads"]], case["dim"], DTYPES[case["dtype"]].itemsize
        live = sum(min(x, case["window"] or x) for x in _lengths(case, case["batch"], case["length"]))
        return {"bytes": 2 * live * hkv * d * size + case["batch"] * hq * (d * (size + 2) + 4),
                "flops": 4 * live * hq * d}
    if case["op"] == "beam":
        count = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": count * DTYPES[case["dtype"]].itemsize, "flops": 4 * count}
    slot = 128 * 128 * case["heads"] * DTYPES[case["dtype"]].itemsize + 9 * case["heads"] * 128 * 2
    if case["what"] == "pages":
        slot = 2 * 64 * 128 * case["heads"] * DTYPES[case["dtype"]].itemsize
    read = written = 0
    for i, row in enumerate(_parents(case)):
        if case["beams"] > 1:
            real = [(p, j) for j, p in enumerate(row) if p >= 0 and p != j]
            read, written = read + len({p for p, _ in real}), written + len(real)
        else:
            written += 1
            read += row[0] >= 0 and (case["rows"] > 4 or i == 0)
    return {"bytes": case["layers"] * slot * (read + written), "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "beam":
        return _exact_beam(s)
    return _exact_move(s)


def _exact_rope(s):
    case, page, rot = s["case"], s["case"]["page"], s["case"]["rot"]
    k_pages, v_pages, q_out = s["k_pages"].double(), s["v_pages"].double(), s["q"].double()
    lens = s["lens"].tolist()
    begin = s["cu"].tolist() if s["cu"] is not None else list(range(len(lens) + 1))
    where = torch.cat([torch.arange(lens[i] - (begin[i + 1] - begin[i]), lens[i]) for i in range(len(lens))]).cuda()
    owner = torch.cat([torch.full((begin[i + 1] - begin[i],), i) for i in range(len(lens))]).cuda()
    turn = torch.polar(torch.full((1,), s["amplitude"], dtype=torch.float64, device="cuda"),
                       torch.outer(where.double(), s["freq"]))[:, None, :]

    def rotated(x):
        y = x.double().clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    q_out = rotated(s["q"])
    index = s["table"].long()[owner, where // page] * page + where % page
    k_pages.view(-1, *k_pages.shape[2:]).index_copy_(0, index, rotated(s["k"]))
    v_pages.view(-1, *v_pages.shape[2:]).index_copy_(0, index, s["v"].double())
    return {"q": q_out, "k_pages": k_pages, "v_pages": v_pages}


def _exact_attention(s):
    case, page = s["case"], s["case"]["page"]
    n, hq, d = s["q"].shape
    hkv = s["k_pages"].shape[2]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        first = max(0, length - case["window"]) if case["window"] else 0
        at = torch.arange(first, length, device="cuda")
        index = s["table"][i].long()[at // page] * page + at % page
        for h in range(hkv):
            q = s["q"][i].double().view(hkv, hq // hkv, d)[h]
            k = s["k_pages"].view(-1, hkv, d)[index, h].double()
            v = s["v_pages"].view(-1, hkv, d)[index, h].double()
            logits = q @ k.T / math.sqrt(d)
            total = torch.logsumexp(logits, 1)
            rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            lse[i, rows] = total
            out[i, rows] = torch.exp(logits - total[:, None]) @ v
    return {"out": out, "lse": lse}


def _exact_beam(s):
    case, values = s["case"], []
    n, b, v = s["logits"].shape
    for i in range(n):
        c = torch.log_softmax(s["logits"][i].double(), -1) + s["scores"][i].double()[:, None]
        for j in range(b):
            if int(s["finished"][i, j]):
                c[j] = -math.inf
                c[j, s["eos"]] = s["scores"][i, j].double()
        best = torch.full((case["out"],), -math.inf, dtype=torch.float64, device="cuda")
        m = min(case["out"], b * v)
        best[:m] = torch.topk(c.flatten(), m).values
        values.append(best)
    return {"scores": torch.stack(values), "parents": None, "tokens": None}


def _exact_move(s):
    pools = [p.double() for p in s["pools"]]
    src, dst = s["src"].tolist(), s["dst"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else [[0]] * len(src)
    for old, new in zip(s["pools"], pools):
        for n, row in enumerate(parents):
            for j, p in enumerate(row):
                if p >= 0:
                    new[dst[n][j]] = old[src[n][p]].double() if src[n][p] > 0 else 0.0
    return pools
